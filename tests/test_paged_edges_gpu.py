"""Edges of the paged cache's calls on the GPU: workspaces of other batches, infinite
sinks, queries and latents, empty sequences in between, and what hidden keys and bad
queries do in each of the attend kernels."""

import numpy as np
import pytest
import torch

import oracle
import sparse_mla_decode_csr_gb300 as smla
from smla_testlib import allowance, bits
from test_paged_gpu import DEV, REC, Batch, attend, check, expect_records, gen, reference, reference_operands, unpack

pytestmark = pytest.mark.gpu

# heads of single tokens that take each kernel: the few-row kernel, narrow tiles of 32
# and 64 rows, pairs of CTAs
KERNELS = {"few": 16, "narrow32": 32, "narrow64": 64, "pair": 128}


# ---- workspaces ----


@pytest.mark.parametrize("heads", [1, 16, 40, 128])
def test_the_workspace_never_grows_when_a_size_shrinks(heads):
    base = dict(n_rows=4096, n_seqs=64, page_size=64, max_pages=128)
    for name, sizes in (("n_rows", [1, 2, 3, 31, 63, 64, 65, 127, 128, 129, 255, 256, 257, 300, 512, 1000, 2048, 4096, 9999]),
                        ("n_seqs", [1, 2, 3, 16, 63, 64, 65, 100, 1000, 4096, 9000]),
                        ("max_pages", [0, 1, 2, 5, 100, 5000]), ("page_size", [1, 3, 64, 100])):
        for rows in (1, 30, 4096):
            got = [smla.smla_paged_attend_workspace_size(**{**base, "n_rows": rows, "num_heads": heads, name: n})
                   for n in sizes]
            assert got == sorted(got) and got[0] > 0, (name, rows)


@pytest.mark.parametrize("heads", [16, 64])
def test_a_step_runs_in_the_workspace_of_the_longest_chunk(heads):
    # a server's workspace: sized once for 2048 rows of 64 sequences
    n = smla.smla_paged_attend_workspace_size(2048, heads, 64, 64, 128)
    ws = torch.full((n + 4096,), 0xAB, dtype=torch.uint8, device=DEV)
    for lens in ([(1, 70 + 9 * b) for b in range(64)], [(2, 64 + b) for b in range(40)], [(1, 5000)], [(90, 90)] * 3):
        c = Batch(lens, 64)
        c.table = torch.nn.functional.pad(c.table, (0, 128 - c.table.shape[1]), value=-1)
        q = torch.randn(c.rows, heads, 576, generator=gen(1)).to(torch.bfloat16)
        out = torch.empty(c.rows, heads, 512, dtype=torch.bfloat16, device=DEV)
        lse = torch.empty(c.rows, heads, device=DEV)
        smla.smla_paged_attend(q.to(DEV), c.cache(), *c.dev(), 1 / 24, None, out, lse, workspace_tensor=ws[:n])
        check(c, q, out, lse, 1 / 24, None, True)
    assert (ws[n:] == 0xAB).all()


# ---- latents that are not finite ----


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
def test_an_infinite_latent_takes_its_blocks_scale_and_no_other(dtype):
    # scale 2^120: +-inf saturates at +-448 (read back: beyond the largest f32), values up
    # to 2^110 (half the least code 2^-9) become zeros of their sign, larger ones are codes
    kind = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}[dtype]
    lat = (torch.randn(4, 512, generator=gen(3)) * 8).to(kind)
    lat[1, 130], lat[1, 131] = float("inf"), -float("inf")
    lat[2, 300] = float("inf")
    lat[3, 17] = float("nan")
    if dtype != "f16":
        lat[1, 140], lat[1, 141] = 2.0 ** 127, -(2.0 ** 112)
    block = lat[1, 128:256].float()
    kv = torch.zeros(1, 4, REC, dtype=torch.uint8, device=DEV)
    table, cu = torch.zeros(1, 1, dtype=torch.int32, device=DEV), torch.tensor([0, 4], dtype=torch.int32, device=DEV)
    sl = torch.tensor([4], dtype=torch.int32, device=DEV)
    smla.smla_paged_write(lat.to(DEV), torch.zeros(4, 64, dtype=kind, device=DEV), kv, table, cu, sl)
    rec = kv.cpu().numpy()[0]
    scale = rec[:, 512:528].copy().view(np.float32)
    assert scale[1, 1] == 2.0 ** 120 and scale[2, 2] == 2.0 ** 120
    codes = oracle.e4m3_table()[rec[1, 128:256]]
    expect = oracle.e4m3_table()[np.asarray(oracle.e4m3_encode_rne(
        torch.where(torch.isinf(block), torch.zeros(()), block).double().numpy() / 2.0 ** 120), np.uint8)]
    expect[2], expect[3] = 448.0, -448.0
    assert np.array_equal(codes, expect) and np.count_nonzero(codes) == (2 if dtype == "f16" else 4)
    zero = codes == 0
    assert np.array_equal(rec[1, 128:256][zero] >> 7, (block.numpy()[zero] < 0).astype(np.uint8))
    assert rec[3, 17] & 0x7F == 0x7F
    # every other block is as if nothing had been there
    want = expect_records(torch.where(torch.isfinite(lat), lat, 0.0), torch.zeros(4, 64))
    for r in range(4):
        for i in range(4):
            if (r, i) not in ((1, 1), (2, 2)):
                keep = [d for d in range(128 * i, 128 * i + 128) if (r, d) != (3, 17)]
                assert np.array_equal(rec[r, keep], want[r, keep])
                assert np.array_equal(rec[r, 512 + 4 * i:516 + 4 * i], want[r, 512 + 4 * i:516 + 4 * i])
    back, rope = torch.empty(4, 512, device=DEV), torch.empty(4, 64, device=DEV)
    smla.smla_paged_read(kv, table, cu, sl, back, rope)
    assert back[1, 130] == float("inf") and back[1, 131] == -float("inf") and torch.isnan(back[3, 17])


# ---- sinks, queries and scores that are not finite ----


@pytest.mark.parametrize("name", sorted(KERNELS))
def test_sinks_that_are_not_finite(name):
    # one row shared between workers, one finished by its own, one without a key
    heads = KERNELS[name]
    c = Batch([(1, 3000), (1, 40), (1, 0)], 64)
    q = torch.randn(c.rows, heads, 576, generator=gen(5)).to(torch.bfloat16)
    sink = torch.randn(heads, generator=gen(6))
    sink[1], sink[3], sink[5] = float("inf"), -float("inf"), float("nan")
    kv, dev = c.cache(), c.dev()
    got = []
    for sk in (sink, torch.where(torch.isfinite(sink), sink, -1e30), None):
        out = torch.empty(c.rows, heads, 512, dtype=torch.bfloat16, device=DEV)
        lse = torch.empty(c.rows, heads, device=DEV)
        smla.smla_paged_attend(q.to(DEV), kv, *dev, 1 / 24, None if sk is None else sk.to(DEV), out, lse)
        got.append((out.cpu(), lse.cpu()))
    (out, lse), (fine, fine_lse), (plain, _) = got
    assert torch.equal(lse, fine_lse)  # no sink enters the LSE
    assert (out[:, 1] == 0).all()
    # a sink of -inf is a weight of zero: as without one, each rounded once to bf16
    assert torch.equal(out[:, 3], fine[:, 3])
    assert ((out[:2, 3].float() - plain[:2, 3].float()).abs() <= 2 * 2.0 ** -8 * plain[:2, 3].float().abs()).all()
    assert torch.isnan(out[:2, 5].float()).all()
    assert (out[2, [0, 1, 2, 3, 4]] == 0).all() and torch.isneginf(lse[2]).all()
    rest = [h for h in range(heads) if h not in (1, 3, 5)]
    assert torch.equal(out[:, rest], fine[:, rest])


@pytest.mark.parametrize("name", sorted(KERNELS))
def test_infinite_queries_and_ropes_follow_their_scores(name):
    # dim 40 of every key is -1 and dim 41 is +1 or -1: q = +inf there gives scores of
    # -inf alone (weights of zero, as without a key), q = -inf scores of +inf (NaN), +inf at
    # dim 41 both (NaN).  Masked pages hold zeros in the tiles, whose product with an
    # infinity is NaN: the mask has to keep it out
    heads = KERNELS[name]
    c = Batch([(1, 3000), (1, 40)], 64)
    c.rec[:, 40], c.rec[:, 41] = 0xB8, np.where(np.arange(c.rec.shape[0]) % 2, 0xB8, 0x38)
    c.rec[:, 512:528] = np.ones(4, np.float32).view(np.uint8)
    c.table[0, 5] = c.table[0, -1] = -1
    inf = float("inf")
    q, _, want, want_lse, _ = attend(c, heads, sink=True)
    bad = q.clone()
    bad[:, 3, 40], bad[:, 5, 40], bad[:, 7, 41] = inf, -inf, inf
    _, _, out, lse, _ = attend(c, heads, q=bad, sink=True)
    assert (out[:, 3] == 0).all() and torch.isneginf(lse[:, 3]).all()
    for h in (5, 7):
        assert torch.isnan(out[:, h].float()).all() and torch.isnan(lse[:, h]).all()
    rest = [h for h in range(heads) if h not in (3, 5, 7)]
    assert torch.equal(out[:, rest], want[:, rest]) and torch.equal(lse[:, rest], want_lse[:, rest])
    # an infinite rope of single keys: heads whose q is negative there see scores of -inf,
    # which drop those keys, the others +inf
    q[:, :, 560] = torch.where(torch.arange(heads) % 2 == 0, -1.0, 1.0)
    keys = [c.slot(0, 2), c.slot(0, 2990 - 64), c.slot(1, 39)]
    c.rec[keys, 528 + 2 * (560 - 512):530 + 2 * (560 - 512)] = np.array([0x7F80], np.uint16).view(np.uint8)
    _, sk, out, lse, _ = attend(c, heads, q=q, sink=True)
    assert torch.isnan(out[:, 1::2].float()).all() and torch.isnan(lse[:, 1::2]).all()
    # the even heads against a cache where those keys' pages hold them no more: 64-bit
    # softmax over the finite scores
    lat, _, rope = unpack(c.rec)
    key = np.concatenate([lat, rope], 1)
    for r, b, p in c.positions():
        ids = [c.slot(b, t) for t in range(p + 1) if c.slot(b, t) >= 0]
        ids = np.array([i for i in ids if i not in keys])
        s = q[r, ::2].double().numpy() @ key[ids].T / 24
        m = s.max(1, keepdims=True)
        w = np.exp(s - m)
        den = w.sum(1, keepdims=True) + np.exp(sk[::2].double().numpy()[:, None] - m)
        ref, spread = (w / den) @ key[ids, :512], (w / den) @ np.abs(key[ids, :512])
        # f32 dot products of 576 terms (doubled for slack), p and the result as bf16
        ds = 2 * 576 * 2.0 ** -24 * (np.abs(q[r, ::2].double().numpy()) @ np.abs(key[ids]).T).max() / 24
        err = np.abs(out[r, ::2].double().cpu().numpy() - ref)
        assert (err <= (2.0 ** -8 + 2 * ds) * spread + 2.0 ** -8 * np.abs(ref)).all()
        e = np.abs(lse[r, ::2].double().cpu().numpy() - (m[:, 0] + np.log(w.sum(1))))
        assert (e <= ds + 2.0 ** -18 * (1 + np.abs(m[:, 0]) + np.log(len(ids)))).all()


# ---- empty sequences in between ----


def ms_of(call):
    call()
    torch.cuda.synchronize()
    ev = [torch.cuda.Event(enable_timing=True) for _ in range(2)]
    ev[0].record()
    call()
    ev[1].record()
    torch.cuda.synchronize()
    return ev[0].elapsed_time(ev[1])


def with_gap(first, gap, rest):
    """cu_rows, seq_lens and block table (one page a sequence, -1 for none) of sequences of
    (rows, length, page), `gap` empty ones behind the `first`."""
    seqs = list(first) + list(rest)
    rows = torch.tensor([n for n, _, _ in seqs], dtype=torch.int32)
    k = len(first)
    n = torch.cat([rows[:k], torch.zeros(gap, dtype=torch.int32), rows[k:]])
    cu = torch.cat([torch.zeros(1, dtype=torch.int32), n.cumsum(0, dtype=torch.int32)])
    sl, table = torch.zeros(len(n), dtype=torch.int32), torch.full((len(n), 1), -1, dtype=torch.int32)
    at = list(range(k)) + list(range(k + gap, k + gap + len(rest)))
    sl[at] = torch.tensor([s for _, s, _ in seqs], dtype=torch.int32)
    table[at, 0] = torch.tensor([p for _, _, p in seqs], dtype=torch.int32)
    return table.to(DEV), cu.to(DEV), sl.to(DEV)


@pytest.mark.parametrize("gap", [0, 1, 2, 33, 1 << 20])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_a_read_finds_rows_behind_empty_sequences(dtype, gap):
    # row 2432 of 16-bit reads shares its warp with the first row behind the gap
    page = 2500
    g = gen(2)
    lat = torch.randn(3 * page, 512, generator=g).to(torch.bfloat16)
    rope = torch.randn(3 * page, 64, generator=g).to(torch.bfloat16)
    rec = oracle.pack_records(bits(lat), bits(rope))
    kv = torch.from_numpy(rec).view(3, page, REC).to(DEV)
    table, cu, sl = with_gap([(2433, 2440, 1)], gap, [(1, 7, 2), (3, 3, 0)])
    kind = torch.bfloat16 if dtype == "bf16" else torch.float32
    out = torch.full((2440, 512), 7.0, dtype=kind, device=DEV)
    out_rope = torch.full((2440, 64), 7.0, dtype=kind, device=DEV)
    ms = ms_of(lambda: smla.smla_paged_read(kv, table, cu, sl, out, out_rope))
    slots = [page + 7 + i for i in range(2433)] + [2 * page + 6, 0, 1, 2]
    vals, _, rp = unpack(rec[slots])
    assert torch.equal(out[:2437].cpu(), torch.from_numpy(vals).to(kind))
    assert torch.equal(out_rope[:2437].cpu(), torch.from_numpy(rp).to(kind))
    assert (out[2437:] == 7.0).all() and (out_rope[2437:] == 7.0).all()
    assert ms < 2.0, ms  # some 20 us; one load after the other through 2^20 sequences: 72 ms


@pytest.mark.parametrize("gap", [1, 2, 3, 31, 32, 33, 1000, 1 << 16])
@pytest.mark.parametrize("heads,rows", [(4, 3), (64, 40), (128, 2), (16, 300)])
def test_attend_goes_past_empty_sequences(heads, rows, gap):
    # several row tiles a worker, so that workers go from one side of the gap to the
    # other; the same rows without the gap, of which the oracle checks a sample
    page = 1024
    c = Batch([(rows, 1024)] * 3, page, spare_pages=0)
    kv = c.cache()
    pages = [int(p) for p in c.table[:, 0]]
    first, rest = [(rows, 1000, pages[0]), (rows, 700, pages[1])], [(rows - 1, 900, pages[2])]
    n = 3 * rows - 1
    q = torch.randn(n, heads, 576, generator=gen(7)).to(torch.bfloat16)
    got, took = [], []
    for g in (0, gap):
        table, cu, sl = with_gap(first, g, rest)
        out = torch.empty(n, heads, 512, dtype=torch.bfloat16, device=DEV)
        lse = torch.empty(n, heads, device=DEV)
        st = torch.zeros(1, dtype=torch.int32, device=DEV)
        qd = q.to(DEV)
        took.append(ms_of(lambda: smla.smla_paged_attend(qd, kv, table, cu, sl, 1 / 24, None, out, lse, status=st)))
        assert int(st) == 0
        got.append((out.cpu(), lse.cpu()))
    c.lens = [(rows, 1000), (rows, 700), (rows - 1, 900)]
    picked = [x for i, x in enumerate((r, b, p) for b, (k, s) in enumerate(c.lens) for r, b, p in
                                      [(b * rows + i, b, s - k + i) for i in range(k)]) if i % max(1, n // 40) == 0]
    idx, ptr = [], [0]
    for _, b, p in picked:
        idx += [pages[b] * page + t for t in range(p + 1)]
        ptr.append(len(idx))
    ids = [r for r, _, _ in picked]
    idx, ptr = np.array(idx, np.int32), np.array(ptr, np.int32)
    qq = q.double().numpy()[ids]
    ref, ref_lse, _ = oracle.sparse_mla_decode(qq, c.rec, idx, ptr, None, 1 / 24, None)
    a_out, a_lse = allowance(qq, c.rec, idx, ptr, None, 1 / 24, None)
    for out, lse in got:
        assert torch.isfinite(out.float()).all() and torch.isfinite(lse).all()
        assert (np.abs(out.double().numpy()[ids] - ref) <= a_out + 2.0 ** -8 * np.abs(ref) + 1e-30).all()
        assert (np.abs(lse.double().numpy()[ids] - ref_lse) <= a_lse + 2.0 ** -18 * (1 + np.abs(ref_lse).max())).all()
    # (all rows, also those that are not in the sample: p and the result as bf16, of values
    # up to ~2)
    assert (got[0][0].float() - got[1][0].float()).abs().max() <= 4 * 2.0 ** -8 * 2
    assert (got[0][1] - got[1][1]).abs().max() <= 1e-4


def test_attend_takes_no_longer_with_a_large_gap():
    # pairs of CTAs: one of them goes past 2^16 empty sequences (60 ms one by one)
    kv = torch.zeros(1, 1024, REC, dtype=torch.uint8, device=DEV)
    table, cu, sl = with_gap([(1, 1000, 0)] * 33, 1 << 16, [(1, 900, 0)] * 20)
    q = torch.zeros(53, 128, 576, dtype=torch.bfloat16, device=DEV)
    out = torch.empty(53, 128, 512, dtype=torch.bfloat16, device=DEV)
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    ms = ms_of(lambda: smla.smla_paged_attend(q, kv, table, cu, sl, 1 / 24, None, out, None, status=st))
    assert int(st) == 0 and ms < 3.0, ms


# ---- each kernel on keys that rows may not see and queries that are bad ----

# (rows of a chunk + empty sequences) by their mean number of rows, which chooses the kernel
EMPTY_FOR = {"pair": 0, "narrow64": 2, "narrow32": 5, "few": 20}


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("name", sorted(EMPTY_FOR))
def test_hidden_keys_reach_no_row_in_any_kernel(name, causal):
    # 10 tokens x 16 heads over 1 + empty sequences: a mean of 160, 54, 27 and 8 rows.  The
    # later tokens' records hold a NaN code, an infinite and a NaN scale, an infinite rope
    c = Batch([(10, 75)] + [(0, 0)] * EMPTY_FOR[name], 16)
    q, _, want, want_lse, _ = attend(c, 16)
    for p, at, value in ((70, slice(7, 8), np.array([0x7F], np.uint8)), (71, slice(512, 516), np.array([np.inf], np.float32)),
                         (72, slice(528, 530), np.array([0x7F80], np.uint16)), (73, slice(512, 516), np.array([np.nan], np.float32))):
        c.rec[c.slot(0, p), at] = value.view(np.uint8)
    i = int(c.table[0, 4]) * 16
    c.rec[i + 11:i + 16] = 0xFF  # slots past the end, in the last page
    _, _, out, lse, _ = attend(c, 16, q=q, causal=causal)
    if causal:
        assert torch.equal(out[:5], want[:5]) and torch.equal(lse[:5], want_lse[:5])
        assert torch.isnan(out[5:].float()).all() and torch.isnan(lse[5:]).all()
    else:
        assert torch.isnan(out.float()).all() and torch.isnan(lse).all()


@pytest.mark.parametrize("name,empty", [("pair", 0), ("narrow64", 1), ("narrow32", 3), ("few", 20)])
def test_a_bad_query_stays_in_its_row_in_any_kernel(name, empty):
    # 10 tokens x 16 heads over 2 + empty sequences: a mean of 80, 54, 32 and 8 rows; long
    # sharp rows beside the bad ones move their references after them
    c = Batch([(9, 100), (1, 900)] + [(0, 0)] * empty, 16, std=2.0)
    q, _, want, want_lse, _ = attend(c, 16, sm_scale=0.5)
    q2 = q.clone()
    q2[4, 3, 17], q2[9, 5, 570], q2[9, 6, 300] = float("nan"), float("nan"), -float("nan")
    _, _, out, lse, _ = attend(c, 16, q=q2, sm_scale=0.5)
    keep = torch.ones(c.rows, 16, dtype=torch.bool)
    for r, h in ((4, 3), (9, 5), (9, 6)):
        assert torch.isnan(out[r, h].float()).all() and torch.isnan(lse[r, h])
        keep[r, h] = False
    assert torch.equal(out.cpu()[keep], want.cpu()[keep]) and torch.equal(lse.cpu()[keep], want_lse.cpu()[keep])


@pytest.mark.parametrize("heads", [30, 64])
def test_narrow_tiles_return_every_code_exactly(heads):
    # one key: out is its latent (as for 16 and 128 heads)
    c = Batch([(1, 1)] * 8, 1)
    codes = np.array([x for x in range(256) if x & 0x7F != 0x7F] + [0, 0], np.uint8)
    scales = [2.0 ** e for e in (-116, -40, -22, -9, 0, 5, 7)] + [0.0]
    for b in range(8):
        s = c.slot(b, 0)
        c.rec[s, :512] = np.concatenate([codes, codes[::-1]])
        c.rec[s, 512:528] = np.full(4, scales[b], np.float32).view(np.uint8)
    q, _, out, lse, _ = attend(c, heads, q=torch.zeros(8, heads, 576, dtype=torch.bfloat16))
    lat = unpack(c.rec)[0]
    for b in range(8):
        assert (out[b].double().cpu().numpy() == lat[c.slot(b, 0)]).all(), scales[b]
    assert (lse == 0).all()


@pytest.mark.parametrize("heads", [10, 20])
def test_narrow_tiles_foreign_scales_round_once(heads):
    # 3 tokens: 30 and 60 rows
    c = Batch([(3, 270)], 16)
    sc = torch.exp2(torch.rand(c.n_pages * 16, 4, generator=gen(4)) * 6 - 4).float().numpy()
    sc[::3] = np.ldexp(1.0, np.random.default_rng(0).integers(-130, 9, sc[::3].shape)).astype(np.float32)
    c.rec[:, 512:528] = sc.view(np.uint8)
    q, _, out, lse, _ = attend(c, heads)
    rows, ref, ref_lse, (a_out, a_lse) = reference_operands(c, q)
    err = np.abs(out.double().cpu().numpy()[rows] - ref) - (a_out + 2.0 ** -8 * np.abs(ref))
    assert err.max() <= 0
    assert (np.abs(lse.double().cpu().numpy()[rows] - ref_lse) <= a_lse + 2.0 ** -18 * (1 + np.abs(ref_lse).max())).all()


@pytest.mark.parametrize("heads", [30, 64])
def test_narrow_tiles_sharp_softmax_and_odd_scales(heads):
    c = Batch([(1, 700), (1, 1500), (1, 64), (1, 65)], 20, std=3.0, page_pad=32, front=1, behind=2)
    c.table[torch.rand(c.table.shape, generator=gen(1)) < 0.05] = -1
    for scale in (1.0, -0.3, 0.0):
        q, sk, out, lse, _ = attend(c, heads, sm_scale=scale, sink=True)
        check(c, q, out, lse, scale, sk, True)


@pytest.mark.parametrize("heads", [30, 64])
def test_narrow_tiles_wait_timeout_sets_the_status_and_leaves_the_context_usable(heads):
    c = Batch([(1, 500), (1, 900)], 64)
    try:
        smla.smla_set_wait_limit(20_000_000, stall_first_wait=True)
        *_, st = attend(c, heads)
        assert st & smla.STATUS_TIMEOUT
    finally:
        smla.smla_set_wait_limit(0)
    q, sk, out, lse, st = attend(c, heads)
    assert st == 0
    check(c, q, out, lse, 1 / 24, sk, True)


@pytest.mark.parametrize("name", sorted(KERNELS))
def test_repeated_launches_give_the_same_bits(name):
    # sums in fixed order, also of row tiles shared between many workers
    heads = KERNELS[name]
    c = Batch([(1, 5000), (1, 900), (1, 50)], 64)
    q, _, want, want_lse, _ = attend(c, heads, sink=True)
    assert torch.isfinite(want.float()).all()
    flush = torch.empty(256 << 20, dtype=torch.uint8, device=DEV)
    for i in range(12):
        flush.fill_(i)
        _, _, out, lse, _ = attend(c, heads, q=q, sink=True)
        assert torch.equal(out, want) and torch.equal(lse, want_lse)


@pytest.mark.parametrize("heads", [4, 30, 64, 128])
@pytest.mark.parametrize("bad", [[0, 6, 3], [7, 0, 0], [5, 5, 2], [-4, 900, -900], [900, 3, 900]])
def test_boundaries_that_decrease_leave_the_tensors_alone(heads, bad):
    # which rows they name is not defined; rows in front of and behind the tensors and the
    # records of the cache stay as they are
    c = Batch([(4, 40), (3, 30)], 16)
    kv, (table, _, sl) = c.cache(), c.dev()
    before = c.buf.clone()
    cu = torch.tensor(bad, dtype=torch.int32, device=DEV)
    guard, n = 5, 7
    q = torch.randn(n, heads, 576, generator=gen(1)).to(torch.bfloat16).to(DEV)
    out = torch.full((n + 2 * guard, heads, 512), 7.0, dtype=torch.bfloat16, device=DEV)
    lse = torch.full((n + 2 * guard, heads), 7.0, device=DEV)
    lat, rope = torch.full((n + 2 * guard, 512), 7.0, device=DEV), torch.full((n + 2 * guard, 64), 7.0, device=DEV)
    mid = slice(guard, guard + n)
    smla.smla_paged_attend(q, kv, table, cu, sl, 1 / 24, None, out[mid], lse[mid])
    smla.smla_paged_read(kv, table, cu, sl, lat[mid], rope[mid])
    torch.cuda.synchronize()
    for t in (out, lse, lat, rope):
        assert (t[:guard] == 7.0).all() and (t[guard + n:] == 7.0).all()
    assert torch.equal(c.buf, before)


@pytest.mark.parametrize("name", sorted(KERNELS))
def test_the_largest_finite_sinks_hold_all_or_none_of_the_weight(name):
    heads = KERNELS[name]
    c = Batch([(1, 3000), (1, 40)], 64)
    q = torch.randn(c.rows, heads, 576, generator=gen(5)).to(torch.bfloat16)
    sink = torch.full((heads,), 3e38)  # times log2(e) beyond the largest f32
    sink[::2] = -3e38
    out = torch.empty(c.rows, heads, 512, dtype=torch.bfloat16, device=DEV)
    lse = torch.empty(c.rows, heads, device=DEV)
    smla.smla_paged_attend(q.to(DEV), c.cache(), *c.dev(), 1 / 24, sink.to(DEV), out, lse)
    assert (out[:, 1::2] == 0).all() and torch.isfinite(lse).all()
    sink[1::2] = 0.0
    rows, ref, ref_lse, (a_out, a_lse) = reference(c, q, 1 / 24, sink, True)
    err = np.abs(out.double().cpu().numpy() - ref)[:, ::2]
    assert (err <= (a_out + 2.0 ** -8 * np.abs(ref))[:, ::2]).all()


# ---- calls at once, and steps in a graph ----


def test_calls_of_every_kernel_at_once_give_the_bits_of_calls_alone():
    # four streams, a kernel each, eight calls in a row without a wait in between
    jobs = []
    for i, (name, heads) in enumerate(sorted(KERNELS.items())):
        c = Batch([(1, 2500), (1, 700)] if name != "pair" else [(3, 1500), (5, 333)], 64, seed=i)
        q, _, want, want_lse, _ = attend(c, heads)
        jobs.append((c, heads, q.to(DEV), c.cache(), c.dev(), want, want_lse, torch.cuda.Stream()))
    got = []
    torch.cuda.synchronize()
    for _ in range(8):
        for c, heads, q, kv, dev, want, want_lse, stream in jobs:
            out, lse = torch.empty_like(want), torch.empty_like(want_lse)
            stream.wait_stream(torch.cuda.current_stream())
            smla.smla_paged_attend(q, kv, *dev, 1 / 24, None, out, lse, stream=stream)
            got.append((out, lse, want, want_lse))
    torch.cuda.synchronize()
    for out, lse, want, want_lse in got:
        assert torch.equal(out, want) and torch.equal(lse, want_lse)


@pytest.mark.parametrize("heads", [16, 64, 128])
def test_a_serving_step_in_a_graph(heads):
    # write, attend and read back as one graph over a batch of fixed size (4 slots, 6 token
    # rows), replayed as sequences grow, move to other pages, finish and start
    page, n_pages, rows = 16, 40, 6
    g = gen(heads)
    rec = oracle.pack_records(bits(torch.randn(n_pages * page, 512, generator=g).to(torch.bfloat16)),
                              bits(torch.randn(n_pages * page, 64, generator=g).to(torch.bfloat16)))
    kv = torch.from_numpy(rec.copy()).view(n_pages, page, REC).to(DEV)
    lat = torch.zeros(rows, 512, dtype=torch.bfloat16, device=DEV)
    rope = torch.zeros(rows, 64, dtype=torch.bfloat16, device=DEV)
    q = torch.zeros(rows, heads, 576, dtype=torch.bfloat16, device=DEV)
    table = torch.full((4, 10), -1, dtype=torch.int32, device=DEV)
    cu, sl = torch.zeros(5, dtype=torch.int32, device=DEV), torch.zeros(4, dtype=torch.int32, device=DEV)
    out = torch.zeros(rows, heads, 512, dtype=torch.bfloat16, device=DEV)
    lse, back = torch.zeros(rows, heads, device=DEV), torch.zeros(rows, 512, device=DEV)
    back_rope, status = torch.zeros(rows, 64, device=DEV), torch.zeros(1, dtype=torch.int32, device=DEV)

    def step():
        smla.smla_paged_write(lat, rope, kv, table, cu, sl, status=status)
        smla.smla_paged_attend(q, kv, table, cu, sl, 1 / 24, None, out, lse, status=status)
        smla.smla_paged_read(kv, table, cu, sl, back, back_rope, status=status)

    step()  # (no rows yet)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for lens in ([(1, 30), (1, 1), (3, 100), (1, 17)], [(2, 32), (0, 0), (1, 101), (1, 18)], [(0, 0), (0, 0), (0, 0), (6, 150)],
                 [(0, 0)] * 4):
        order = torch.randperm(n_pages, generator=g).to(torch.int32)
        c = Batch([(0, 0)] * 4, page)
        c.lens, c.n_pages, c.rows, c.rec = lens, n_pages, rows, rec
        c.table = torch.full((4, 10), -1, dtype=torch.int32)
        at = 0
        for b, (_, s) in enumerate(lens):
            k = -(-s // page)
            c.table[b, :k] = order[at:at + k]
            at += k
        c.cu = torch.tensor([0] + [sum(n for n, _ in lens[:b + 1]) for b in range(4)], dtype=torch.int32)
        new, new_rope = (torch.randn(rows, d, generator=g).to(torch.bfloat16) for d in (512, 64))
        qq = torch.randn(rows, heads, 576, generator=g).to(torch.bfloat16)
        for there, here in ((lat, new), (rope, new_rope), (q, qq), (table, c.table), (cu, c.cu),
                            (sl, torch.tensor([s for _, s in lens], dtype=torch.int32))):
            there.copy_(here)
        for t in (out, lse, back, back_rope):
            t.fill_(7.0)
        graph.replay()
        torch.cuda.synchronize()
        for r, b, p in c.positions():
            rec[c.slot(b, p)] = oracle.pack_records(bits(new[r:r + 1]), bits(new_rope[r:r + 1]))[0]
        assert np.array_equal(kv.view(-1, REC).cpu().numpy(), rec)
        check(c, qq, out, lse, 1 / 24, None, True)
        vals, _, rp = unpack(rec)
        n = int(c.cu[-1])
        slots = [c.slot(b, p) for _, b, p in c.positions()]
        assert np.array_equal(back[:n].cpu().double().numpy(), vals[slots]) and (back[n:] == 7.0).all()
        assert np.array_equal(back_rope[:n].cpu().double().numpy(), rp[slots]) and (back_rope[n:] == 7.0).all()
        assert int(status) == 0

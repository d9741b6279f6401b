"""The paged cache on the GPU against plain 64-bit evaluations: records written
bit for bit, records read back, attention of new tokens over them."""

import numpy as np
import pytest
import torch

import oracle
import sparse_mla_decode_csr_gb300 as smla
from smla_testlib import U32, allowance, bits

pytestmark = pytest.mark.gpu
DEV = "cuda"
REC = 656
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


def gen(seed):
    return torch.Generator().manual_seed(seed)


class Batch:
    """Sequences of (token rows, length) in a paged cache with shuffled pages.

    rec: the cache's records by slot as numpy (filled by the oracle's writer);
    page_pad: bytes between pages, front/behind: token rows of no sequence."""

    def __init__(self, lens, page, seed=0, spare_pages=2, page_pad=0, front=0, behind=0, std=1.0):
        g = gen(seed)
        self.lens, self.page, self.front = lens, page, front
        pages = [max(0, -(-s // page)) for _, s in lens]
        self.n_pages = sum(pages) + spare_pages
        order = torch.randperm(self.n_pages, generator=g).to(torch.int32)
        self.table = torch.full((len(lens), max(pages + [1])), -1, dtype=torch.int32)
        at = 0
        for b, k in enumerate(pages):
            self.table[b, :k] = order[at:at + k]
            at += k
        self.cu = torch.tensor([front] + [front + sum(n for n, _ in lens[:b + 1]) for b in range(len(lens))],
                               dtype=torch.int32)
        self.seq_lens = torch.tensor([s for _, s in lens], dtype=torch.int32)
        self.rows = int(self.cu[-1]) + behind
        slots = self.n_pages * page
        lat = (torch.randn(slots, 512, generator=g) * std).to(torch.bfloat16)
        rope = torch.randn(slots, 64, generator=g).to(torch.bfloat16)
        self.rec = oracle.pack_records(bits(lat), bits(rope))
        self.pad = page_pad
        self.g = g

    def cache(self):
        """The records on the device, pages page_pad bytes apart."""
        stride = self.page * REC + self.pad
        buf = torch.full((self.n_pages, stride), 0xEE, dtype=torch.uint8)
        buf[:, :self.page * REC] = torch.from_numpy(self.rec).view(self.n_pages, -1)
        self.buf = buf.to(DEV)
        return self.buf[:, :self.page * REC].view(self.n_pages, self.page, REC)

    def dev(self):
        return self.table.to(DEV), self.cu.to(DEV), self.seq_lens.to(DEV)

    def slot(self, b, p):
        """Slot of position p of sequence b, or -1 when masked."""
        if p < 0 or p // self.page >= self.table.shape[1]:
            return -1
        i = int(self.table[b, p // self.page])
        return -1 if i < 0 or i >= self.n_pages else i * self.page + p % self.page

    def positions(self):
        """(row, sequence, position) of every token row."""
        for b, (n, s) in enumerate(self.lens):
            for i in range(n):
                yield int(self.cu[b]) + i, b, s - n + i


# ---- write and read --------------------------------------------------------


def expect_records(lat, rope):
    """Records of the rule in 64 bits, for inputs of any type."""
    x = lat.double().numpy().reshape(-1, 4, 128)
    y = np.maximum(np.abs(x).max(2), 1e-4) / 448.0
    man, exp = np.frexp(y)
    scale = np.ldexp(1.0, np.where(man == 0.5, exp - 1, exp))
    code = oracle.e4m3_encode_rne((x / scale[..., None]).reshape(-1))
    n = lat.shape[0]
    return np.concatenate([np.asarray(code, np.uint8).reshape(n, 512), scale.astype(np.float32).view(np.uint8),
                           bits(rope.to(torch.bfloat16)).view(np.uint8).reshape(n, 128)], 1)


COPY_CASES = [
    # lens, page, page_pad, front, behind
    ([(1, 1)], 1, 0, 0, 0),
    ([(5, 9), (0, 4), (1, 70), (33, 33)], 16, 32, 2, 3),
    ([(3, 100)] * 70, 48, 0, 0, 1),
    ([(700, 1000), (999, 999)], 64, 16, 1, 40),
    ([(2601, 2605)], 100, 0, 0, 1),  # 16-bit reads of two rows a warp, the last one alone
]


@pytest.mark.parametrize("dtype", sorted(TYPES))
@pytest.mark.parametrize("lens,page,pad,front,behind", COPY_CASES)
def test_write_is_bit_exact_and_touches_nothing_else(lens, page, pad, front, behind, dtype):
    c = Batch(lens, page, page_pad=pad, front=front, behind=behind)
    lat = (torch.randn(c.rows, 512, generator=c.g) * torch.exp2(torch.randint(-20, 12, (c.rows, 1), generator=c.g)))
    lat, rope = lat.to(TYPES[dtype]), torch.randn(c.rows, 64, generator=c.g).to(TYPES[dtype])
    lat[0] = 0.0  # the floor of the scale
    kv = c.cache()
    want = expect_records(lat, rope)
    if dtype == "bf16":
        assert np.array_equal(want, oracle.pack_records(bits(lat), bits(rope)))
    rec = c.rec.copy()
    for r, b, p in c.positions():
        rec[c.slot(b, p)] = want[r]
    wide = torch.zeros(c.rows, 640, dtype=TYPES[dtype], device=DEV)  # strided inputs
    wide[:, :512], wide[:, 512:576] = lat.to(DEV), rope.to(DEV)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    smla.smla_paged_write(wide[:, :512], wide[:, 512:576], kv, *c.dev(), status=status)
    got = c.buf.cpu()
    assert np.array_equal(got[:, :page * REC].reshape(-1, REC).numpy(), rec)
    assert (got[:, page * REC:] == 0xEE).all()
    assert int(status) == 0


@pytest.mark.parametrize("dtype", sorted(TYPES))
@pytest.mark.parametrize("lens,page,pad,front,behind", COPY_CASES)
def test_read_gives_the_records_values(lens, page, pad, front, behind, dtype):
    c = Batch(lens, page, page_pad=pad, front=front, behind=behind)
    lat, _, rope = unpack(c.rec)
    got = torch.full((c.rows, 640), 7.0, dtype=TYPES[dtype], device=DEV)
    want = torch.full((c.rows, 576), 7.0, dtype=torch.float64)
    for r, b, p in c.positions():
        want[r] = torch.from_numpy(np.concatenate([lat[c.slot(b, p)], rope[c.slot(b, p)]]))
    smla.smla_paged_read(c.cache(), *c.dev(), got[:, :512], got[:, 512:576])
    # one rounding to the type: the same double rounded by torch
    assert torch.equal(got[:, :576].cpu(), want.to(TYPES[dtype]))
    assert (got[:, 576:] == 7.0).all()


def unpack(rec):
    """f64 latent, scales and rope of records."""
    codes = oracle.e4m3_table()[rec[:, :512]]
    scale = rec[:, 512:528].copy().view(np.float32).astype(np.float64)
    rope = oracle.bf16_to_f64(rec[:, 528:].copy().view(np.uint16))
    return codes * np.repeat(scale, 128, 1), scale, rope


def test_masked_positions_are_skipped_and_flagged():
    c = Batch([(40, 40), (40, 30), (8, 200), (8, 8)], 16)
    c.table[0, 1] = -1                  # a page that is not there: silent
    c.seq_lens[2] = 16 * c.table.shape[1] + 4  # the last four rows lie past the table
    c.lens[2] = (8, int(c.seq_lens[2]))
    c.table[2, -1] = 0
    c.table[3, 0] = c.n_pages - 1
    lat = torch.randn(c.rows, 512, generator=c.g).to(torch.bfloat16)
    rope = torch.randn(c.rows, 64, generator=c.g).to(torch.bfloat16)
    want = oracle.pack_records(bits(lat), bits(rope))
    for oob in (False, True):
        if oob:
            c.table[3, 0] = c.n_pages
        status = torch.zeros(1, dtype=torch.int32, device=DEV)
        kv = c.cache()
        smla.smla_paged_write(lat.to(DEV), rope.to(DEV), kv, *c.dev(), status=status)
        rec = c.rec.copy()
        for r, b, p in c.positions():
            if c.slot(b, p) >= 0:
                rec[c.slot(b, p)] = want[r]
        assert np.array_equal(kv.reshape(-1, REC).cpu().numpy(), rec)
        assert int(status) == smla.STATUS_INDEX_OOB  # sequence 2 in both, sequence 3's page in the second
        l2 = torch.full((c.rows, 512), 7.0, device=DEV)
        r2 = torch.full((c.rows, 64), 7.0, device=DEV)
        smla.smla_paged_read(kv, *c.dev(), l2, r2)
        vals, _, rp = unpack(rec)
        for r, b, p in c.positions():
            s = c.slot(b, p)
            assert torch.equal(l2[r].cpu().double(), torch.from_numpy(vals[s] if s >= 0 else np.zeros(512)))
            assert torch.equal(r2[r].cpu().double(), torch.from_numpy(rp[s] if s >= 0 else np.zeros(64)))


def test_write_of_values_that_are_not_finite():
    lat = torch.randn(3, 512)
    lat[0, 3], lat[1, 200], lat[1, 201] = float("nan"), float("inf"), -float("inf")
    kv = torch.zeros(1, 3, REC, dtype=torch.uint8, device=DEV)
    smla.smla_paged_write(lat.to(DEV), torch.zeros(3, 64, device=DEV), kv, torch.zeros(1, 1, dtype=torch.int32, device=DEV),
                          torch.tensor([0, 3], dtype=torch.int32, device=DEV),
                          torch.tensor([3], dtype=torch.int32, device=DEV))
    rec = kv.cpu().numpy()[0]
    assert rec[0, 3] & 0x7F == 0x7F
    top = 2.0 ** 120  # pow2ceil(largest f32 / 448)
    assert rec[1, 512:528].view(np.float32)[1] == top
    assert oracle.e4m3_value(rec[1, 200]) == 448 and oracle.e4m3_value(rec[1, 201]) == -448
    fine = lat.clone()
    fine[0, 3] = 0.0
    want = expect_records(fine, torch.zeros(3, 64))
    assert np.array_equal(rec[2], want[2]) and np.array_equal(np.delete(rec[0], 3), np.delete(want[0], 3))


def test_read_passes_nan_codes_and_foreign_scales_on():
    c = Batch([(6, 6)], 8)
    c.rec[c.slot(0, 1), 5] = 0x7F
    c.rec[c.slot(0, 2), 512:528] = np.array([0.3, 0.0, -1.5, 3.0], np.float32).view(np.uint8)
    lat, _, rope = unpack(c.rec)
    out = torch.empty(6, 512, device=DEV)
    smla.smla_paged_read(c.cache(), *c.dev(), out, torch.empty(6, 64, device=DEV))
    want = np.stack([lat[c.slot(0, p)] for p in range(6)])
    got = out.cpu().numpy()
    assert np.isnan(got[1, 5]) and np.isnan(want[1, 5])
    want[1, 5] = got[1, 5] = 0.0
    # an f32 product of an exact code and an f32 scale: one rounding, half a step of 2^-23
    assert (np.abs(got - want) <= 2.0 ** -24 * np.abs(want)).all()


# ---- attention --------------------------------------------------------------


def reference(c, q, sm_scale, sink, causal):
    """The oracle's decode over explicit key lists, with the rounding allowance."""
    idx, ptr, rows = [], [0], []
    for r, b, p in c.positions():
        end = p + 1 if causal else c.lens[b][1]
        idx += [c.slot(b, t) for t in range(max(end, 0))]
        ptr.append(len(idx))
        rows.append(r)
    idx, ptr = np.array(idx, np.int32), np.array(ptr, np.int32)
    qq = q.double().numpy()[rows]
    s = None if sink is None else sink.double().numpy()
    out, lse, _ = oracle.sparse_mla_decode(qq, c.rec, idx, ptr, None, sm_scale, s)
    return rows, out, lse, allowance(qq, c.rec, idx, ptr, None, sm_scale, s)


def check(c, q, out, lse, sm_scale, sink, causal, extra=0.0):
    """Every element within the bound of its roundings: the allowance (f32
    scores, p as bf16, see smla_testlib) plus bf16's half step of the result;
    the LSE within its scores' error plus 2^-18 (1 + max |s|) for exponentials,
    logarithm and f32 sums of at most a few hundred tiles."""
    rows, ref, ref_lse, (a_out, a_lse) = reference(c, q, sm_scale, sink, causal)
    got, got_lse = out.double().cpu().numpy(), lse.double().cpu().numpy()
    err = np.abs(got[rows] - ref) - (a_out + 2.0 ** -8 * np.abs(ref) + extra + 1e-30)
    assert np.isfinite(got[rows]).all()
    assert err.max(initial=-1) <= 0, f"out exceeds its bound by {err.max():.3g} at {np.unravel_index(err.argmax(), err.shape)}"
    assert np.array_equal(np.isneginf(got_lse[rows]), np.isneginf(ref_lse))
    fin = np.isfinite(ref_lse)
    e = np.abs(got_lse[rows][fin] - ref_lse[fin]) - (a_lse[fin] + 2.0 ** -18 * (1 + np.abs(ref_lse[fin]).max(initial=0)))
    assert e.max(initial=-1) <= 0, f"lse exceeds its bound by {e.max():.3g}"
    others = np.setdiff1d(np.arange(c.rows), rows)
    assert (got[others] == 7.0).all() and (got_lse[others] == 7.0).all()  # rows of no sequence


def attend(c, heads, *, causal=True, sink=False, sm_scale=1 / 24, q=None, kv=None, run=None, seed=5):
    if q is None:
        q = torch.randn(c.rows, heads, 576, generator=gen(seed)).to(torch.bfloat16)
    sk = torch.randn(heads, generator=gen(seed + 1)) if sink else None
    out = torch.full((c.rows, heads, 512), 7.0, dtype=torch.bfloat16, device=DEV)
    lse = torch.full((c.rows, heads), 7.0, device=DEV)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    (run or smla.smla_paged_attend)(q.to(DEV), c.cache() if kv is None else kv, *c.dev(), sm_scale,
                                    None if sk is None else sk.to(DEV), out, lse, causal=causal, status=status)
    torch.cuda.synchronize()
    return q, sk, out, lse, int(status)


@pytest.mark.parametrize("heads", [16, 1, 7, 33, 64, 100, 128])
def test_attend_one_token(heads):
    c = Batch([(1, 1), (1, 64), (1, 65), (1, 130), (1, 63)], 16)
    q, sk, out, lse, st = attend(c, heads, sink=True)
    check(c, q, out, lse, 1 / 24, sk, True)
    assert st == 0


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("heads,page", [(16, 16), (7, 1), (64, 48), (128, 64), (1, 100), (40, 128)])
def test_attend_chunks(heads, page, causal):
    c = Batch([(1, 300), (9, 9), (17, 200), (0, 50), (130 if heads < 8 else 21, 140), (2, 64)], page, front=1, behind=2,
              page_pad=16)
    q, sk, out, lse, st = attend(c, heads, causal=causal, sink=heads != 64)
    check(c, q, out, lse, 1 / 24, sk, causal)
    assert st == 0


@pytest.mark.parametrize("heads,lens", [(16, [(1, 9000)]), (64, [(3, 5000), (2, 1), (1, 2500)]),
                                        (128, [(2, 3500)]), (8, [(40, 2000)] * 3)])
def test_attend_splits_long_rows_over_pairs(heads, lens):
    c = Batch(lens, 64)
    q, sk, out, lse, _ = attend(c, heads, sink=True)
    check(c, q, out, lse, 1 / 24, sk, True)


def test_attend_many_sequences():
    r = np.random.default_rng(3)
    c = Batch([(int(r.integers(0, 4)), int(r.integers(4, 90))) for _ in range(900)], 32)
    q, sk, out, lse, _ = attend(c, 4)
    check(c, q, out, lse, 1 / 24, sk, True)


@pytest.mark.parametrize("heads", [5, 16, 30, 64])
@pytest.mark.parametrize("page", [1, 20, 64])
def test_both_kernels_on_the_same_rows(heads, page):
    # empty sequences lower the mean number of rows, which chooses the kernel: the
    # same rows through tiles of 16, 32 or 64 rows and through pairs of CTAs
    base = [(3, 200), (20, 150), (1, 64), (65 // heads + 1, 333)]
    outs = []
    for empty in (0, 60):
        c = Batch(base + [(0, 0)] * empty, page)
        q, sk, out, lse, st = attend(c, heads, sink=True)
        check(c, q, out, lse, 1 / 24, sk, True)
        outs.append((out.float(), lse))
    # both within 2^-8 (p) + 2^-8 (result) of the exact value, of values up to ~2
    assert (outs[0][0] - outs[1][0]).abs().max() <= 4 * 2.0 ** -8 * 2
    assert (outs[0][1] - outs[1][1]).abs().max() <= 1e-4


@pytest.mark.parametrize("heads,rows", [(16, 1), (64, 1), (128, 2), (16, 200)])
def test_attend_a_very_long_sequence(heads, rows):
    # 400,000 positions over 5 distinct pages (a prefix may repeat): the exact softmax
    # weighs every slot by how often a row sees it
    c = Batch([(5 * 64, 5 * 64)], 64, spare_pages=0)
    n_pages, length = 6250, 400_000
    pick = torch.randint(0, 5, (n_pages,), generator=gen(3))
    table = c.table[0][pick].view(1, -1).contiguous()
    q = torch.randn(rows, heads, 576, generator=gen(1)).to(torch.bfloat16)
    out = torch.empty(rows, heads, 512, dtype=torch.bfloat16, device=DEV)
    lse = torch.empty(rows, heads, device=DEV)
    smla.smla_paged_attend(q.to(DEV), c.cache(), table.to(DEV), torch.tensor([0, rows], dtype=torch.int32, device=DEV),
                           torch.tensor([length], dtype=torch.int32, device=DEV), 1 / 24, None, out, lse)
    lat, _, rope = unpack(c.rec)
    keys = np.concatenate([lat, rope], 1)
    ids = table[0].numpy()
    for r in sorted({0, rows // 2, rows - 1}):
        seen = length - rows + r + 1
        count = np.bincount(ids[:seen // 64], minlength=5).repeat(64).astype(np.float64)
        if seen % 64:
            tail = int(ids[seen // 64]) * 64
            count[tail:tail + seen % 64] += 1
        s = q[r].double().numpy() @ keys.T / 24
        m = s.max(1, keepdims=True)
        w = np.exp(s - m) * count
        ref_lse = (m[:, 0] + np.log(w.sum(1)))
        ref = (w / w.sum(1, keepdims=True)) @ lat
        spread = (w / w.sum(1, keepdims=True)) @ np.abs(lat)
        # p and the result as bf16, scores in f32 (576 terms), an f32 sum of up to
        # 6250 tiles' sums: 6250 * 2^-24 relative at most
        ds = 2 * 576 * U32 * (np.abs(q[r].double().numpy()) @ np.abs(keys).T).max() / 24
        tol = (2.0 ** -8 + 2 * ds + 6250 * U32) * spread + 2.0 ** -8 * np.abs(ref)
        assert (np.abs(out[r].double().cpu().numpy() - ref) <= tol).all()
        assert (np.abs(lse[r].double().cpu().numpy() - ref_lse) <= ds + 6250 * U32 + 2.0 ** -18 * (1 + np.abs(ref_lse))).all()


def test_a_nan_query_row_stays_in_its_row():
    c = Batch([(9, 100), (1, 300)], 16)
    q, _, want, want_lse, _ = attend(c, 16)
    q2 = q.clone()
    q2[4, 3, 17], q2[4, 5, 570] = float("nan"), float("inf")
    _, _, out, lse, _ = attend(c, 16, q=q2)
    assert torch.isnan(out[4, 3].float()).all() and torch.isnan(lse[4, 3])
    keep = torch.ones(c.rows, 16, dtype=torch.bool)
    keep[4, 3] = keep[4, 5] = False
    assert torch.equal(out.cpu()[keep], want.cpu()[keep]) and torch.equal(lse.cpu()[keep], want_lse.cpu()[keep])


def test_row_boundaries_outside_the_tensors_are_clamped():
    c = Batch([(4, 40), (3, 30)], 16)
    kv, (table, cu, sl) = c.cache(), c.dev()
    cu = torch.tensor([-5, 4, 1000], dtype=torch.int32, device=DEV)  # rows 0..3, 4..6
    q, _, want, want_lse, _ = attend(c, 16)
    out, lse = torch.empty_like(want), torch.empty_like(want_lse)
    smla.smla_paged_attend(q.to(DEV), kv, table, cu, sl, 1 / 24, None, out, lse)
    assert torch.equal(out, want) and torch.equal(lse, want_lse)
    # boundaries that decrease name rows twice or not at all: no access leaves the tensors
    for bad in ([0, 6, 3], [7, 0, 0], [5, 5, 2]):
        smla.smla_paged_attend(q.to(DEV), kv, table, torch.tensor(bad, dtype=torch.int32, device=DEV), sl, 1 / 24, None,
                               out, lse)
        lat, rope = torch.zeros(7, 512, device=DEV), torch.zeros(7, 64, device=DEV)
        smla.smla_paged_read(kv, table, torch.tensor(bad, dtype=torch.int32, device=DEV), sl, lat, rope)
    torch.cuda.synchronize()


def test_attend_without_pages_or_table():
    q = torch.randn(2, 16, 576, generator=gen(0)).to(torch.bfloat16).to(DEV)
    cu, sl = torch.tensor([0, 2], dtype=torch.int32, device=DEV), torch.tensor([9], dtype=torch.int32, device=DEV)
    for kv, table in ((torch.empty(0, 16, REC, dtype=torch.uint8, device=DEV), torch.zeros(1, 3, dtype=torch.int32, device=DEV)),
                      (torch.zeros(2, 16, REC, dtype=torch.uint8, device=DEV), torch.zeros(1, 0, dtype=torch.int32, device=DEV))):
        out, lse = torch.full((2, 16, 512), 7.0, dtype=torch.bfloat16, device=DEV), torch.zeros(2, 16, device=DEV)
        status = torch.zeros(1, dtype=torch.int32, device=DEV)
        smla.smla_paged_attend(q, kv, table, cu, sl, 1 / 24, None, out, lse, status=status)
        assert (out == 0).all() and torch.isneginf(lse).all()
        assert int(status) == smla.STATUS_INDEX_OOB


def test_attend_sharp_softmax_moves_the_reference():
    # scores of some hundreds: the running reference moves often
    c = Batch([(6, 700), (1, 1500)], 64, std=3.0)
    q, sk, out, lse, _ = attend(c, 16, sm_scale=1.0, sink=True)
    check(c, q, out, lse, 1.0, sk, True)
    for scale in (-0.3, 0.0):
        q, sk, out, lse, _ = attend(c, 16, sm_scale=scale)
        check(c, q, out, lse, scale, sk, True)


def test_attend_rows_without_keys():
    # positions before the sequence's start, empty sequences, pages that are not there
    c = Batch([(6, 3), (4, 0), (3, 70), (2, 20)], 16)
    c.table[2, :] = -1
    for causal in (True, False):
        q, sk, out, lse, st = attend(c, 16, causal=causal, sink=True)
        check(c, q, out, lse, 1 / 24, sk, causal)
        assert st == 0
        first = out.float().cpu()
        assert (first[3 if not causal else 0:3] == 0).all() and torch.isneginf(lse[6:10]).all()
        assert (first[6:13] == 0).all() and torch.isneginf(lse[10:13]).all()


def test_attend_bad_pages_are_masked_and_flagged():
    c = Batch([(5, 200), (1, 300)], 16)
    c.table[0, 2], c.table[0, 7] = -1, c.n_pages + 3
    c.table[1, 0] = 2 ** 31 - 1
    q, sk, out, lse, st = attend(c, 16)
    check(c, q, out, lse, 1 / 24, sk, True)
    assert st == smla.STATUS_INDEX_OOB
    # a length past the table: its positions are masked too
    c = Batch([(3, 64)], 16)
    c.seq_lens[0] = 90
    c.lens = [(3, 90)]
    q, sk, out, lse, st = attend(c, 16)
    check(c, q, out, lse, 1 / 24, sk, True)
    assert st == smla.STATUS_INDEX_OOB


def test_attend_strided_q_and_out():
    c = Batch([(7, 90)], 16)
    qb = torch.randn(c.rows, 12, 600, generator=gen(1)).to(torch.bfloat16).to(DEV)
    ob = torch.full((c.rows, 12, 520), 3.0, dtype=torch.bfloat16, device=DEV)
    q, out = qb[:, ::2, 8:584], ob[:, 1::2, :512]
    lse = torch.empty(c.rows, 6, device=DEV)
    smla.smla_paged_attend(q, c.cache(), *c.dev(), 1 / 24, None, out, lse)
    check(c, q.cpu(), out, lse, 1 / 24, None, True)
    assert (ob[:, ::2] == 3.0).all() and (ob[:, :, 512:] == 3.0).all()
    smla.smla_paged_attend(q, c.cache(), *c.dev(), 1 / 24, None, out, None)  # without an LSE


@pytest.mark.parametrize("heads", [16, 128])
def test_attend_returns_every_code_exactly(heads):
    # one key: out is its latent, so every E4M3 code at scales over the fast path's
    # range (subnormal codes included) comes back as bf16(e4m3 * scale)
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


@pytest.mark.parametrize("heads", [16, 128])
def test_attend_foreign_scales_round_once(heads):
    c = Batch([(3, 70)], 16)
    sc = torch.exp2(torch.rand(c.n_pages * 16, 4, generator=gen(4)) * 6 - 4).float().numpy()
    sc[::3] = np.ldexp(1.0, np.random.default_rng(0).integers(-130, 9, sc[::3].shape)).astype(np.float32)
    c.rec[:, 512:528] = sc.view(np.uint8)
    q, sk, out, lse, _ = attend(c, heads)
    # what enters the products is bf16(f32(e4m3 * scale)): the bound gets the half
    # step of k and v
    rows, ref, ref_lse, (a_out, a_lse) = reference_operands(c, q)
    err = np.abs(out.double().cpu().numpy()[rows] - ref) - (a_out + 2.0 ** -8 * np.abs(ref))
    assert err.max() <= 0
    assert (np.abs(lse.double().cpu().numpy()[rows] - ref_lse) <= a_lse + 2.0 ** -18 * (1 + np.abs(ref_lse).max())).all()


def reference_operands(c, q):
    idx, ptr, rows = [], [0], []
    for r, b, p in c.positions():
        idx += [c.slot(b, t) for t in range(p + 1)]
        ptr.append(len(idx))
        rows.append(r)
    idx, ptr = np.array(idx, np.int32), np.array(ptr, np.int32)
    qq = q.double().numpy()[rows]
    out, lse, _ = oracle.sparse_mla_decode(qq, c.rec, idx, ptr, None, 1 / 24, None)
    return rows, out, lse, allowance(qq, c.rec, idx, ptr, None, 1 / 24, None, operand_rel=2.0 ** -8)


@pytest.mark.parametrize("empty", [0, 20])
def test_what_a_row_may_not_see_never_reaches_it(empty):
    # the chunk's later tokens and the slots past the end hold NaN codes, infinite
    # scales and infinite rope: rows before them are as if they were not there
    # (empty sequences choose the kernel of few rows)
    c = Batch([(10, 75)] + [(0, 0)] * empty, 16)
    q, _, want, want_lse, _ = attend(c, 16)
    for p, kind in ((70, 0), (71, 1), (72, 2), (73, 3)):
        s = c.slot(0, p)
        if kind == 0:
            c.rec[s, 7] = 0x7F
        elif kind == 1:
            c.rec[s, 512:516] = np.array([np.inf], np.float32).view(np.uint8)
        elif kind == 2:
            c.rec[s, 528:530] = np.array([0x7F80], np.uint16).view(np.uint8)
        else:
            c.rec[s, 512:516] = np.array([np.nan], np.float32).view(np.uint8)
    i = int(c.table[0, 4]) * 16
    c.rec[i + 11:i + 16] = 0xFF  # slots past the end, in the last page
    _, _, out, lse, _ = attend(c, 16, q=q)
    assert torch.equal(out[:5], want[:5]) and torch.equal(lse[:5], want_lse[:5])
    assert torch.isnan(out[5:].float()).all() and torch.isnan(lse[5:]).all()


def test_attend_agrees_with_the_sparse_decode_on_the_same_cache():
    # write, attend, read back, and the flat decode over the same records
    c = Batch([(4, 300), (1, 120), (12, 12)], 32)
    kv = c.cache()
    lat = torch.randn(c.rows, 512, generator=gen(8)).to(torch.bfloat16).to(DEV)
    rope = torch.randn(c.rows, 64, generator=gen(9)).to(torch.bfloat16).to(DEV)
    table, cu, sl = c.dev()
    smla.smla_paged_write(lat, rope, kv, table, cu, sl)
    flat = kv.view(-1, REC)
    c.rec = flat.cpu().numpy()
    q, sk, out, lse, _ = attend(c, 16, sink=True, kv=kv)
    check(c, q, out, lse, 1 / 24, sk, True)
    idx, ptr = [], [0]
    for r, b, p in c.positions():
        idx += [c.slot(b, t) for t in range(p + 1)]
        ptr.append(len(idx))
    out2, lse2 = torch.empty_like(out), torch.empty_like(lse)
    smla.smla_decode(q.to(DEV), flat, flat.shape[0], torch.tensor(idx, dtype=torch.int32, device=DEV),
                     torch.tensor(ptr, dtype=torch.int32, device=DEV), None, 1 / 24, sk.to(DEV), out2, lse2,
                     kernel=smla.KERNEL_TENSOR_CORE_BF16)
    # both are within 2^-8 (p) + 2^-8 (result) of the exact value, on values up to ~1.5
    assert (out.float() - out2.float()).abs().max() <= 4 * 2.0 ** -8 * 1.5
    assert (lse - lse2).abs().max() <= 1e-4
    l2, r2 = torch.empty_like(lat), torch.empty_like(rope)
    smla.smla_paged_read(kv, table, cu, sl, l2, r2)
    vals, _, _ = unpack(oracle.pack_records(bits(lat), bits(rope)))
    assert torch.equal(l2.cpu().double(), torch.from_numpy(vals)) and torch.equal(r2, rope)


def test_attend_beyond_four_gigabytes():
    page, n_pages = 64, 110_000  # 4.6 GB of records
    kv = torch.zeros(n_pages, page, REC, dtype=torch.uint8, device=DEV)
    c = Batch([(3, 150)], page, spare_pages=0)
    small = c.cache()
    far = torch.tensor([n_pages - 1, n_pages - 2, n_pages // 2 + 1][:c.n_pages])
    kv[far.to(DEV)] = small
    table = far.to(torch.int32)[c.table.long()].to(DEV)
    q = torch.randn(3, 16, 576, generator=gen(0)).to(torch.bfloat16)
    out, lse = torch.empty(3, 16, 512, dtype=torch.bfloat16, device=DEV), torch.empty(3, 16, device=DEV)
    smla.smla_paged_attend(q.to(DEV), kv, table, c.cu.to(DEV), c.seq_lens.to(DEV), 1 / 24, None, out, lse)
    check(c, q, out, lse, 1 / 24, None, True)
    lat = torch.randn(3, 512, generator=gen(1)).to(torch.bfloat16).to(DEV)
    rope = torch.randn(3, 64, generator=gen(2)).to(torch.bfloat16).to(DEV)
    smla.smla_paged_write(lat, rope, kv, table, c.cu.to(DEV), c.seq_lens.to(DEV))
    l2, r2 = torch.empty_like(lat), torch.empty_like(rope)
    smla.smla_paged_read(kv, table, c.cu.to(DEV), c.seq_lens.to(DEV), l2, r2)
    vals, _, _ = unpack(oracle.pack_records(bits(lat), bits(rope)))
    assert torch.equal(l2.cpu().double(), torch.from_numpy(vals)) and torch.equal(r2, rope)


def test_two_graphs_replayed_at_once_with_new_lengths():
    cases = [Batch([(2, 2000), (1, 700)], 32, seed=s) for s in (1, 2)]
    work = []
    for i, c in enumerate(cases):
        q = torch.randn(c.rows, 16, 576, generator=gen(20 + i)).to(torch.bfloat16).to(DEV)
        kv, (table, cu, sl) = c.cache(), c.dev()
        out = torch.zeros(c.rows, 16, 512, dtype=torch.bfloat16, device=DEV)
        lse = torch.zeros(c.rows, 16, device=DEV)
        smla.smla_paged_attend(q, kv, table, cu, sl, 1 / 24, None, out, lse)
        torch.cuda.synchronize()
        graph, stream = torch.cuda.CUDAGraph(), torch.cuda.Stream()
        with torch.cuda.graph(graph, stream=stream):
            smla.smla_paged_attend(q, kv, table, cu, sl, 1 / 24, None, out, lse)
        work.append((c, graph, stream, q, out, lse, sl, kv, table, cu))
    for lens in ([(2, 2000), (1, 700)], [(2, 130), (1, 1900)]):
        for c, graph, stream, q, out, lse, sl, kv, table, cu in work:
            c.lens = lens
            c.table[1, :60] = c.table[0, :60]  # enough pages for either length
            table.copy_(c.table)
            c.seq_lens = torch.tensor([s for _, s in lens], dtype=torch.int32)
            sl.copy_(c.seq_lens)
            out.fill_(7.0)
        torch.cuda.synchronize()
        for _ in range(3):
            for c, graph, stream, *_ in work:
                with torch.cuda.stream(stream):
                    graph.replay()
        torch.cuda.synchronize()
        for c, graph, stream, q, out, lse, *_ in work:
            check(c, q.cpu(), out, lse, 1 / 24, None, True)


def test_streams_and_repeated_calls_give_the_same_bits():
    c = Batch([(3, 3000), (5, 800)], 64)
    q, _, want, want_lse, _ = attend(c, 16)
    kv, tabs, qd = c.cache(), c.dev(), q.to(DEV)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(3)]
    got = []
    for i in range(9):
        s = streams[i % 3]
        out, lse = torch.empty_like(want), torch.empty_like(want_lse)
        smla.smla_paged_attend(qd, kv, *tabs, 1 / 24, None, out, lse,
                               stream=s if i % 2 else s.cuda_stream)
        got.append((out, lse))
    torch.cuda.synchronize()
    for out, lse in got:
        assert torch.equal(out, want) and torch.equal(lse, want_lse)


def test_workspace_of_the_stated_size_suffices():
    c = Batch([(2, 1500), (40, 400)], 64)
    q, _, want, _, _ = attend(c, 16)
    n = smla.smla_paged_attend_workspace_size(c.rows, 16, 2, 64, c.table.shape[1])
    ws = torch.full((n + 4096,), 0xAB, dtype=torch.uint8, device=DEV)
    out, lse = torch.empty_like(want), torch.empty(c.rows, 16, device=DEV)
    smla.smla_paged_attend(q.to(DEV), c.cache(), *c.dev(), 1 / 24, None, out, lse, workspace_tensor=ws[:n])
    assert torch.equal(out, want) and (ws[n:] == 0xAB).all()
    with pytest.raises(smla.SmlaError) as e:
        smla.smla_paged_attend(q.to(DEV), c.cache(), *c.dev(), 1 / 24, None, out, lse, workspace_tensor=ws[:n - 256])
    assert e.value.code == smla.SMLA_ERR_WORKSPACE


def test_empty_batches_do_nothing():
    c = Batch([(0, 50), (0, 0)], 16, behind=3)
    q, _, out, lse, _ = attend(c, 16)
    assert (out == 7.0).all() and (lse == 7.0).all()
    z = torch.zeros(0, dtype=torch.int32, device=DEV)
    e = torch.empty
    smla.smla_paged_write(e(0, 512, device=DEV), e(0, 64, device=DEV), c.cache(), z.view(0, 0),
                          torch.zeros(1, dtype=torch.int32, device=DEV), z)


@pytest.mark.parametrize("heads", [16, 128])
def test_attend_wait_timeout_sets_the_status_and_leaves_the_context_usable(heads):
    c = Batch([(1, 500), (4, 900)], 64)
    try:
        smla.smla_set_wait_limit(20_000_000, stall_first_wait=True)
        *_, st = attend(c, heads)
        assert st & smla.STATUS_TIMEOUT
    finally:
        smla.smla_set_wait_limit(0)
    q, sk, out, lse, st = attend(c, heads)
    assert st == 0
    check(c, q, out, lse, 1 / 24, sk, True)


@pytest.mark.parametrize("seed", range(16))
def test_attend_batches_drawn_at_random(seed):
    # every head count, odd row tiles, more rows than positions, tables that end
    # before the sequence does, pages without a record
    r = np.random.default_rng(100 + seed)
    heads = int(r.choice([1, 3, 7, 16, 18, 33, 40, 64, 90, 128]))
    page = int(r.choice([1, 5, 16, 24, 64, 100]))
    most = 2400 // heads
    lens = [(int(r.integers(0, most)), int(r.integers(0, 700))) for _ in range(int(r.integers(1, 7)))]
    lens.append((1 + most // 3, 400))
    c = Batch(lens, page, seed=seed, front=int(r.integers(0, 3)), behind=int(r.integers(0, 3)), page_pad=48)
    if seed % 2:
        c.table = c.table[:, :max(1, c.table.shape[1] * 2 // 3)].contiguous()
    c.table[torch.rand(c.table.shape, generator=gen(seed)) < 0.08] = -1
    causal, sink = bool(r.integers(0, 4)), bool(r.integers(0, 2))
    q, sk, out, lse, _ = attend(c, heads, causal=causal, sink=sink)
    check(c, q, out, lse, 1 / 24, sk, causal)


def test_sequences_that_share_their_first_pages():
    c = Batch([(3, 200), (1, 170), (20, 100)], 16)
    c.table[1, :8] = c.table[0, :8]
    c.table[2, :4] = c.table[0, :4]
    c.table[2, 4] = c.table[2, 3]  # the same page twice in one history
    q, sk, out, lse, st = attend(c, 16)
    check(c, q, out, lse, 1 / 24, sk, True)
    assert st == 0


def test_attend_refuses_a_scale_that_is_no_finite_f32():
    c = Batch([(1, 20)], 16)
    for scale in (1e40, float("inf"), float("nan")):
        with pytest.raises(smla.SmlaError) as e:
            attend(c, 16, sm_scale=scale)
        assert e.value.code == smla.SMLA_ERR_SHAPE


def test_attend_a_chunk_of_over_a_thousand_row_tiles():
    # 128 heads: a row tile is one token, and the schedule looks for a worker's first
    # one among 1100 in two steps; a sample of the rows is compared
    c = Batch([(2, 40), (1100, 1130), (1, 3)], 64)
    q, sk, out, lse, st = attend(c, 128, sink=True)
    assert st == 0 and torch.isfinite(out.float()).all()
    picked = [x for x in c.positions()][::37]
    idx, ptr = [], [0]
    for _, b, p in picked:
        idx += [c.slot(b, t) for t in range(p + 1)]
        ptr.append(len(idx))
    rows = [r for r, _, _ in picked]
    idx, ptr = np.array(idx, np.int32), np.array(ptr, np.int32)
    qq, s = q.double().numpy()[rows], sk.double().numpy()
    ref, ref_lse, _ = oracle.sparse_mla_decode(qq, c.rec, idx, ptr, None, 1 / 24, s)
    a_out, a_lse = allowance(qq, c.rec, idx, ptr, None, 1 / 24, s)
    err = np.abs(out.double().cpu().numpy()[rows] - ref) - (a_out + 2.0 ** -8 * np.abs(ref) + 1e-30)
    assert err.max() <= 0
    e = np.abs(lse.double().cpu().numpy()[rows] - ref_lse) - (a_lse + 2.0 ** -18 * (1 + np.abs(ref_lse).max()))
    assert e.max() <= 0


# ---- tiles of few rows: empty sequences keep the mean number of rows at 16 or less ----

EMPTY = [(0, 0)] * 60


@pytest.mark.parametrize("page", [1, 20, 64])
@pytest.mark.parametrize("heads,lens", [
    (16, [(1, 95), (1, 96), (1, 97), (2, 192), (1, 1), (5, 3), (1, 700)]), (5, [(7, 1000), (3, 64), (1, 65), (40, 260)]),
    (1, [(33, 33), (16, 500), (17, 1200)]), (16, [(1, 20000)]), (8, [(2, 129), (9, 4000)])])
def test_few_rows(heads, lens, page):
    c = Batch(lens + EMPTY, page, front=2, behind=1, page_pad=32)
    c.table[torch.rand(c.table.shape, generator=gen(1)) < 0.05] = -1
    for causal in (True, False):
        q, sk, out, lse, st = attend(c, heads, causal=causal, sink=causal)
        check(c, q, out, lse, 1 / 24, sk, causal)
        assert st == 0


def test_few_rows_sharp_softmax_and_odd_scales():
    c = Batch([(3, 700), (1, 1500)] + EMPTY, 64, std=3.0)
    for scale in (1.0, -0.3, 0.0):
        q, sk, out, lse, _ = attend(c, 16, sm_scale=scale, sink=True)
        check(c, q, out, lse, scale, sk, True)


def test_few_rows_foreign_scales_round_once():
    c = Batch([(3, 270), (1, 100)] + EMPTY, 16)
    sc = torch.exp2(torch.rand(c.n_pages * 16, 4, generator=gen(4)) * 6 - 4).float().numpy()
    c.rec[:, 512:528] = sc.view(np.uint8)
    q, sk, out, lse, _ = attend(c, 16)
    rows, ref, ref_lse, (a_out, a_lse) = reference_operands(c, q)
    err = np.abs(out.double().cpu().numpy()[rows] - ref) - (a_out + 2.0 ** -8 * np.abs(ref))
    assert err.max() <= 0
    assert (np.abs(lse.double().cpu().numpy()[rows] - ref_lse) <= a_lse + 2.0 ** -18 * (1 + np.abs(ref_lse).max())).all()


def test_few_rows_a_nan_query_row_stays_in_its_row():
    c = Batch([(2, 100), (1, 300)] + EMPTY, 16)
    q, _, want, want_lse, _ = attend(c, 16)
    q2 = q.clone()
    q2[1, 3, 17], q2[1, 5, 570] = float("nan"), float("inf")
    _, _, out, lse, _ = attend(c, 16, q=q2)
    assert torch.isnan(out[1, 3].float()).all() and torch.isnan(lse[1, 3])
    keep = torch.ones(c.rows, 16, dtype=torch.bool)
    keep[1, 3] = keep[1, 5] = False
    assert torch.equal(out.cpu()[keep], want.cpu()[keep]) and torch.equal(lse.cpu()[keep], want_lse.cpu()[keep])


def test_few_rows_many_launches_give_the_same_bits():
    c = Batch([(1, 900), (2, 3000), (1, 50)] + EMPTY, 64)
    q, _, want, want_lse, _ = attend(c, 16)
    kv, q = c.cache(), q.to(DEV)
    flush = torch.empty(256 << 20, dtype=torch.uint8, device=DEV)
    for _ in range(24):
        flush.fill_(1)
        out, lse = torch.empty_like(want), torch.empty_like(want_lse)
        smla.smla_paged_attend(q, kv, *c.dev(), 1 / 24, None, out, lse)
        assert torch.equal(out, want) and torch.equal(lse, want_lse)


def test_few_rows_wait_timeout_sets_the_status_and_leaves_the_context_usable():
    c = Batch([(1, 500), (2, 900)] + EMPTY, 64)
    try:
        smla.smla_set_wait_limit(20_000_000, stall_first_wait=True)
        *_, st = attend(c, 16)
        assert st & smla.STATUS_TIMEOUT
    finally:
        smla.smla_set_wait_limit(0)
    q, sk, out, lse, st = attend(c, 16)
    assert st == 0
    check(c, q, out, lse, 1 / 24, sk, True)

"""smla_paged_append on the GPU: records with rotated rope, rotated queries, against the
rule in 64 bits."""

import numpy as np
import pytest
import torch

import sparse_mla_decode_csr_gb300 as smla
from test_paged_gpu import DEV, REC, TYPES, Batch, expect_records, gen, unpack

pytestmark = pytest.mark.gpu
FREQ = [10000.0 ** (-i / 32) for i in range(32)]
U = 2.0 ** -24


def rotated(x, pos, freq=FREQ, interleaved=True, scale=1.0):
    """x [rows, ..., 64] (f64) rotated by the rows' positions in 64 bits, and the bound of
    the kernel's error before its rounding to bf16.

    Cosine and sine: the angle in half turns is rounded to f32 (relative U of at most one
    half turn: pi U radians) from a fraction cut after 2^-32 turns (2 pi 2^-32), sincospif
    is within 2 U of its values below 1; all times the scale, one rounding.  Together
    under 8 U scale.  Each result is two products and a sum: (8 + 3) U scale (|x| + |y|)."""
    angle = torch.as_tensor(pos, dtype=torch.float64)[:, None] * torch.tensor(freq, dtype=torch.float64)
    angle = angle.view(angle.shape[0], *[1] * (x.dim() - 2), 32)
    c, s = angle.cos() * scale, angle.sin() * scale
    a, b = (x[..., 0::2], x[..., 1::2]) if interleaved else (x[..., :32], x[..., 32:])
    lo, hi, size = a * c - b * s, a * s + b * c, (a.abs() + b.abs()) * 11 * U * abs(scale)
    if interleaved:
        return torch.stack([lo, hi], -1).flatten(-2), torch.stack([size, size], -1).flatten(-2)
    return torch.cat([lo, hi], -1), torch.cat([size, size], -1)


def check_rotated(got, x, pos, what="", **kw):
    """got (bf16) within half a step (2^-8) of what lies within the bound of the exact value."""
    want, bound = rotated(x.double(), pos, **kw)
    err = (got.double().cpu() - want).abs() - (2.0 ** -8 * (want.abs() + bound) + bound)
    assert err.max() <= 0, f"{what}: {err.max():.3g} over the bound"


def inputs(c, heads, dtype, seed=3):
    g = gen(seed)
    lat = torch.randn(c.rows, 512, generator=g) * torch.exp2(torch.randint(-20, 12, (c.rows, 1), generator=g))
    rope, q = torch.randn(c.rows, 64, generator=g), torch.randn(c.rows, heads, 64, generator=g)
    return [t.to(TYPES[dtype]) for t in (lat, rope, q)]


def check_append(c, lat, rope, buf, before, pos, what="", **kw):
    """The cache's bytes after an append: latent and scales bit for bit, the rope within
    its bound, everything else untouched."""
    rec = buf[:, :c.page * REC].reshape(-1, REC).cpu().numpy()
    want = expect_records(lat, rope)
    slots, rows, at = [], [], []
    for r, b, p in c.positions():
        if c.slot(b, p) >= 0:
            slots.append(c.slot(b, p)), rows.append(r), at.append(p if pos is None else int(pos[r]))
    assert np.array_equal(rec[slots, :528], want[rows, :528])
    got = torch.from_numpy(rec[slots, 528:].copy()).view(torch.bfloat16)
    if rows:
        check_rotated(got, rope[rows], at, what, **kw)
    others = np.setdiff1d(np.arange(len(rec)), slots)
    assert np.array_equal(rec[others], before[others])
    assert (buf[:, c.page * REC:] == 0xEE).all()


CASES = [
    # lens, page, page_pad, front, behind, heads
    ([(1, 1)], 1, 0, 0, 0, 1),
    ([(5, 9), (0, 4), (1, 70), (33, 33)], 16, 32, 2, 3, 16),
    ([(3, 100)] * 70, 48, 0, 0, 1, 7),
    ([(300, 1000), (99, 99)], 64, 16, 1, 40, 17),
    ([(20, 30), (1, 5)], 100, 0, 0, 0, 128),
    ([(2, 4), (3, 3)], 5, 0, 1, 0, 40),
]


@pytest.mark.parametrize("interleaved", [True, False])
@pytest.mark.parametrize("dtype", sorted(TYPES))
@pytest.mark.parametrize("lens,page,pad,front,behind,heads", CASES)
def test_append(lens, page, pad, front, behind, heads, dtype, interleaved):
    c = Batch(lens, page, page_pad=pad, front=front, behind=behind)
    lat, rope, q = inputs(c, heads, dtype)
    lat[0] = 0.0
    kv = c.cache()
    wide = torch.zeros(c.rows, 640, dtype=TYPES[dtype], device=DEV)  # strided inputs
    wide[:, :512], wide[:, 512:576] = lat.to(DEV), rope.to(DEV)
    qw = torch.zeros(c.rows, heads, 192, dtype=TYPES[dtype], device=DEV)
    qw[..., 128:] = q.to(DEV)
    out = torch.full((c.rows, heads, 576), 7.0, dtype=torch.bfloat16, device=DEV)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    smla.smla_paged_append(wide[:, :512], wide[:, 512:576], kv, *c.dev(), smla.smla_rotation_turns(FREQ),
                           q_rope=qw[..., 128:], q_out=out[..., 512:], interleaved=interleaved, status=status)
    check_append(c, lat, rope, c.buf, c.rec, None, "rope", interleaved=interleaved)
    mine = {r: p for r, _, p in c.positions()}
    rows = sorted(mine)
    check_rotated(out[rows, :, 512:], q[rows], [mine[r] for r in rows], "q", interleaved=interleaved)
    assert (out[..., :512] == 7.0).all()
    others = [r for r in range(c.rows) if r not in mine]
    assert (out[others] == 7.0).all()
    assert int(status) == 0


@pytest.mark.parametrize("interleaved", [True, False])
def test_positions_of_their_own_at_any_distance(interleaved):
    # where an f32 angle would be off by whole turns; frequencies above one radian and negative ones
    pos = [0, 1, -1, 100_000, 1_000_003, 2 ** 24 + 1, 2 ** 30, 2 ** 31 - 1, -(2 ** 31), 77]
    freq = [2.5, -1.0, 0.0, 1e-6] + FREQ[:28]
    c = Batch([(10, 200)], 16)
    lat, rope, q = inputs(c, 3, "f32")
    kv = c.cache()
    out = torch.zeros(10, 3, 64, dtype=torch.bfloat16, device=DEV)
    smla.smla_paged_append(lat.to(DEV), rope.to(DEV), kv, *c.dev(), smla.smla_rotation_turns(torch.tensor(freq)),
                           q_rope=q.to(DEV), q_out=out, positions=torch.tensor(pos, dtype=torch.int32, device=DEV),
                           interleaved=interleaved, rope_scale=-1.25)
    # The oracle's angle, an f64 product, is off by half a step: 2^-53 of up to 2^31 * 2.5
    # radians, 2^-20.7.  The first seven positions' are below 2^-28, within the bound's slack.
    freq64 = torch.tensor(freq).double().tolist()  # (the table's are these f32 values)
    want, bound = rotated(q.double(), pos, freq64, interleaved, -1.25)
    slack = torch.tensor([abs(p) > 2 ** 24 + 1 for p in pos]).double().view(-1, 1, 1) * 2.0 ** -20.7 * 1.25
    slack = slack * 2 * q.abs().amax().double()
    err = (out.double().cpu() - want).abs() - (2.0 ** -8 * (want.abs() + bound) + bound + slack)
    assert err.max() <= 0
    rec = kv.view(-1, REC)[[c.slot(0, 190 + i) for i in range(10)]].cpu()
    got = rec[:, 528:].contiguous().view(torch.bfloat16).double()
    want, bound = rotated(rope.double(), pos, freq64, interleaved, -1.25)
    err = (got - want).abs() - (2.0 ** -8 * (want.abs() + bound) + bound + slack[:, 0] * rope.abs().amax() / q.abs().amax())
    assert err.max() <= 0


def test_position_zero_returns_the_values():
    c = Batch([(4, 4)], 16)
    lat, rope, q = inputs(c, 5, "bf16")
    zero = torch.zeros(4, dtype=torch.int32, device=DEV)
    kv, turns = c.cache(), smla.smla_rotation_turns(FREQ)
    for interleaved in (True, False):
        out = torch.empty(4, 5, 64, dtype=torch.bfloat16, device=DEV)
        smla.smla_paged_append(lat.to(DEV), rope.to(DEV), kv, *c.dev(), turns, q_rope=q.to(DEV), q_out=out,
                               positions=zero, interleaved=interleaved)
        assert torch.equal(out.cpu(), q)
        plain = torch.empty_like(kv).copy_(kv)
        smla.smla_paged_write(lat.to(DEV), rope.to(DEV), plain, *c.dev())
        assert torch.equal(plain, kv)


@pytest.mark.parametrize("interleaved", [True, False])
def test_queries_in_place_and_none(interleaved):
    c = Batch([(9, 40), (3, 300)], 16, behind=2)
    lat, rope, q = inputs(c, 19, "bf16")
    turns, kv = smla.smla_rotation_turns(FREQ), c.cache()
    out = torch.full((c.rows, 19, 64), 7.0, dtype=torch.bfloat16, device=DEV)
    args = (lat.to(DEV), rope.to(DEV), kv, *c.dev(), turns)
    smla.smla_paged_append(*args, q_rope=q.to(DEV), q_out=out, interleaved=interleaved)
    whole = torch.full((c.rows, 19, 576), 3.0, dtype=torch.bfloat16, device=DEV)
    whole[..., 512:] = q.to(DEV)
    smla.smla_paged_append(*args, q_rope=whole[..., 512:], q_out=whole[..., 512:], interleaved=interleaved)
    assert torch.equal(whole[:12, :, 512:], out[:12]) and (whole[..., :512] == 3.0).all()
    assert torch.equal(whole[12:, :, 512:].cpu(), q[12:]) and (out[12:] == 7.0).all()
    once = kv.clone()
    kv2 = c.cache()
    smla.smla_paged_append(args[0], args[1], kv2, *args[3:], interleaved=interleaved)
    assert torch.equal(kv2, once)


def test_masked_rows_turn_their_queries_and_are_flagged():
    c = Batch([(40, 40), (40, 30), (8, 200), (8, 8)], 16)
    c.table[0, 1] = -1
    c.seq_lens[2] = 16 * c.table.shape[1] + 4  # the last four rows lie past the table
    c.lens[2] = (8, int(c.seq_lens[2]))
    c.table[2, -1] = 0
    lat, rope, q = inputs(c, 2, "f16")
    for oob in (False, True):
        c.table[3, 0] = c.n_pages if oob else c.n_pages - 1
        status = torch.zeros(1, dtype=torch.int32, device=DEV)
        out = torch.zeros(c.rows, 2, 64, dtype=torch.bfloat16, device=DEV)
        smla.smla_paged_append(lat.to(DEV), rope.to(DEV), c.cache(), *c.dev(), smla.smla_rotation_turns(FREQ),
                               q_rope=q.to(DEV), q_out=out, status=status)
        check_append(c, lat, rope, c.buf, c.rec, None)
        check_rotated(out, q, [p for _, _, p in c.positions()])
        assert int(status) == smla.STATUS_INDEX_OOB


def test_values_that_are_not_finite():
    c = Batch([(3, 3)], 16)
    lat, rope, q = inputs(c, 1, "f32")
    rope[1, 0], rope[1, 2], q[2, 0, 5] = float("nan"), float("inf"), float("inf")
    out = torch.zeros(3, 1, 64, dtype=torch.bfloat16, device=DEV)
    kv = c.cache()
    smla.smla_paged_append(lat.to(DEV), rope.to(DEV), kv, *c.dev(), smla.smla_rotation_turns(FREQ), q_rope=q.to(DEV),
                           q_out=out)
    _, _, r = unpack(kv.view(-1, REC).cpu().numpy())
    got = r[c.slot(0, 1)]
    assert np.isnan(got[:2]).all() and np.isinf(got[2:4]).all() and np.isfinite(got[4:]).all()
    o = out[2, 0].float().cpu()
    assert torch.isinf(o[4:6]).all() and torch.isfinite(o[:4]).all() and torch.isfinite(o[6:]).all()


def test_many_empty_sequences_and_clamped_boundaries():
    lens = [(2, 20)] + [(0, 7)] * 700 + [(3, 9)] + [(0, 0)] * 1500 + [(1, 1)]
    c = Batch(lens, 16)
    lat, rope, q = inputs(c, 3, "bf16")
    kv = c.cache()
    out = torch.zeros(6, 3, 64, dtype=torch.bfloat16, device=DEV)
    table, cu, sl = c.dev()
    cu[0], cu[-1] = -9, 4000
    smla.smla_paged_append(lat.to(DEV), rope.to(DEV), kv, table, cu, sl, smla.smla_rotation_turns(FREQ),
                           q_rope=q.to(DEV), q_out=out)
    check_append(c, lat, rope, c.buf, c.rec, None)
    check_rotated(out, q, [p for _, _, p in c.positions()])


def test_append_refuses_a_scale_that_is_no_finite_f32():
    c = Batch([(1, 2)], 16)
    lat, rope, _ = inputs(c, 1, "bf16")
    for scale in (1e40, float("inf"), float("nan")):
        with pytest.raises(smla.SmlaError) as e:
            smla.smla_paged_append(lat.to(DEV), rope.to(DEV), c.cache(), *c.dev(), smla.smla_rotation_turns(FREQ),
                                   rope_scale=scale)
        assert e.value.code == smla.SMLA_ERR_SHAPE


def test_append_beyond_four_gigabytes():
    page, n_pages = 64, 110_000  # 4.6 GB of records
    kv = torch.zeros(n_pages, page, REC, dtype=torch.uint8, device=DEV)
    c = Batch([(70, 150)], page, spare_pages=0)
    far = torch.tensor([n_pages - 1, n_pages - 2, n_pages // 2 + 1][:c.n_pages])
    table = far.to(torch.int32)[c.table.long()].to(DEV)
    lat, rope, _ = inputs(c, 1, "bf16")
    smla.smla_paged_append(lat.to(DEV), rope.to(DEV), kv, table, c.cu.to(DEV), c.seq_lens.to(DEV),
                           smla.smla_rotation_turns(FREQ))
    c.rec[:] = 0
    got = kv[far.to(DEV)].view(len(far), -1)
    check_append(c, lat, rope, got, c.rec, None)

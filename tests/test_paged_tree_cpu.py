"""The rotation table, and the argument checks of the append and tree calls, on the
host: the C entry points before any CUDA call, and the binding's checks of tensors."""

import ctypes
import math
from fractions import Fraction

import pytest
import torch

import sparse_mla_decode_csr_gb300 as smla
from test_paged_cpu import BAD, BATCH_CASES, SHARED, attend_params, batch, tensors

# 1 / (2 pi) to 50 decimal places, from pi's
PI = Fraction(314159265358979323846264338327950288419716939937510, 10 ** 50)


def turns_of(freq):
    return [int(v) for v in smla.smla_rotation_turns(freq, device="cpu")]


def test_turns_are_the_fraction_of_a_turn():
    r = torch.Generator().manual_seed(1)
    freq = [0.0, 1.0, -1.0, math.pi, 2 * math.pi, -2 * math.pi, 1e-3, -1e-17, 1e-19, 2.0 ** 32, -(2.0 ** 32), 123456.789]
    freq += [10000.0 ** (-i / 32) for i in range(10)]
    freq += (torch.randn(32 - len(freq), generator=r, dtype=torch.float64) * 1000).tolist()
    for f, t in zip(freq, turns_of(freq)):
        want = Fraction(f) / (2 * PI) * 2 ** 64
        off = (Fraction(t) - want) % 2 ** 64
        off = min(off, 2 ** 64 - off)
        # one rounding to a whole step, and 1 / (2 pi) and its product to 106 bits
        assert off <= Fraction(1, 2) + abs(want) / 2 ** 100, f


def test_turns_refuse_what_is_no_angle():
    good = [0.5] * 32
    for bad in (float("nan"), float("inf"), -float("inf"), 2.0 ** 32 * 1.001):
        with pytest.raises(smla.SmlaError) as e:
            smla.smla_rotation_turns(good[:31] + [bad], device="cpu")
        assert e.value.code == BAD["shape"]
    for bad in (good[:31], good + [0.5], torch.zeros(4, 8)):
        with pytest.raises(smla.SmlaError):
            smla.smla_rotation_turns(bad, device="cpu")
    assert smla.lib.smla_rotation_turns(None, None) == -1


# ---- the C entry points ----


def append_params(b=None, **kw):
    p = smla.PagedAppendParams()
    p.batch = b if b is not None else batch()
    p.latent, p.latent_stride, p.rope, p.rope_stride = 0x50000, 512, 0x60000, 64
    p.dtype, p.interleaved, p.turns, p.rope_scale = 0, 1, 0x70000, 1.0
    p.num_heads, p.q_rope, p.q_out = 16, 0x80000, 0x90000
    p.q_rope_stride_row, p.q_rope_stride_head = 16 * 64, 64
    p.q_out_stride_row, p.q_out_stride_head = 16 * 576, 576
    for k, v in kw.items():
        setattr(p, k, v)
    return p


@pytest.mark.parametrize("kw,code", BATCH_CASES)
def test_append_accept_and_attend_reject_a_bad_batch(kw, code):
    b = batch(**kw)
    assert smla.lib.smla_paged_append(ctypes.byref(append_params(b)), None) == code
    assert smla.lib.smla_paged_accept(ctypes.byref(b), 0x50000, 8, 8, 0x60000, None) == code
    p = attend_params(b)
    assert smla.lib.smla_paged_attend_tree(ctypes.byref(p), 0x70000, 2, 2, None, 0, None) == code


@pytest.mark.parametrize("kw,code", [
    (dict(latent=None), -1), (dict(rope=None), -1), (dict(turns=None), -1), (dict(q_rope=None), -1), (dict(q_out=None), -1),
    (dict(dtype=3), -2), (dict(dtype=-1), -2), (dict(num_heads=-1), -2), (dict(num_heads=129), -2),
    (dict(rope_scale=float("nan")), -2), (dict(rope_scale=float("inf")), -2),
    (dict(latent_stride=511), -3), (dict(rope_stride=63), -3), (dict(q_rope_stride_head=56), -3),
    (dict(q_out_stride_head=56), -3), (dict(q_rope_stride_row=1016), -3), (dict(q_out_stride_row=576), -3),
    (dict(q_rope_stride_row=-1024), -3), (dict(q_out_stride_head=-64), -3),
    (dict(latent=0x50008), -4), (dict(rope=0x60008), -4), (dict(turns=0x70004), -4), (dict(positions=0xA0002), -4),
    (dict(q_rope=0x80008), -4), (dict(q_out=0x90008), -4), (dict(q_rope_stride_head=68, q_rope_stride_row=16 * 68), -4),
    (dict(q_out_stride_head=580, q_out_stride_row=16 * 580), -4), (dict(q_rope_stride_row=16 * 64 + 4), -4),
])
def test_append_rejects_bad_tensors(kw, code):
    assert smla.lib.smla_paged_append(ctypes.byref(append_params(**kw)), None) == code


def test_append_without_queries_asks_for_none():
    # (no device here: what passes the checks ends there)
    p = append_params(num_heads=0, q_rope=None, q_out=None)
    assert smla.lib.smla_paged_append(ctypes.byref(p), None) in (BAD["device"], -8)
    p.dtype, p.q_rope_stride_head = 2, 3
    assert smla.lib.smla_paged_append(ctypes.byref(p), None) in (BAD["device"], -8)


TREE = dict(parents=0x50000, cu=0x30000, lens=0x40000, rows=10, seqs=2, mask=0x60000, stride=2, words=2,
            positions=0x70000, status=None, stream=None)


@pytest.mark.parametrize("kw,code", [
    (dict(parents=None), -1), (dict(cu=None), -1), (dict(lens=None), -1), (dict(mask=None), -1),
    (dict(mask=None, words=0, positions=None), -1),
    (dict(rows=-1), -2), (dict(rows=(1 << 30) + 1), -2), (dict(seqs=-1), -2), (dict(seqs=(1 << 24) + 1), -2),
    (dict(words=-1), -2), (dict(words=(1 << 25) + 1, stride=1 << 26), -2), (dict(stride=1), -3), (dict(mask=0x60002), -4),
    (dict(rows=0, parents=None), 0), (dict(seqs=0, cu=None, lens=None), 0),
])
def test_tree_rejects_bad_arguments(kw, code):
    assert smla.lib.smla_paged_tree(*{**TREE, **kw}.values()) == code


@pytest.mark.parametrize("args,code", [
    ((None, 2, 2), -1), ((0x70000, 1, 2), -3), ((0x70002, 2, 2), -4), ((0x70000, 2, -1), -2),
    ((0x70000, 1 << 26, (1 << 25) + 1), -2)])
def test_attend_tree_rejects_bad_masks(args, code):
    assert smla.lib.smla_paged_attend_tree(ctypes.byref(attend_params()), *args, None, 0, None) == code


@pytest.mark.parametrize("args,code", [
    ((None, 8, 8, 0x60000), -1), ((0x50000, 8, 8, None), -1), ((0x50000, 8, -1, 0x60000), -2),
    ((0x50000, 7, 8, 0x60000), -3), ((0x50002, 8, 8, 0x60000), -4), ((0x50000, 8, 8, 0x60002), -4)])
def test_accept_rejects_bad_arguments(args, code):
    assert smla.lib.smla_paged_accept(ctypes.byref(batch()), *args, None) == code


def test_null_structs_and_empty_batches():
    assert smla.lib.smla_paged_append(None, None) == -1
    assert smla.lib.smla_paged_attend_tree(None, None, 0, 0, None, 0, None) == -1
    assert smla.lib.smla_paged_accept(None, None, 0, 0, None, None) == -1
    for kw in (dict(n_rows=0), dict(n_seqs=0)):
        b = batch(cu_rows=None, seq_lens=None, kv_cache=None, block_table=None, **kw)
        p = append_params(b, latent=None, rope=None, turns=None, q_rope=None, q_out=None)
        assert smla.lib.smla_paged_append(ctypes.byref(p), None) == 0
        p = attend_params(b, q=None, out=None)
        assert smla.lib.smla_paged_attend_tree(ctypes.byref(p), None, 0, 0, None, 0, None) == 0
    b = batch(cu_rows=None, seq_lens=None, kv_cache=None, block_table=None, n_seqs=0)
    assert smla.lib.smla_paged_accept(ctypes.byref(b), None, 0, 0, None, None) == 0
    # without rows there are lengths to write all the same
    assert smla.lib.smla_paged_accept(ctypes.byref(batch(n_rows=0, cu_rows=None)), 0x50000, 8, 8, 0x60000, None) == -1


# ---- the binding ----

I32 = torch.int32


def more(**kw):
    t = tensors()
    t.update(turns=torch.zeros(32, dtype=torch.int64), qr=torch.zeros(5, 4, 64), qo=torch.zeros(5, 4, 64, dtype=torch.bfloat16),
             pos=torch.zeros(5, dtype=I32), mask=torch.zeros(5, 2, dtype=I32), parents=torch.zeros(5, dtype=I32),
             path=torch.zeros(2, 3, dtype=I32), new=torch.zeros(2, dtype=I32))
    t.update(kw)
    return t


def call_append(t):
    smla.smla_paged_append(t["lat"], t["rope"], t["kv"], t["table"], t["cu"], t["sl"], t["turns"], q_rope=t["qr"],
                           q_out=t["qo"], positions=t["pos"], status=t["status"])


def call_tree(t):
    smla.smla_paged_tree(t["parents"], t["cu"], t["sl"], t["mask"], t["pos"], status=t["status"])


def call_attend_tree(t):
    smla.smla_paged_attend_tree(t["q"], t["kv"], t["table"], t["cu"], t["sl"], t["mask"], 0.05, t["sink"], t["out"],
                                t["lse"], status=t["status"], workspace_tensor=t.get("ws"))


def call_accept(t):
    smla.smla_paged_accept(t["kv"], t["table"], t["cu"], t["sl"], t["path"], t["new"], status=t["status"])


@pytest.mark.parametrize("kw,why", SHARED)
@pytest.mark.parametrize("call", [call_append, call_attend_tree, call_accept])
def test_the_binding_checks_the_batch(call, kw, why):
    with pytest.raises(smla.SmlaError) as e:
        call(more(**kw))
    assert e.value.code == BAD[why]


@pytest.mark.parametrize("kw,why", [
    (dict(lat=torch.zeros(5, 512, dtype=torch.float64)), "shape"), (dict(rope=torch.zeros(5, 64, dtype=torch.float16)), "shape"),
    (dict(lat=torch.zeros(5, 1024)[:, ::2]), "stride"), (dict(rope=torch.zeros(4, 64)), "shape"),
    (dict(turns=torch.zeros(32)), "shape"), (dict(turns=torch.zeros(31, dtype=torch.int64)), "shape"),
    (dict(turns=torch.zeros(64, dtype=torch.int64)[::2]), "shape"),
    (dict(pos=torch.zeros(5, dtype=torch.int64)), "shape"), (dict(pos=torch.zeros(4, dtype=I32)), "shape"),
    (dict(pos=torch.zeros(10, dtype=I32)[::2]), "stride"),
    (dict(qr=None), "null"), (dict(qo=None), "null"),
    (dict(qr=torch.zeros(5, 4, 64, dtype=torch.bfloat16)), "shape"), (dict(qo=torch.zeros(5, 4, 64)), "shape"),
    (dict(qr=torch.zeros(5, 4, 63)), "shape"), (dict(qr=torch.zeros(5, 3, 64)), "shape"), (dict(qr=torch.zeros(5, 256)), "shape"),
    (dict(qo=torch.zeros(5, 256, dtype=torch.bfloat16)), "shape"),
    (dict(qr=torch.zeros(5, 4, 128)[..., ::2]), "stride"), (dict(qo=torch.zeros(5, 4, 128, dtype=torch.bfloat16)[..., ::2]), "stride"),
    (dict(), "device"),
])
def test_the_binding_checks_append(kw, why):
    with pytest.raises(smla.SmlaError) as e:
        call_append(more(**kw))
    assert e.value.code == BAD[why]


MASKS = [(dict(mask=torch.zeros(5, 2)), "shape"), (dict(mask=torch.zeros(4, 2, dtype=I32)), "shape"),
         (dict(mask=torch.zeros(10, dtype=I32)), "shape"), (dict(mask=torch.zeros(5, 4, dtype=I32)[:, ::2]), "stride")]


@pytest.mark.parametrize("kw,why", MASKS + [
    (dict(mask=None), "null"), (dict(q=torch.zeros(5, 4, 576)), "shape"), (dict(out=torch.zeros(5, 4, 512)), "shape"),
    (dict(sink=torch.zeros(3)), "shape"), (dict(ws=torch.zeros(1, dtype=torch.uint8).expand(1 << 30)), "stride"),
    (dict(lse=torch.zeros(4, 5)), "shape"), (dict(), "device")])
def test_the_binding_checks_attend_tree(kw, why):
    with pytest.raises(smla.SmlaError) as e:
        call_attend_tree(more(**kw))
    assert e.value.code == BAD[why]


@pytest.mark.parametrize("kw,why", MASKS + [
    (dict(parents=torch.zeros(5)), "shape"), (dict(parents=torch.zeros(5, 1, dtype=I32)), "shape"),
    (dict(parents=torch.zeros(10, dtype=I32)[::2]), "stride"), (dict(pos=torch.zeros(10, dtype=I32)[::2]), "stride"),
    (dict(pos=torch.zeros(6, dtype=I32)), "shape"), (dict(pos=torch.zeros(5)), "shape"),
    (dict(cu=torch.zeros(2, dtype=I32)), "shape"), (dict(cu=torch.zeros(6, dtype=I32)[::2]), "stride"),
    (dict(sl=torch.zeros(2)), "shape"), (dict(sl=torch.zeros(4, dtype=I32)[::2]), "stride"),
    (dict(status=torch.zeros(1)), "shape"), (dict(), "device")])
def test_the_binding_checks_tree(kw, why):
    with pytest.raises(smla.SmlaError) as e:
        call_tree(more(**kw))
    assert e.value.code == BAD[why]


@pytest.mark.parametrize("kw,why", [
    (dict(path=torch.zeros(2, 3)), "shape"), (dict(path=torch.zeros(3, 3, dtype=I32)), "shape"),
    (dict(path=torch.zeros(6, dtype=I32)), "shape"), (dict(path=torch.zeros(2, 6, dtype=I32)[:, ::2]), "stride"),
    (dict(new=torch.zeros(2)), "shape"), (dict(new=torch.zeros(3, dtype=I32)), "shape"),
    (dict(new=torch.zeros(4, dtype=I32)[::2]), "stride"), (dict(), "device")])
def test_the_binding_checks_accept(kw, why):
    with pytest.raises(smla.SmlaError) as e:
        call_accept(more(**kw))
    assert e.value.code == BAD[why]


def test_packed_append_has_the_c_layout():
    values = list(range(101, 113))
    rest = [201, 202, 203, 204, 1, 0, 207, 0.25, 209, 210, 211, 212, 213, 214, 215, 216]
    assert bytes(smla.PagedAppendParams(smla.PagedBatch(*values), *rest)) == smla._pack_append(*values, *rest)

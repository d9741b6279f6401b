"""The paged cache's argument checks, on the host: the C entry points before any
CUDA call, and the binding's checks of tensors."""

import ctypes

import pytest
import torch

import sparse_mla_decode_csr_gb300 as smla

BAD = dict(null=-1, shape=-2, stride=-3, align=-4, device=-7)


def batch(**kw):
    b = smla.PagedBatch()
    b.kv_cache, b.n_pages, b.page_size, b.page_stride = 0x10000, 8, 16, 16 * 656
    b.block_table, b.block_table_stride, b.max_pages = 0x20000, 4, 4
    b.cu_rows, b.seq_lens, b.n_rows, b.n_seqs = 0x30000, 0x40000, 10, 2
    for k, v in kw.items():
        setattr(b, k, v)
    return b


BATCH_CASES = [
    (dict(n_rows=-1), -2), (dict(n_rows=(1 << 30) + 1), -2), (dict(n_seqs=-1), -2), (dict(n_seqs=(1 << 24) + 1), -2),
    (dict(n_pages=-1), -2), (dict(page_size=0), -2), (dict(max_pages=-1), -2),
    (dict(max_pages=1 << 20, page_size=2048, page_stride=2048 * 656, block_table_stride=1 << 20), -2),
    (dict(cu_rows=None), -1), (dict(seq_lens=None), -1), (dict(block_table=None), -1), (dict(kv_cache=None), -1),
    (dict(page_stride=16 * 656 - 16), -3), (dict(block_table_stride=3), -3),
    (dict(page_stride=16 * 656 + 8), -4), (dict(kv_cache=0x10008), -4),
]


@pytest.mark.parametrize("kw,code", BATCH_CASES)
def test_every_entry_point_rejects_a_bad_batch(kw, code):
    b = batch(**kw)
    for f in (smla.lib.smla_paged_write, smla.lib.smla_paged_read):
        assert f(ctypes.byref(b), 0x50000, 512, 0x60000, 64, 0, None) == code
    assert smla.lib.smla_paged_attend(ctypes.byref(attend_params(b)), None, 0, None) == code


def attend_params(b=None, **kw):
    p = smla.PagedAttendParams()
    p.batch = b if b is not None else batch()
    p.num_heads, p.causal, p.sm_scale = 16, 1, 0.05
    p.q, p.q_stride_row, p.q_stride_head = 0x50000, 16 * 576, 576
    p.out, p.out_stride_row, p.out_stride_head = 0x60000, 16 * 512, 512
    for k, v in kw.items():
        setattr(p, k, v)
    return p


@pytest.mark.parametrize("args,code", [
    ((None, 512, 0x60000, 64, 0), -1), ((0x50000, 512, None, 64, 0), -1),
    ((0x50000, 511, 0x60000, 64, 0), -3), ((0x50000, 512, 0x60000, 63, 0), -3),
    ((0x50008, 512, 0x60000, 64, 0), -4), ((0x50000, 512, 0x60004, 64, 0), -4),
    ((0x50000, 516, 0x60000, 64, 0), -4), ((0x50000, 514, 0x60000, 64, 2), -4),
    ((0x50000, 512, 0x60000, 64, 3), -2), ((0x50000, 512, 0x60000, 64, -1), -2),
])
def test_write_and_read_reject_bad_tensors(args, code):
    b = batch()
    for f in (smla.lib.smla_paged_write, smla.lib.smla_paged_read):
        assert f(ctypes.byref(b), *args, None) == code


@pytest.mark.parametrize("kw,code", [
    (dict(num_heads=0), -2), (dict(num_heads=129), -2), (dict(sm_scale=float("nan")), -2),
    (dict(sm_scale=float("inf")), -2), (dict(q=None), -1), (dict(out=None), -1),
    (dict(q_stride_head=575), -3), (dict(out_stride_head=504), -3), (dict(q_stride_row=576), -3),
    (dict(out_stride_row=512), -3), (dict(q_stride_row=-16), -3), (dict(q=0x50008), -4), (dict(out=0x60004), -4),
    (dict(q_stride_row=16 * 576 + 4), -4), (dict(out_stride_head=516, out_stride_row=16 * 516), -4),
])
def test_attend_rejects_bad_tensors(kw, code):
    assert smla.lib.smla_paged_attend(ctypes.byref(attend_params(**kw)), None, 0, None) == code


def test_null_structs_are_named():
    assert smla.lib.smla_paged_attend(None, None, 0, None) == -1
    assert smla.lib.smla_paged_write(None, 0x50000, 512, 0x60000, 64, 0, None) == -1
    assert smla.lib.smla_paged_read(None, 0x50000, 512, 0x60000, 64, 0, None) == -1
    assert smla.lib.smla_paged_attend_workspace_size(None) == 0


@pytest.mark.parametrize("kw", [dict(n_rows=0), dict(n_seqs=0)])
def test_empty_batches_are_a_noop(kw):
    b = batch(cu_rows=None, seq_lens=None, kv_cache=None, block_table=None, **kw)
    assert smla.lib.smla_paged_write(ctypes.byref(b), None, 0, None, 0, 0, None) == 0
    assert smla.lib.smla_paged_read(ctypes.byref(b), None, 0, None, 0, 2, None) == 0
    p = attend_params(b, q=None, out=None)
    assert smla.lib.smla_paged_attend(ctypes.byref(p), None, 0, None) == 0
    assert smla.lib.smla_paged_attend_workspace_size(ctypes.byref(p)) == 0


def tensors(rows=5, heads=4, pages=6, page=16, seqs=2, width=3):
    return dict(
        kv=torch.zeros(pages, page, 656, dtype=torch.uint8), table=torch.zeros(seqs, width, dtype=torch.int32),
        cu=torch.zeros(seqs + 1, dtype=torch.int32), sl=torch.zeros(seqs, dtype=torch.int32),
        lat=torch.zeros(rows, 512), rope=torch.zeros(rows, 64),
        q=torch.zeros(rows, heads, 576, dtype=torch.bfloat16), out=torch.zeros(rows, heads, 512, dtype=torch.bfloat16),
        lse=torch.zeros(rows, heads), sink=torch.zeros(heads), status=torch.zeros(1, dtype=torch.int32))


def call_write(t):
    smla.smla_paged_write(t["lat"], t["rope"], t["kv"], t["table"], t["cu"], t["sl"], status=t["status"])


def call_read(t):
    smla.smla_paged_read(t["kv"], t["table"], t["cu"], t["sl"], t["lat"], t["rope"], status=t["status"])


def call_attend(t):
    smla.smla_paged_attend(t["q"], t["kv"], t["table"], t["cu"], t["sl"], 0.05, t["sink"], t["out"], t["lse"],
                           status=t["status"], workspace_tensor=t.get("ws"))


SHARED = [
    (dict(kv=torch.zeros(6, 16, 655, dtype=torch.uint8)), "shape"),
    (dict(kv=torch.zeros(6, 16, 656, dtype=torch.int8)), "shape"),
    (dict(kv=torch.zeros(96, 656, dtype=torch.uint8)), "shape"),
    (dict(kv=torch.zeros(0, 1 << 31, 656, dtype=torch.uint8)), "shape"),
    (dict(kv=torch.zeros(6, 16, 1312, dtype=torch.uint8)[..., ::2]), "stride"),
    (dict(kv=torch.zeros(6, 16, 672, dtype=torch.uint8)[..., :656]), "stride"),
    (dict(table=torch.zeros(2, 3, dtype=torch.int64)), "shape"),
    (dict(table=torch.zeros(3, 3, dtype=torch.int32)), "shape"),
    (dict(table=torch.zeros(2, 6, dtype=torch.int32)[:, ::2]), "stride"),
    (dict(cu=torch.zeros(2, dtype=torch.int32)), "shape"),
    (dict(cu=torch.zeros(6, dtype=torch.int32)[::2]), "stride"),
    (dict(sl=torch.zeros(2)), "shape"),
    (dict(sl=torch.zeros(4, dtype=torch.int32)[::2]), "stride"),
    (dict(status=torch.zeros(1)), "shape"),
    (dict(), "device"),  # host tensors
]


@pytest.mark.parametrize("kw,why", SHARED + [
    (dict(lat=torch.zeros(5, 512, dtype=torch.float64)), "shape"),
    (dict(rope=torch.zeros(5, 64, dtype=torch.bfloat16)), "shape"),
    (dict(lat=torch.zeros(5, 511)), "shape"), (dict(rope=torch.zeros(4, 64)), "shape"),
    (dict(lat=torch.zeros(5, 1024)[:, ::2]), "stride"),
])
@pytest.mark.parametrize("call", [call_write, call_read])
def test_the_binding_checks_write_and_read(call, kw, why):
    with pytest.raises(smla.SmlaError) as e:
        call({**tensors(), **kw})
    assert e.value.code == BAD[why]


@pytest.mark.parametrize("kw,why", SHARED + [
    (dict(q=torch.zeros(5, 4, 576)), "shape"), (dict(q=torch.zeros(5, 4, 512, dtype=torch.bfloat16)), "shape"),
    (dict(out=torch.zeros(5, 4, 512)), "shape"), (dict(out=torch.zeros(5, 3, 512, dtype=torch.bfloat16)), "shape"),
    (dict(q=torch.zeros(5, 4, 1152, dtype=torch.bfloat16)[..., ::2]), "stride"),
    (dict(sink=torch.zeros(3)), "shape"), (dict(sink=torch.zeros(4, dtype=torch.bfloat16)), "shape"),
    (dict(ws=torch.zeros(1, dtype=torch.uint8).expand(1 << 30)), "stride"),
    (dict(lse=torch.zeros(4, 5)), "shape"), (dict(lse=torch.zeros(5, 8)[:, ::2]), "shape"),
])
def test_the_binding_checks_attend(kw, why):
    with pytest.raises(smla.SmlaError) as e:
        call_attend({**tensors(), **kw})
    assert e.value.code == BAD[why]


@pytest.mark.parametrize("kw", [dict(n_rows=(1 << 30) + 1), dict(n_seqs=(1 << 24) + 1), dict(page_size=0),
                                dict(page_size=1 << 16, max_pages=1 << 15), dict(num_heads=0), dict(num_heads=129)])
def test_the_workspace_of_invalid_sizes_is_zero(kw):
    sizes = dict(dict(n_rows=4, num_heads=16, n_seqs=2, page_size=16, max_pages=4), **kw)
    assert smla.smla_paged_attend_workspace_size(**sizes) == 0


def test_packed_structs_have_the_c_layout():
    # every field with a value of its own, through the formats that the calls use
    values = list(range(101, 113))
    assert bytes(smla.PagedBatch(*values)) == smla._pack_batch(*values)
    rest = [201, 1, 203, 204, 205, 0.25, 207, 208, 209, 210, 211]
    assert bytes(smla.PagedAttendParams(smla.PagedBatch(*values), *rest)) == smla._pack_attend(*values, *rest)

"""Python binding of libsmla.so: sparse MLA decode over fp8_ds_mla records.

Argument marshalling only.  Every step of the computation runs in the CUDA
kernels of libsmla.so; there is no CPU or PyTorch fallback, and importing
fails loudly when the library has not been built (``python -c "import
__graft_entry__ as g; g.build()"``).  PyTorch supplies device memory and
streams.  The entry points keep the names of the C ABI in include/smla.h.
"""

from __future__ import annotations

import ctypes
import os
import struct
from typing import Optional

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libsmla.so")

RECORD_BYTES = 656
LATENT_DIM = 512
ROPE_DIM = 64
QK_DIM = 576
MAX_HEADS = 64
MAX_SPLITS = 64
STATUS_INDEX_OOB = 0x1
STATUS_TIMEOUT = 0x2
STATUS_SMEM_LAYOUT = 0x4
STATUS_FOREIGN_SCALE = 0x8
KERNEL_TENSOR_CORE = 0       # default: native fp8 where supported, else bf16 tensor cores
KERNEL_CUDA_CORE = 1
KERNEL_TENSOR_CORE_BF16 = 2
KERNEL_TENSOR_CORE_FP8 = 3
NOALLOC_SCRATCH_BYTES = 64 << 20  # SMLA_NOALLOC_SCRATCH_BYTES
PAGED_MAX_HEADS = 128
MAX_ROWS = 1 << 30  # token rows of a call
DTYPES = {torch.bfloat16: 0, torch.float16: 1, torch.float32: 2}  # SMLA_DTYPE_*
SMLA_ERR_NULL = -1
SMLA_ERR_SHAPE = -2
SMLA_ERR_STRIDE = -3
SMLA_ERR_WORKSPACE = -5
SMLA_ERR_DEVICE = -7


class SmlaError(RuntimeError):
    def __init__(self, code: int, what: str):
        super().__init__(f"{what}: {strerror(code)} (status {code})")
        self.code = code


class DecodeParams(ctypes.Structure):
    _fields_ = [
        ("n_q", ctypes.c_int32),
        ("num_heads", ctypes.c_int32),
        ("q", ctypes.c_void_p),
        ("q_stride_row", ctypes.c_int64),
        ("q_stride_head", ctypes.c_int64),
        ("kv_cache", ctypes.c_void_p),
        ("n_kv_rows", ctypes.c_int64),
        ("indices", ctypes.c_void_p),
        ("n_indices", ctypes.c_int64),
        ("indptr", ctypes.c_void_p),
        ("lens", ctypes.c_void_p),
        ("max_row_len", ctypes.c_int32),
        ("has_invalid", ctypes.c_int32),
        ("sm_scale", ctypes.c_float),
        ("sink", ctypes.c_void_p),
        ("out", ctypes.c_void_p),
        ("out_stride_row", ctypes.c_int64),
        ("out_stride_head", ctypes.c_int64),
        ("lse", ctypes.c_void_p),
        ("n_valid", ctypes.c_void_p),
        ("status", ctypes.c_void_p),
        ("num_splits", ctypes.c_int32),
        ("kernel", ctypes.c_int32),
    ]


class PlanInfo(ctypes.Structure):
    _fields_ = [
        ("kernel", ctypes.c_int32),
        ("grid", ctypes.c_int32),
        ("tile_len", ctypes.c_int32),
        ("num_splits", ctypes.c_int32),
        ("chunk_len", ctypes.c_int32),
        ("partial_slots", ctypes.c_int32),
        ("merge_kernel", ctypes.c_int32),
        ("trim_kernel", ctypes.c_int32),
        ("head_groups", ctypes.c_int32),
        ("workspace_bytes", ctypes.c_int64),
    ]


class PagedBatch(ctypes.Structure):
    _fields_ = [
        ("kv_cache", ctypes.c_void_p),
        ("n_pages", ctypes.c_int64),
        ("page_stride", ctypes.c_int64),
        ("page_size", ctypes.c_int32),
        ("max_pages", ctypes.c_int32),
        ("block_table", ctypes.c_void_p),
        ("block_table_stride", ctypes.c_int64),
        ("cu_rows", ctypes.c_void_p),
        ("seq_lens", ctypes.c_void_p),
        ("n_rows", ctypes.c_int64),
        ("n_seqs", ctypes.c_int32),
        ("status", ctypes.c_void_p),
    ]


class PagedAttendParams(ctypes.Structure):
    _fields_ = [
        ("batch", PagedBatch),
        ("num_heads", ctypes.c_int32),
        ("causal", ctypes.c_int32),
        ("q", ctypes.c_void_p),
        ("q_stride_row", ctypes.c_int64),
        ("q_stride_head", ctypes.c_int64),
        ("sm_scale", ctypes.c_float),
        ("sink", ctypes.c_void_p),
        ("out", ctypes.c_void_p),
        ("out_stride_row", ctypes.c_int64),
        ("out_stride_head", ctypes.c_int64),
        ("lse", ctypes.c_void_p),
    ]


class PagedAppendParams(ctypes.Structure):
    _fields_ = [
        ("batch", PagedBatch),
        ("latent", ctypes.c_void_p),
        ("latent_stride", ctypes.c_int64),
        ("rope", ctypes.c_void_p),
        ("rope_stride", ctypes.c_int64),
        ("dtype", ctypes.c_int32),
        ("interleaved", ctypes.c_int32),
        ("turns", ctypes.c_void_p),
        ("rope_scale", ctypes.c_float),
        ("num_heads", ctypes.c_int32),
        ("positions", ctypes.c_void_p),
        ("q_rope", ctypes.c_void_p),
        ("q_rope_stride_row", ctypes.c_int64),
        ("q_rope_stride_head", ctypes.c_int64),
        ("q_out", ctypes.c_void_p),
        ("q_out_stride_row", ctypes.c_int64),
        ("q_out_stride_head", ctypes.c_int64),
    ]


def _load():
    if not os.path.exists(LIB_PATH):
        raise ImportError(
            f"{LIB_PATH} is not built: run `python -c \"import __graft_entry__ as g; g.build()\"`")
    lib = ctypes.CDLL(LIB_PATH)
    lib.smla_plan.argtypes = [ctypes.POINTER(DecodeParams), ctypes.c_int32, ctypes.POINTER(PlanInfo)]
    lib.smla_plan.restype = ctypes.c_int
    lib.smla_decode_workspace_size.argtypes = [ctypes.POINTER(DecodeParams)]
    lib.smla_decode_workspace_size.restype = ctypes.c_size_t
    lib.smla_decode.argtypes = [ctypes.POINTER(DecodeParams), ctypes.c_void_p, ctypes.c_size_t,
                                ctypes.c_void_p]
    lib.smla_decode.restype = ctypes.c_int
    lib.smla_decode_noalloc.argtypes = [ctypes.POINTER(DecodeParams), ctypes.c_void_p]
    lib.smla_decode_noalloc.restype = ctypes.c_int
    lib.smla_pack_records.argtypes = [ctypes.c_void_p, ctypes.c_int64, ctypes.c_void_p,
                                      ctypes.c_int64, ctypes.c_int64, ctypes.c_void_p,
                                      ctypes.c_void_p]
    lib.smla_pack_records.restype = ctypes.c_int
    for name in ("smla_paged_write", "smla_paged_read"):
        f = getattr(lib, name)
        f.argtypes = [ctypes.POINTER(PagedBatch), ctypes.c_void_p, ctypes.c_int64, ctypes.c_void_p,
                      ctypes.c_int64, ctypes.c_int32, ctypes.c_void_p]
        f.restype = ctypes.c_int
    lib.smla_paged_attend_workspace_size.argtypes = [ctypes.POINTER(PagedAttendParams)]
    lib.smla_paged_attend_workspace_size.restype = ctypes.c_size_t
    lib.smla_paged_attend.argtypes = [ctypes.POINTER(PagedAttendParams), ctypes.c_void_p, ctypes.c_size_t,
                                      ctypes.c_void_p]
    lib.smla_paged_attend.restype = ctypes.c_int
    lib.smla_rotation_turns.argtypes = [ctypes.c_void_p, ctypes.c_void_p]
    lib.smla_rotation_turns.restype = ctypes.c_int
    lib.smla_paged_append.argtypes = [ctypes.POINTER(PagedAppendParams), ctypes.c_void_p]
    lib.smla_paged_append.restype = ctypes.c_int
    lib.smla_paged_tree.argtypes = [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int64,
                                    ctypes.c_int32, ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32,
                                    ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p]
    lib.smla_paged_tree.restype = ctypes.c_int
    lib.smla_paged_attend_tree.argtypes = [ctypes.POINTER(PagedAttendParams), ctypes.c_void_p, ctypes.c_int64,
                                           ctypes.c_int32, ctypes.c_void_p, ctypes.c_size_t, ctypes.c_void_p]
    lib.smla_paged_attend_tree.restype = ctypes.c_int
    lib.smla_paged_accept.argtypes = [ctypes.POINTER(PagedBatch), ctypes.c_void_p, ctypes.c_int64,
                                      ctypes.c_int32, ctypes.c_void_p, ctypes.c_void_p]
    lib.smla_paged_accept.restype = ctypes.c_int
    lib.smla_strerror.argtypes = [ctypes.c_int]
    lib.smla_strerror.restype = ctypes.c_char_p
    lib.smla_device_check.argtypes = []
    lib.smla_device_check.restype = ctypes.c_int
    lib.smla_set_wait_limit.argtypes = [ctypes.c_uint64, ctypes.c_int]
    lib.smla_set_wait_limit.restype = ctypes.c_int
    return lib


lib = _load()

try:
    from . import _smla as _native  # noqa: E402  (built beside libsmla.so, which it calls)
except ImportError as e:
    raise ImportError("_smla.so is not built for this Python and PyTorch: run "
                      "`python -c \"import __graft_entry__ as g; g.build()\"`") from e

EXPORTED_SYMBOLS = ("smla_plan", "smla_decode_workspace_size", "smla_decode", "smla_decode_noalloc",
                    "smla_pack_records", "smla_paged_write", "smla_paged_read",
                    "smla_paged_attend_workspace_size", "smla_paged_attend",
                    "smla_rotation_turns", "smla_paged_append", "smla_paged_tree", "smla_paged_attend_tree",
                    "smla_paged_accept",
                    "smla_strerror", "smla_device_check", "smla_set_wait_limit")


def strerror(code: int) -> str:
    return lib.smla_strerror(int(code)).decode()


def _ptr(t: Optional[torch.Tensor]) -> Optional[int]:
    return None if t is None else t.data_ptr()


def _stream(stream) -> Optional[int]:
    if stream is None:
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, torch.cuda.Stream):
        return stream.cuda_stream
    return int(stream)


def _plan_params(n_q, num_heads, max_row_len=0, n_indices=0, num_splits=0,
                 kernel=KERNEL_TENSOR_CORE, has_invalid=False) -> DecodeParams:
    p = DecodeParams()
    p.n_q, p.num_heads, p.max_row_len, p.n_indices = int(n_q), int(num_heads), int(max_row_len), int(n_indices)
    p.num_splits, p.kernel, p.has_invalid = int(num_splits), int(kernel), int(bool(has_invalid))
    return p


def smla_plan(n_q: int, num_heads: int, max_row_len: int = 0, n_indices: int = 0,
              num_splits: int = 0, num_sms: int = 0, kernel: int = KERNEL_TENSOR_CORE,
              has_invalid: bool = False) -> PlanInfo:
    """The launch plan of a decode call (pure host arithmetic when num_sms > 0)."""
    info = PlanInfo()
    p = _plan_params(n_q, num_heads, max_row_len, n_indices, num_splits, kernel, has_invalid)
    rc = lib.smla_plan(ctypes.byref(p), int(num_sms), ctypes.byref(info))
    if rc != 0:
        raise SmlaError(rc, "smla_plan")
    return info


def smla_decode_workspace_size(n_q: int, num_heads: int, max_row_len: int = 0,
                               n_indices: int = 0, num_splits: int = 0,
                               kernel: int = KERNEL_TENSOR_CORE, has_invalid: bool = False) -> int:
    p = _plan_params(n_q, num_heads, max_row_len, n_indices, num_splits, kernel, has_invalid)
    return int(lib.smla_decode_workspace_size(ctypes.byref(p)))


_WS: dict = {}


def workspace(nbytes: int, device, layout=None) -> Optional[torch.Tensor]:
    """A cached workspace of at least nbytes on device, ready for a call with
    the given layout key (n_q, heads, plan).

    smla_decode needs the per-row ticket counters at the start of the
    workspace to be zero, and leaves them zero; a call with another layout may
    have written partials over that region, so the counters are re-zeroed
    (on the current stream) whenever the layout changes.
    """
    if nbytes == 0:
        return None
    dev = torch.device(device)
    key = (dev.type, dev.index)
    ws, last = _WS.get(key, (None, None))
    if ws is None or ws.numel() < nbytes:
        ws = torch.zeros(max(nbytes, 1 << 20), dtype=torch.uint8, device=dev)
    elif layout != last:
        n_q = layout[0] if layout else ws.numel() // 4
        ws[: min(ws.numel(), 8 * n_q + 256)].zero_()
    _WS[key] = (ws, layout)
    return ws


def smla_decode(q: torch.Tensor, kv_cache: torch.Tensor, n_kv_rows: int, indices: torch.Tensor,
                indptr: torch.Tensor, lens: Optional[torch.Tensor], sm_scale: float,
                sink: Optional[torch.Tensor], out: torch.Tensor, lse: Optional[torch.Tensor],
                stream=None, *, max_row_len: int = 0, has_invalid: bool = False,
                n_valid: Optional[torch.Tensor] = None, status: Optional[torch.Tensor] = None,
                num_splits: int = 0, workspace_tensor: Optional[torch.Tensor] = None,
                kernel: int = KERNEL_TENSOR_CORE) -> None:
    """Sparse MLA decode into ``out`` (bf16 [n_q, H, 512]) and ``lse`` (f32 [n_q, H]).

    q: bf16 [n_q, H, 576]; kv_cache: uint8 [n_kv_rows, 656]; indices/indptr/lens:
    int32; sink: f32 [H] or None; n_valid: int32 [n_q] or None; status: int32 [1]
    or None.  All tensors on the current CUDA device.  See include/smla.h.
    """
    assert q.dtype == torch.bfloat16 and q.dim() == 3 and q.stride(2) == 1
    assert out.dtype == torch.bfloat16 and out.dim() == 3 and out.stride(2) == 1
    assert kv_cache.dtype == torch.uint8
    for t in (indices, indptr, lens, n_valid, status):
        assert t is None or t.dtype == torch.int32
    assert sink is None or sink.dtype == torch.float32
    assert lse is None or (lse.dtype == torch.float32 and lse.is_contiguous())
    n_q, heads = int(q.shape[0]), int(q.shape[1])
    p = DecodeParams()
    p.n_q, p.num_heads = n_q, heads
    p.q, p.q_stride_row, p.q_stride_head = q.data_ptr(), q.stride(0), q.stride(1)
    p.kv_cache, p.n_kv_rows = kv_cache.data_ptr(), int(n_kv_rows)
    p.indices, p.n_indices = _ptr(indices), int(indices.numel())
    p.indptr, p.lens = _ptr(indptr), _ptr(lens)
    p.max_row_len, p.has_invalid = int(max_row_len), int(bool(has_invalid))
    p.sm_scale = float(sm_scale)
    p.sink = _ptr(sink)
    p.out, p.out_stride_row, p.out_stride_head = out.data_ptr(), out.stride(0), out.stride(1)
    p.lse, p.n_valid, p.status = _ptr(lse), _ptr(n_valid), _ptr(status)
    p.num_splits = int(num_splits)
    p.kernel = int(kernel)
    ws = workspace_tensor
    if ws is None:
        plan = PlanInfo()
        rc = lib.smla_plan(ctypes.byref(p), 0, ctypes.byref(plan))
        if rc != 0:
            raise SmlaError(rc, "smla_plan")
        ws = workspace(int(plan.workspace_bytes), q.device,
                       (n_q, heads, plan.kernel, plan.grid, plan.num_splits, plan.chunk_len, plan.trim_kernel))
    rc = lib.smla_decode(ctypes.byref(p), _ptr(ws), 0 if ws is None else ws.numel(), _stream(stream))
    if rc != 0:
        raise SmlaError(rc, "smla_decode")


def smla_decode_noalloc(q: torch.Tensor, kv_cache: torch.Tensor, n_kv_rows: int,
                        indices: torch.Tensor, indptr: torch.Tensor, lens: Optional[torch.Tensor],
                        sm_scale: float, sink: Optional[torch.Tensor], out: torch.Tensor,
                        lse: Optional[torch.Tensor], stream=None, *, max_row_len: int = 0,
                        has_invalid: bool = False, n_valid: Optional[torch.Tensor] = None,
                        status: Optional[torch.Tensor] = None, num_splits: int = 0,
                        kernel: int = KERNEL_TENSOR_CORE) -> None:
    """smla_decode with the library's fixed device scratch as workspace (no
    allocation on the call path; for callers that cannot allocate device
    memory at call time).  Arguments as smla_decode.  Calls on one device
    share that scratch: calls that may overlap on the GPU must be ordered.
    The first call on a device sets up the scratch address; make it before
    any stream capture.  See include/smla.h."""
    assert q.dtype == torch.bfloat16 and q.dim() == 3 and q.stride(2) == 1
    assert out.dtype == torch.bfloat16 and out.dim() == 3 and out.stride(2) == 1
    assert kv_cache.dtype == torch.uint8
    for t in (indices, indptr, lens, n_valid, status):
        assert t is None or t.dtype == torch.int32
    assert sink is None or sink.dtype == torch.float32
    assert lse is None or (lse.dtype == torch.float32 and lse.is_contiguous())
    p = DecodeParams()
    p.n_q, p.num_heads = int(q.shape[0]), int(q.shape[1])
    p.q, p.q_stride_row, p.q_stride_head = q.data_ptr(), q.stride(0), q.stride(1)
    p.kv_cache, p.n_kv_rows = kv_cache.data_ptr(), int(n_kv_rows)
    p.indices, p.n_indices = _ptr(indices), int(indices.numel())
    p.indptr, p.lens = _ptr(indptr), _ptr(lens)
    p.max_row_len, p.has_invalid = int(max_row_len), int(bool(has_invalid))
    p.sm_scale = float(sm_scale)
    p.sink = _ptr(sink)
    p.out, p.out_stride_row, p.out_stride_head = out.data_ptr(), out.stride(0), out.stride(1)
    p.lse, p.n_valid, p.status = _ptr(lse), _ptr(n_valid), _ptr(status)
    p.num_splits, p.kernel = int(num_splits), int(kernel)
    rc = lib.smla_decode_noalloc(ctypes.byref(p), _stream(stream))
    if rc == SMLA_ERR_WORKSPACE:
        raise SmlaError(rc, f"smla_decode_noalloc: the call needs more than the "
                            f"{NOALLOC_SCRATCH_BYTES}-byte fixed scratch")
    if rc != 0:
        raise SmlaError(rc, "smla_decode_noalloc")


def smla_pack_records(latent: torch.Tensor, rope: torch.Tensor, kv_out: torch.Tensor,
                      stream=None) -> None:
    """Record writer: bf16 latent [n, 512] + bf16 rope [n, 64] -> uint8 kv_out [n, 656]."""
    assert latent.dtype == torch.bfloat16 and rope.dtype == torch.bfloat16
    assert kv_out.dtype == torch.uint8 and kv_out.is_contiguous()
    assert latent.stride(1) == 1 and rope.stride(1) == 1
    n = int(latent.shape[0])
    assert rope.shape[0] == n and kv_out.numel() >= n * RECORD_BYTES
    rc = lib.smla_pack_records(latent.data_ptr(), latent.stride(0), rope.data_ptr(), rope.stride(0),
                               n, kv_out.data_ptr(), _stream(stream))
    if rc != 0:
        raise SmlaError(rc, "smla_pack_records")


# ---- the paged cache ----
#
# These calls can take less time on the GPU than their checks do here.  Well-formed calls
# on the current stream are therefore made by _smla.so (csrc/smla_binding.cpp), which
# answers False to all others and does nothing for them: they go through the checks
# here, which name what is wrong.  A launch that failed there is raised.  The checks read each tensor's properties once, the
# messages are made on failure, and the C structs are packed as bytes.

_BATCH_FORMAT = "PqqiiPqPPqi4xP"
_pack_batch = struct.Struct(_BATCH_FORMAT).pack
_pack_attend = struct.Struct(_BATCH_FORMAT + "iiPqqf4xPPqqP").pack
_pack_append = struct.Struct(_BATCH_FORMAT + "PqPqiiPfiPPqqPqq").pack


def _packed(name: str, restype, *argtypes):
    f = lib[name]  # a function object of its own, beside the typed one
    f.restype, f.argtypes = restype, (ctypes.c_void_p, *argtypes)
    return f


_copy_args = (ctypes.c_void_p, ctypes.c_int64, ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_void_p)
_write_packed = _packed("smla_paged_write", ctypes.c_int, *_copy_args)
_read_packed = _packed("smla_paged_read", ctypes.c_int, *_copy_args)
_workspace_packed = _packed("smla_paged_attend_workspace_size", ctypes.c_size_t)
_attend_packed = _packed("smla_paged_attend", ctypes.c_int, ctypes.c_void_p, ctypes.c_size_t, ctypes.c_void_p)
_attend_tree_packed = _packed("smla_paged_attend_tree", ctypes.c_int, ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32,
                              ctypes.c_void_p, ctypes.c_size_t, ctypes.c_void_p)
_append_packed = _packed("smla_paged_append", ctypes.c_int, ctypes.c_void_p)
_accept_packed = _packed("smla_paged_accept", ctypes.c_int, ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32,
                         ctypes.c_void_p, ctypes.c_void_p)


def _fail(code: int, what: str, why: str):
    raise SmlaError(code, f"{what}: {why}")


def _made(what: str, answer) -> bool:
    """Whether _smla.so has made the call; raises when it has and a launch failed."""
    if answer is True or answer is False:
        return answer
    raise SmlaError(answer, what)


def _launch_stream(stream, device: int) -> int:
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(device)
    return stream.cuda_stream if isinstance(stream, torch.cuda.Stream) else int(stream)


def _current_device(what: str, tensors) -> int:
    """The current CUDA device, on which every tensor has to be (the launch goes there)."""
    first = tensors[0].get_device()
    for t in tensors:
        if t is not None and (not t.is_cuda or t.get_device() != first):
            _fail(SMLA_ERR_DEVICE, what, "the tensors are not on one CUDA device")
    if first != torch.cuda.current_device():
        _fail(SMLA_ERR_DEVICE, what, "a tensor is not on the current CUDA device")
    return first


def _paged_batch(what: str, kv_cache: torch.Tensor, block_table: torch.Tensor, cu_rows: torch.Tensor,
                 seq_lens: torch.Tensor, n_rows: int, status: Optional[torch.Tensor]) -> tuple:
    """The C batch of a paged cache uint8 [n_pages, page_size, 656] (pages may be
    strided) and its int32 tables, checked: the fields of PagedBatch."""
    if kv_cache.dtype != torch.uint8 or kv_cache.dim() != 3 or kv_cache.shape[2] != RECORD_BYTES:
        _fail(SMLA_ERR_SHAPE, what, f"kv_cache is uint8 [n_pages, page_size, {RECORD_BYTES}]")
    n_pages, page_size, _ = kv_cache.shape
    if page_size >> 30:
        _fail(SMLA_ERR_SHAPE, what, "a page has at most 2^30 records")
    page_stride, record_stride, byte_stride = kv_cache.stride()
    # (a dimension of one element, or an empty cache, may carry any stride)
    if n_pages and page_size and (byte_stride != 1 or (page_size > 1 and record_stride != RECORD_BYTES)):
        _fail(SMLA_ERR_STRIDE, what, "the records of a page are contiguous")
    i32 = torch.int32
    if (block_table.dtype != i32 or cu_rows.dtype != i32 or seq_lens.dtype != i32 or block_table.dim() != 2 or
            cu_rows.dim() != 1 or seq_lens.dim() != 1):
        _fail(SMLA_ERR_SHAPE, what, "block_table is int32 [n_seqs, max_pages], cu_rows and seq_lens int32 vectors")
    n_seqs, max_pages = block_table.shape
    table_stride, entry_stride = block_table.stride()
    if seq_lens.shape[0] != n_seqs or cu_rows.shape[0] != n_seqs + 1:
        _fail(SMLA_ERR_SHAPE, what, "n_seqs + 1 entries of cu_rows and n_seqs of seq_lens for n_seqs rows of block_table")
    if n_seqs and ((max_pages > 1 and entry_stride != 1) or cu_rows.stride(0) != 1 or
                   (n_seqs > 1 and seq_lens.stride(0) != 1)):
        _fail(SMLA_ERR_STRIDE, what, "block_table rows, cu_rows and seq_lens are contiguous")
    if status is not None and (status.dtype != i32 or status.numel() < 1):
        _fail(SMLA_ERR_SHAPE, what, "status is int32 [1]")
    return (kv_cache.data_ptr(), n_pages, page_stride if n_pages > 1 else page_size * RECORD_BYTES, page_size, max_pages,
            block_table.data_ptr(), table_stride if n_seqs > 1 else max_pages, cu_rows.data_ptr(), seq_lens.data_ptr(),
            n_rows, n_seqs, 0 if status is None else status.data_ptr())


def _rows(what, latent, rope) -> tuple:
    """Rows, dtype and strides of latent [rows, 512] and rope [rows, 64], checked."""
    dtype = DTYPES.get(latent.dtype)
    if dtype is None or rope.dtype != latent.dtype:
        _fail(SMLA_ERR_SHAPE, what, "latent and rope of one type, bf16, f16 or f32")
    if latent.dim() != 2 or rope.dim() != 2:
        _fail(SMLA_ERR_SHAPE, what, f"latent [rows, {LATENT_DIM}] and rope [rows, {ROPE_DIM}]")
    n, dims = latent.shape
    if dims != LATENT_DIM or rope.shape[0] != n or rope.shape[1] != ROPE_DIM:
        _fail(SMLA_ERR_SHAPE, what, f"latent [rows, {LATENT_DIM}] and rope [rows, {ROPE_DIM}]")
    ls, l1 = latent.stride()
    rs, r1 = rope.stride()
    if n and (l1 != 1 or r1 != 1):
        _fail(SMLA_ERR_STRIDE, what, "the rows of latent and rope are contiguous")
    if n <= 1:  # (the stride of a single row says nothing)
        ls, rs = LATENT_DIM, ROPE_DIM
    return n, dtype, ls, rs


def _paged_copy(what, call, kv_cache, block_table, cu_rows, seq_lens, latent, rope, stream, status) -> None:
    n, dtype, ls, rs = _rows(what, latent, rope)
    batch = _paged_batch(what, kv_cache, block_table, cu_rows, seq_lens, n, status)
    device = _current_device(what, (latent, rope, kv_cache, block_table, cu_rows, seq_lens, status))
    rc = call(_pack_batch(*batch), latent.data_ptr(), ls, rope.data_ptr(), rs, dtype, _launch_stream(stream, device))
    if rc != 0:
        raise SmlaError(rc, what)


def smla_paged_write(latent: torch.Tensor, rope: torch.Tensor, kv_cache: torch.Tensor, block_table: torch.Tensor,
                     cu_rows: torch.Tensor, seq_lens: torch.Tensor, stream=None, *,
                     status: Optional[torch.Tensor] = None) -> None:
    """Writes the records of new token rows into a paged cache.

    latent [rows, 512], rope [rows, 64]: bf16, f16 or f32.  kv_cache: uint8
    [n_pages, page_size, 656].  Sequence b owns rows cu_rows[b]:cu_rows[b + 1],
    which are its positions up to seq_lens[b] - 1 (seq_lens counts them);
    position p lives in page block_table[b, p // page_size].  Rows whose page id
    is negative are skipped; ids >= n_pages and positions past the table are
    skipped and set STATUS_INDEX_OOB.  The rows' positions must lie in different
    slots.  An infinite latent takes its whole block of 128 values to the scale
    2^120, where ordinary values become zero.  See include/smla.h."""
    if _made("smla_paged_write", _native.write(kv_cache, block_table, cu_rows, seq_lens, latent, rope, stream, status)):
        return
    _paged_copy("smla_paged_write", _write_packed, kv_cache, block_table, cu_rows, seq_lens, latent, rope,
                stream, status)


def smla_paged_read(kv_cache: torch.Tensor, block_table: torch.Tensor, cu_rows: torch.Tensor, seq_lens: torch.Tensor,
                    latent: torch.Tensor, rope: torch.Tensor, stream=None, *,
                    status: Optional[torch.Tensor] = None) -> None:
    """Reads records of a paged cache back into latent [rows, 512] and rope
    [rows, 64] (bf16, f16 or f32).  Batch as smla_paged_write: row r of sequence
    b gets position seq_lens[b] - (cu_rows[b + 1] - r); masked positions give
    zeros, rows of no sequence are left as they were.  See include/smla.h."""
    if _made("smla_paged_read", _native.read(kv_cache, block_table, cu_rows, seq_lens, latent, rope, stream, status)):
        return
    _paged_copy("smla_paged_read", _read_packed, kv_cache, block_table, cu_rows, seq_lens, latent, rope,
                stream, status)


def smla_paged_attend_workspace_size(n_rows: int, num_heads: int, n_seqs: int, page_size: int, max_pages: int) -> int:
    """Workspace bytes of smla_paged_attend for these sizes on the current device.
    They never grow when n_rows, n_seqs, page_size or max_pages shrinks."""
    p = PagedAttendParams()
    p.num_heads = int(num_heads)
    p.batch.n_rows, p.batch.n_seqs = int(n_rows), int(n_seqs)
    p.batch.page_size, p.batch.max_pages = int(page_size), int(max_pages)
    return int(lib.smla_paged_attend_workspace_size(ctypes.byref(p)))


def _attend(what: str, q, kv_cache, block_table, cu_rows, seq_lens, mask, sm_scale, sink, out, lse, stream, causal,
            status, workspace_tensor) -> None:
    if _made(what, _native.attend(kv_cache, block_table, cu_rows, seq_lens, q, sm_scale, sink, out, lse, causal, stream, status,
                                  workspace_tensor, mask)):
        return
    if q.dtype != torch.bfloat16 or q.dim() != 3 or q.shape[2] != QK_DIM:
        _fail(SMLA_ERR_SHAPE, what, f"q is bf16 [rows, heads, {QK_DIM}]")
    n, heads, _ = q.shape
    if out.dtype != torch.bfloat16 or out.shape != (n, heads, LATENT_DIM):
        _fail(SMLA_ERR_SHAPE, what, f"out is bf16 [rows, heads, {LATENT_DIM}]")
    q_row, q_head, q1 = q.stride()
    o_row, o_head, o1 = out.stride()
    if n and (q1 != 1 or o1 != 1):
        _fail(SMLA_ERR_STRIDE, what, "the last dimension of q and out is contiguous")
    # (the stride of a dimension of one element says nothing)
    if heads == 1:
        q_head, o_head = QK_DIM, LATENT_DIM
    if n <= 1:
        q_row, o_row = heads * q_head, heads * o_head
    if sink is not None and (sink.dtype != torch.float32 or sink.shape != (heads,) or not sink.is_contiguous()):
        _fail(SMLA_ERR_SHAPE, what, "sink is f32 [heads]")
    if lse is not None and (lse.dtype != torch.float32 or lse.shape != (n, heads) or not lse.is_contiguous()):
        _fail(SMLA_ERR_SHAPE, what, "lse is contiguous f32 [rows, heads]")
    if workspace_tensor is not None and not workspace_tensor.is_contiguous():
        _fail(SMLA_ERR_STRIDE, what, "workspace_tensor is contiguous")
    if mask is not None:
        mask_row, words = _mask_layout(what, mask, n)
    batch = _paged_batch(what, kv_cache, block_table, cu_rows, seq_lens, n, status)
    device = _current_device(what, (q, out, sink, lse, kv_cache, block_table, cu_rows, seq_lens, status,
                                    workspace_tensor, mask))
    try:
        p = _pack_attend(*batch, heads, 1 if causal else 0, q.data_ptr(), q_row, q_head, sm_scale,
                         0 if sink is None else sink.data_ptr(), out.data_ptr(), o_row, o_head,
                         0 if lse is None else lse.data_ptr())
    except OverflowError:
        _fail(SMLA_ERR_SHAPE, what, "sm_scale is no finite f32")
    s = _launch_stream(stream, device)
    ws = workspace_tensor
    if ws is None:
        nbytes = _workspace_packed(p)
        if nbytes:
            # a block of this call's own, on its stream: calls on other streams and
            # other captured graphs never share it
            if stream is None:
                ws = kv_cache.new_empty(nbytes)
            else:
                if not isinstance(stream, torch.cuda.Stream):
                    stream = torch.cuda.ExternalStream(s) if s else torch.cuda.default_stream()
                with torch.cuda.stream(stream):
                    ws = kv_cache.new_empty(nbytes)
    ws_at, ws_bytes = (None, 0) if ws is None else (ws.data_ptr(), ws.nbytes)
    if mask is None:
        rc = _attend_packed(p, ws_at, ws_bytes, s)
    else:
        rc = _attend_tree_packed(p, mask.data_ptr(), mask_row, words, ws_at, ws_bytes, s)
    if rc != 0:
        raise SmlaError(rc, what)


def smla_paged_attend(q: torch.Tensor, kv_cache: torch.Tensor, block_table: torch.Tensor, cu_rows: torch.Tensor,
                      seq_lens: torch.Tensor, sm_scale: float, sink: Optional[torch.Tensor], out: torch.Tensor,
                      lse: Optional[torch.Tensor], stream=None, *, causal: bool = True,
                      status: Optional[torch.Tensor] = None, workspace_tensor: Optional[torch.Tensor] = None) -> None:
    """Attention of new token rows over a paged cache, into ``out`` (bf16
    [rows, H, 512]) and ``lse`` (f32 [rows, H] or None).

    q: bf16 [rows, H, 576], H up to 128; batch as smla_paged_write (the rows'
    own records are read from the cache: write them first).  A row at position
    p sees positions 0..p (causal) or its whole sequence; sink: f32 [H] or None.
    workspace_tensor: uint8, smla_paged_attend_workspace_size bytes; without it
    one is allocated for this call on its stream.  See include/smla.h."""
    _attend("smla_paged_attend", q, kv_cache, block_table, cu_rows, seq_lens, None, sm_scale, sink, out, lse, stream,
            causal, status, workspace_tensor)


# ---- rotation and trees of drafted tokens ----


def smla_rotation_turns(inv_freq, device=None) -> torch.Tensor:
    """The rotation table of smla_paged_append: int64 [32] on `device` (the current CUDA
    device by default) from the 32 angles per position, in radians (a tensor or a
    sequence).  Made on the host; keep it for all calls."""
    f = torch.as_tensor(inv_freq, dtype=torch.float64).cpu().contiguous()
    if f.shape != (ROPE_DIM // 2,):
        _fail(SMLA_ERR_SHAPE, "smla_rotation_turns", f"{ROPE_DIM // 2} angles per position")
    turns = torch.empty(ROPE_DIM // 2, dtype=torch.int64)
    rc = lib.smla_rotation_turns(f.data_ptr(), turns.data_ptr())
    if rc != 0:
        raise SmlaError(rc, "smla_rotation_turns")
    return turns.to("cuda" if device is None else device)


def _queries(what: str, x: torch.Tensor, name: str, n: int) -> tuple:
    """Heads and strides of a rope part [rows, heads, 64], checked."""
    if x.dim() != 3 or x.shape[0] != n or x.shape[2] != ROPE_DIM:
        _fail(SMLA_ERR_SHAPE, what, f"{name} is [rows, heads, {ROPE_DIM}]")
    heads = x.shape[1]
    row, head, one = x.stride()
    if n and heads and one != 1:
        _fail(SMLA_ERR_STRIDE, what, f"the last dimension of {name} is contiguous")
    # (the stride of a dimension of one element says nothing)
    if heads <= 1:
        head = ROPE_DIM
    return heads, row if n > 1 else heads * head, head


def smla_paged_append(latent: torch.Tensor, rope: torch.Tensor, kv_cache: torch.Tensor, block_table: torch.Tensor,
                      cu_rows: torch.Tensor, seq_lens: torch.Tensor, turns: torch.Tensor, stream=None, *,
                      q_rope: Optional[torch.Tensor] = None, q_out: Optional[torch.Tensor] = None,
                      positions: Optional[torch.Tensor] = None, interleaved: bool = True, rope_scale: float = 1.0,
                      status: Optional[torch.Tensor] = None) -> None:
    """smla_paged_write with the rope of keys and queries rotated on the way.

    latent [rows, 512], rope [rows, 64] and q_rope [rows, H, 64]: bf16, f16 or
    f32, before the rotation.  The records get the rotated rope, q_out (bf16
    [rows, H, 64], e.g. q[..., 512:]) the rotated queries; it may be q_rope
    itself.  turns: smla_rotation_turns.  A row turns by its position in the
    cache, or by positions (int32 [rows], e.g. of smla_paged_tree); pairs are
    dims (2k, 2k + 1), or (k, k + 32) without interleaved; rope_scale
    multiplies the results.  Batch and masked rows as smla_paged_write.  See
    include/smla.h."""
    what = "smla_paged_append"
    if _made(what, _native.append(kv_cache, block_table, cu_rows, seq_lens, latent, rope, turns, q_rope, q_out, positions,
                                  interleaved, rope_scale, stream, status)):
        return
    n, dtype, ls, rs = _rows(what, latent, rope)
    if turns.dtype != torch.int64 or turns.shape != (ROPE_DIM // 2,) or not turns.is_contiguous():
        _fail(SMLA_ERR_SHAPE, what, f"turns is int64 [{ROPE_DIM // 2}], made by smla_rotation_turns")
    if positions is not None and (positions.dtype != torch.int32 or positions.shape != (n,)):
        _fail(SMLA_ERR_SHAPE, what, "positions is int32 [rows]")
    if positions is not None and n > 1 and positions.stride(0) != 1:
        _fail(SMLA_ERR_STRIDE, what, "positions is contiguous")
    if (q_rope is None) != (q_out is None):
        _fail(SMLA_ERR_NULL, what, "q_rope and q_out belong together")
    heads = q_row = q_head = o_row = o_head = 0
    if q_rope is not None:
        if q_rope.dtype != latent.dtype or q_out.dtype != torch.bfloat16:
            _fail(SMLA_ERR_SHAPE, what, "q_rope has the type of latent, q_out is bf16")
        heads, q_row, q_head = _queries(what, q_rope, "q_rope", n)
        out_heads, o_row, o_head = _queries(what, q_out, "q_out", n)
        if heads != out_heads:
            _fail(SMLA_ERR_SHAPE, what, "q_rope and q_out have the same heads")
    batch = _paged_batch(what, kv_cache, block_table, cu_rows, seq_lens, n, status)
    device = _current_device(what, (latent, rope, kv_cache, block_table, cu_rows, seq_lens, turns, q_rope, q_out,
                                    positions, status))
    p = _pack_append(*batch, latent.data_ptr(), ls, rope.data_ptr(), rs, dtype, 1 if interleaved else 0,
                     turns.data_ptr(), rope_scale, heads, 0 if positions is None else positions.data_ptr(),
                     0 if q_rope is None else q_rope.data_ptr(), q_row, q_head,
                     0 if q_out is None else q_out.data_ptr(), o_row, o_head)
    rc = _append_packed(p, _launch_stream(stream, device))
    if rc != 0:
        raise SmlaError(rc, what)


def _mask_layout(what: str, mask: torch.Tensor, n: int) -> tuple:
    """Row stride and words of a mask int32 [rows, words], checked."""
    if mask.dtype != torch.int32 or mask.dim() != 2 or mask.shape[0] != n:
        _fail(SMLA_ERR_SHAPE, what, "mask is int32 [rows, words]")
    words = mask.shape[1]
    row, one = mask.stride()
    if n and words > 1 and one != 1:
        _fail(SMLA_ERR_STRIDE, what, "the rows of mask are contiguous")
    return row if n > 1 else words, words


def smla_paged_tree(parents: torch.Tensor, cu_rows: torch.Tensor, seq_lens: torch.Tensor,
                    mask: Optional[torch.Tensor], positions: Optional[torch.Tensor], stream=None, *,
                    status: Optional[torch.Tensor] = None) -> None:
    """Masks and positions of trees of drafted tokens, from their parents.

    The token rows of sequence b are the nodes of its tree, a parent before its
    children; parents (int32 [rows]): a row's parent node, negative for a root.
    mask (int32 [rows, words] or None): bit j % 32 of word j // 32 is set for
    the node itself and its ancestors; positions (int32 [rows] or None): the
    position of node 0 plus the node's depth.  A parent that is not a lower
    node, or a node that the words cannot hold, sets STATUS_INDEX_OOB.  See
    include/smla.h."""
    what = "smla_paged_tree"
    if _made(what, _native.tree(parents, cu_rows, seq_lens, mask, positions, stream, status)):
        return
    i32 = torch.int32
    if parents.dtype != i32 or cu_rows.dtype != i32 or seq_lens.dtype != i32 or parents.dim() != 1 or \
            cu_rows.dim() != 1 or seq_lens.dim() != 1:
        _fail(SMLA_ERR_SHAPE, what, "parents, cu_rows and seq_lens are int32 vectors")
    n, n_seqs = parents.shape[0], seq_lens.shape[0]
    if cu_rows.shape[0] != n_seqs + 1:
        _fail(SMLA_ERR_SHAPE, what, "n_seqs + 1 entries of cu_rows for n_seqs of seq_lens")
    if positions is not None and (positions.dtype != i32 or positions.shape != (n,)):
        _fail(SMLA_ERR_SHAPE, what, "positions is int32 [rows]")
    if n_seqs and (cu_rows.stride(0) != 1 or (n_seqs > 1 and seq_lens.stride(0) != 1)) or \
            n > 1 and (parents.stride(0) != 1 or (positions is not None and positions.stride(0) != 1)):
        _fail(SMLA_ERR_STRIDE, what, "parents, cu_rows, seq_lens and positions are contiguous")
    if status is not None and (status.dtype != i32 or status.numel() < 1):
        _fail(SMLA_ERR_SHAPE, what, "status is int32 [1]")
    mask_row, words = (0, 0) if mask is None else _mask_layout(what, mask, n)
    device = _current_device(what, (parents, cu_rows, seq_lens, mask, positions, status))
    rc = lib.smla_paged_tree(parents.data_ptr(), cu_rows.data_ptr(), seq_lens.data_ptr(), n, n_seqs, _ptr(mask),
                             mask_row, words, _ptr(positions), _ptr(status), _launch_stream(stream, device))
    if rc != 0:
        raise SmlaError(rc, what)


def smla_paged_attend_tree(q: torch.Tensor, kv_cache: torch.Tensor, block_table: torch.Tensor, cu_rows: torch.Tensor,
                           seq_lens: torch.Tensor, mask: torch.Tensor, sm_scale: float, sink: Optional[torch.Tensor],
                           out: torch.Tensor, lse: Optional[torch.Tensor], stream=None, *, causal: bool = False,
                           status: Optional[torch.Tensor] = None,
                           workspace_tensor: Optional[torch.Tensor] = None) -> None:
    """smla_paged_attend for trees of drafted tokens: of its sequence's token rows a
    row sees row j if bit j % 32 of word j // 32 of its mask (int32 [rows, words],
    e.g. of smla_paged_tree) is set, and of earlier positions all.  With causal
    a row in addition sees no position behind its own (the same for trees, and the
    keys of later nodes are passed over).  Everything else, the workspace's size
    included, as smla_paged_attend.  See include/smla.h."""
    what = "smla_paged_attend_tree"
    if mask is None:
        _fail(SMLA_ERR_NULL, what, "mask is int32 [rows, words]")
    _attend(what, q, kv_cache, block_table, cu_rows, seq_lens, mask, sm_scale, sink, out, lse,
            stream, causal, status, workspace_tensor)


def smla_paged_accept(kv_cache: torch.Tensor, block_table: torch.Tensor, cu_rows: torch.Tensor,
                      seq_lens: torch.Tensor, path: torch.Tensor, new_lens: torch.Tensor, stream=None, *,
                      n_rows: int = MAX_ROWS, status: Optional[torch.Tensor] = None) -> None:
    """Keeps the accepted path of each tree of drafted tokens.

    path: int32 [n_seqs, width], rising nodes of each tree, then negative
    entries.  The record of the i-th node of the path moves to the position of
    node 0 plus i, and new_lens[b] (int32 [n_seqs], which may be seq_lens) becomes
    the position of node 0 plus the number of nodes.  An entry that is no node or
    does not rise ends the path and sets STATUS_INDEX_OOB.  n_rows: rows of the
    token tensors, which clamp cu_rows in the other calls.  See include/smla.h."""
    what = "smla_paged_accept"
    if _made(what, _native.accept(kv_cache, block_table, cu_rows, seq_lens, path, new_lens, n_rows, stream, status)):
        return
    batch = _paged_batch(what, kv_cache, block_table, cu_rows, seq_lens, int(n_rows), status)
    n_seqs = seq_lens.shape[0]
    if path.dtype != torch.int32 or path.dim() != 2 or path.shape[0] != n_seqs:
        _fail(SMLA_ERR_SHAPE, what, "path is int32 [n_seqs, width]")
    if new_lens.dtype != torch.int32 or new_lens.shape != (n_seqs,):
        _fail(SMLA_ERR_SHAPE, what, "new_lens is int32 [n_seqs]")
    width = path.shape[1]
    if n_seqs and ((width > 1 and path.stride(1) != 1) or (n_seqs > 1 and new_lens.stride(0) != 1)):
        _fail(SMLA_ERR_STRIDE, what, "the rows of path and new_lens are contiguous")
    device = _current_device(what, (kv_cache, block_table, cu_rows, seq_lens, path, new_lens, status))
    rc = _accept_packed(_pack_batch(*batch), path.data_ptr(), path.stride(0) if n_seqs > 1 else width, width,
                        new_lens.data_ptr(), _launch_stream(stream, device))
    if rc != 0:
        raise SmlaError(rc, what)


def smla_device_check() -> int:
    return int(lib.smla_device_check())


def smla_set_wait_limit(limit_ns: int, stall_first_wait: bool = False) -> None:
    """Limit of every in-kernel pipeline wait (0: the 2 s default), and the
    timeout-path test switch; see smla.h."""
    rc = lib.smla_set_wait_limit(int(limit_ns), int(bool(stall_first_wait)))
    if rc != 0:
        raise SmlaError(rc, "smla_set_wait_limit")

"""The calls beside the rest of a process: other Python threads, errors of other libraries."""

import ctypes
import threading
import time

import pytest
import torch

import sparse_mla_decode_csr_gb300 as smla
from test_paged_gpu import DEV, Batch
from test_paged_tree_gpu import step, step_state

pytestmark = pytest.mark.gpu
CALLS = ("write", "read", "append", "tree", "attend", "attend_tree", "accept")


def calls(seed=5):
    """One call of each kind on a small batch, by name."""
    c = Batch([(3, 40), (2, 9)], 16)
    s = step_state(c, 16, seed)
    step(s)
    lat, rope, new = s["lat"].clone(), s["rope"].clone(), torch.zeros_like(s["new"])
    batch = (s["kv"], s["table"], s["cu"], s["sl"])
    out, lse = torch.empty_like(s["out"]), torch.empty_like(s["lse"])
    ws = torch.empty(smla.smla_paged_attend_workspace_size(c.rows, 16, 2, 16, s["table"].shape[1]), dtype=torch.uint8, device=DEV)
    return {
        "write": lambda: smla.smla_paged_write(s["lat"], s["rope"], *batch),
        "read": lambda: smla.smla_paged_read(*batch, lat, rope),
        "append": lambda: smla.smla_paged_append(s["lat"], s["rope"], *batch, s["turns"]),
        "tree": lambda: smla.smla_paged_tree(s["parents"], s["cu"], s["sl"], s["mask"], s["pos"]),
        "attend": lambda: smla.smla_paged_attend(s["q"], *batch, 1 / 24, None, out, lse, workspace_tensor=ws),
        "attend_tree": lambda: smla.smla_paged_attend_tree(s["q"], *batch, s["mask"], 1 / 24, None, out, lse, workspace_tensor=ws),
        "accept": lambda: smla.smla_paged_accept(*batch, s["path"], new),
    }


@pytest.fixture
def cudart():
    """The runtime that PyTorch and libsmla.so use; no error is left in it."""
    torch.cuda.synchronize()
    lib = ctypes.CDLL("libcudart.so.13")
    yield lib
    lib.cudaGetLastError()


@pytest.mark.parametrize("name", CALLS)
def test_a_launch_that_blocks_leaves_other_threads_running(name, cudart):
    # a stream that stands still for a second (a host function that sleeps) lets launches queue up
    # until the next one waits; the other Python threads go on meanwhile
    call, stream, longest = calls()[name], torch.cuda.Stream(), []
    call()
    torch.cuda.synchronize()
    sleep = ctypes.cast(ctypes.CDLL(None).usleep, ctypes.c_void_p)

    def work():
        with torch.cuda.stream(stream):
            assert cudart.cudaLaunchHostFunc(ctypes.c_void_p(stream.cuda_stream), sleep, ctypes.c_void_p(999_999)) == 0
            start = time.perf_counter()
            for _ in range(20_000):
                before = time.perf_counter()
                call()
                longest.append(time.perf_counter() - before)
                if before - start > 0.9:
                    break

    thread = threading.Thread(target=work)
    thread.start()
    gap, last = 0.0, time.perf_counter()
    while thread.is_alive():
        time.sleep(0.001)
        now = time.perf_counter()
        gap, last = max(gap, now - last), now
    thread.join()
    torch.cuda.synchronize()
    assert max(longest) > 0.3, "no launch waited"
    assert gap < max(longest) / 2


def decode_calls():
    """The decode by each kernel, its form without allocation, and the record writer."""
    n, h = 40, 16
    lat, rope = torch.randn(n, 512, device=DEV).bfloat16(), torch.randn(n, 64, device=DEV).bfloat16()
    kv = torch.zeros(n, 656, dtype=torch.uint8, device=DEV)
    smla.smla_pack_records(lat, rope, kv)
    q, out = torch.randn(2, h, 576, device=DEV).bfloat16(), torch.empty(2, h, 512, device=DEV).bfloat16()
    idx = torch.arange(n, dtype=torch.int32, device=DEV)
    ptr = torch.tensor([0, 20, 40], dtype=torch.int32, device=DEV)
    args = (q, kv, n, idx, ptr, None, 1 / 24, None, out, torch.empty(2, h, device=DEV))
    found = {"pack": lambda: smla.smla_pack_records(lat, rope, kv), "noalloc": lambda: smla.smla_decode_noalloc(*args)}
    for kernel in (smla.KERNEL_CUDA_CORE, smla.KERNEL_TENSOR_CORE_BF16, smla.KERNEL_TENSOR_CORE_FP8):
        for padded in (False, True):
            kw = dict(kernel=kernel, has_invalid=padded)
            size = smla.smla_decode_workspace_size(2, h, 0, n, **kw)
            ws = torch.zeros(size, dtype=torch.uint8, device=DEV)
            found[f"decode_{kernel}_{padded}"] = lambda ws=ws, kw=kw: smla.smla_decode(*args, workspace_tensor=ws, **kw)
    return found


def test_an_error_of_another_library_is_no_failure_of_a_launch(cudart, monkeypatch):
    # the last error of the process's runtime, made by a call that names no device: not a launch's of
    # these calls, which go through at the first try, and still there behind them (except where a
    # kernel's shared memory is set, when the runtime itself drops it)
    everything = {**calls(), **decode_calls()}
    for call in everything.values():
        call()
    torch.cuda.synchronize()

    def second_try(*_):
        raise AssertionError("the call was made again")

    monkeypatch.setattr(smla, "_current_device", second_try)
    for name, call in everything.items():
        bad = cudart.cudaSetDevice(4096)
        assert bad != 0
        call()
        if name in ("write", "read", "append", "tree", "accept", "pack"):
            assert cudart.cudaPeekAtLastError() == bad, name
    cudart.cudaGetLastError()
    torch.cuda.synchronize()


@pytest.mark.parametrize("name", CALLS)
def test_a_launch_that_fails_is_raised_and_not_made_again(name, cudart, monkeypatch):
    # a stream whose capture has been made invalid (by a synchronisation) takes no launch
    call, stream, graph = calls()[name], torch.cuda.Stream(), ctypes.c_void_p()
    call()
    torch.cuda.synchronize()
    handle, relaxed = ctypes.c_void_p(stream.cuda_stream), 2

    def second_try(*_):
        raise AssertionError("the call was made again")

    monkeypatch.setattr(smla, "_current_device", second_try)
    assert cudart.cudaStreamBeginCapture(handle, relaxed) == 0
    try:
        assert cudart.cudaStreamSynchronize(handle) != 0
        with torch.cuda.stream(stream):
            with pytest.raises(smla.SmlaError) as e:
                call()
        assert e.value.code == -8
    finally:
        cudart.cudaStreamEndCapture(handle, ctypes.byref(graph))
        cudart.cudaGetLastError()
    assert not graph
    call()
    torch.cuda.synchronize()


def test_threads_with_streams_of_their_own_get_what_one_gets():
    # four Python threads make whole steps at once, each on its stream, over batches of its own
    def batch(i):
        return [[(20, 300), (9, 100)], [(3, 40), (2, 9)], [(1, 700)] * 9, [(60, 200)]][i]

    def state(i):
        c = Batch(batch(i), 16, seed=i)
        return step_state(c, 16, 90 + i)

    def bits_of(s):
        return [s[k] for k in ("mask", "pos", "q", "kv", "out", "lse", "new")]

    want = []
    for i in range(4):
        s = state(i)
        step(s)
        torch.cuda.synchronize()
        want.append(bits_of(s))
    states = [[state(i) for _ in range(12)] for i in range(4)]
    streams, failed = [torch.cuda.Stream() for _ in range(4)], []
    torch.cuda.synchronize()
    start = threading.Barrier(4)

    def work(i):
        try:
            with torch.cuda.stream(streams[i]):
                start.wait(10)
                for s in states[i]:
                    step(s)
        except Exception as e:
            failed.append(e)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert failed == []
    for i in range(4):
        for s in states[i]:
            assert all(torch.equal(a, b) for a, b in zip(bits_of(s), want[i]))

"""The paged calls of _smla.so beside the rest of a process: other Python threads."""

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

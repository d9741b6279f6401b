"""Rules that the attend kernels' source keeps, where no run can show a fault: a compiler may
or may not bring a warp's lanes back together behind a branch."""

import os
import re

import pytest

SOURCE = os.path.join(os.path.dirname(__file__), "..", "sparse_mla_decode_csr_gb300", "csrc", "smla_paged_attend.cu")


def functions():
    """name -> body of every device function, without comments."""
    text = re.sub(r"//[^\n]*", "", open(SOURCE).read())
    text = re.sub(r"__(?:cluster_dims|launch_bounds)__\([^()]*\)", "", text)
    found = {}
    for m in re.finditer(r"(?:__device__|__global__)[^;{}()]*?\b(\w+)\([^;{}]*?\)\s*(?:const\s*)?\{", text):
        depth, i = 1, m.end()
        while depth:
            depth += {"{": 1, "}": -1}.get(text[i], 0)
            i += 1
        found.setdefault(m.group(1), "")
        found[m.group(1)] += text[m.end():i]
    return found


COMPUTE = ("softmax_role", "narrow_softmax_role", "few_compute_role")


def test_the_functions_are_found():
    assert set(COMPUTE) | {"wait_for", "load_q_tmem", "find_range", "paged_attend_kernel", "paged_merge_kernel"} <= set(functions())


def test_lanes_meet_after_every_wait():
    # a lane may leave a wait's loop earlier than its neighbours; tensor-memory accesses
    # and barriers that follow belong to the whole warp
    for name, body in functions().items():
        if "wait_for(" in body:
            assert name in ("warp_wait", "meet_after"), name
    assert re.search(r"wait_for\([^;]*;\s*__syncwarp\(\);", functions()["meet_after"])
    assert re.search(r"__all_sync\(0xffffffffu, wait_for\(", functions()["warp_wait"])


def test_lanes_meet_before_every_barrier_of_warps():
    for name, body in functions().items():
        for m in re.finditer(r"\bnamed_barrier(?:_or)?\(", body):
            lead = body[:m.start()].rstrip()
            lead = lead[:lead.rfind(";") + 1]
            assert lead.endswith("__syncwarp();"), name


@pytest.mark.parametrize("name", COMPUTE)
def test_no_lane_leaves_a_loop_over_tensor_memory(name):
    assert "continue" not in functions()[name]

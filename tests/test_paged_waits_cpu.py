"""Every wait of the attend kernels' source brings its lanes back together: a lane may leave a
wait's loop earlier than its neighbours, and tensor-memory accesses, MMAs and barriers that follow
belong to the whole warp.  (The pair kernel's waits beside those of test_paged_source_cpu.)"""

import re

import pytest

import test_paged_source_cpu as source

# what may poll a barrier: the waits themselves, and roles of one thread
POLLS = {"mbar_try_wait": {"wait_on", "wait_for", "thread_wait", "next_softmax", "scheduler_role"},
         "mbar_test": {"copier_role"},
         "mbar_wait": {"copier_role", "paged_attend_kernel", "paged_attend_narrow_kernel", "paged_attend_few_kernel"},
         "thread_wait": {"pair_wait", "meet_pair", "next_thread"},
         "next_thread": {"copier_role"}}
ONE_THREAD = {"copier_role": r"if \(\(threadIdx\.x & 31\) == 0\) copier_role\(",
              "scheduler_role": r"if \(\(threadIdx\.x & 31\) == 0\) scheduler_role\("}
# what is between a poll and the next step of the warp
MEETS = {"pair_wait": r"return __all_sync\(0xffffffffu, thread_wait\(ms, bar, parity\)\);",
         "meet_pair": r"thread_wait\(ms, bar, parity\);\s*__syncwarp\(\);",
         "next_softmax": r"while \(!\(got = mbar_try_wait\([^;]*\)\)\)\s*if \([^;]*\) break;\s*if \(!__all_sync\(0xffffffffu, got\)\)",
         "next_unit": r"if \(!pair_wait\(",
         "warp_wait": r"return __all_sync\(0xffffffffu, wait_for\("}


def faults(found):
    bad = []
    for name, body in found.items():
        for poll, allowed in POLLS.items():
            if re.search(rf"\b{poll}\(", body) and name not in allowed:
                bad.append(f"{name} polls by {poll}")
        # an elected thread alone waits for its MMAs
        if name.startswith("paged_attend"):
            for m in re.finditer(r"\bmbar_wait\(", body):
                if "elect_one()" not in body[:m.start()][-600:]:
                    bad.append(f"{name} waits by more than an elected thread")
    bad += [f"{name} does not bring its lanes together" for name, rule in MEETS.items() if not re.search(rule, found[name])]
    bad += [f"{name} is not one thread's" for name, rule in ONE_THREAD.items()
            if not re.search(rule, found["paged_attend_kernel"])]
    # the softmax warps go on whatever a wait answers: their waits are the ones that meet
    for name in source.COMPUTE:
        waits = set(re.findall(r"\b(\w*wait\w*|meet\w*)\(", found[name]))
        if not waits <= {"meet_pair", "meet_after", "tmem_wait_ld", "tmem_wait_st"}:
            bad.append(f"{name} waits by {sorted(waits)}")
    return bad


def test_every_wait_brings_its_lanes_together():
    assert faults(source.functions()) == []


@pytest.mark.parametrize("name,what,instead", [
    ("meet_pair", "__syncwarp();", ""), ("pair_wait", "__all_sync(0xffffffffu, ", "("),
    ("next_softmax", "__all_sync(0xffffffffu, got)", "got"), ("softmax_role", "meet_pair(", "thread_wait("),
    ("issuer_pv_role", "pair_wait(", "thread_wait("), ("loader_role", "pair_wait(", "mbar_try_wait("),
    ("paged_attend_kernel", "if ((threadIdx.x & 31) == 0) scheduler_role(", "scheduler_role(")])
def test_a_wait_without_its_meeting_is_found(name, what, instead):
    found = source.functions()
    assert what in found[name]
    found[name] = found[name].replace(what, instead)
    assert faults(found) != []

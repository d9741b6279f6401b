"""Rules of the kernels that are launched as dependents of what is before them in the stream, where
no run can show a fault: such a kernel may be resident while the one before it still writes, so
nothing that it reads may go through the read-only path, or set out before its wait."""

import os
import re

import pytest

from test_paged_source_cpu import functions as attend_functions

CSRC = os.path.join(os.path.dirname(__file__), "..", "sparse_mla_decode_csr_gb300", "csrc")
DEPENDENTS = {"smla_paged_append.cu": ["paged_append_kernel"],
              "smla_paged_tree.cu": ["paged_tree_kernel", "paged_accept_kernel"]}
BATCH = ("cu_at", "seq_len_at", "record_at", "seq_of_row")  # what reads the batch's arrays


def source(name):
    return re.sub(r"//[^\n]*", "", open(os.path.join(CSRC, name)).read())


@pytest.mark.parametrize("name", sorted(DEPENDENTS))
def test_dependents_read_nothing_through_the_read_only_path(name):
    text = source(name)
    # __restrict__ makes a pointer to const one that the compiler may read that way
    for word in ("__ldg", "_now(", ".nc", "__restrict__"):
        assert word not in text, word
    for f in BATCH + ("load_i32",):
        assert not re.search(rf"\b{f}\s*\(", text) and not re.search(rf"\b{f}<(?!kFresh>)", text), f
    headers = source("smla_paged_copy.cuh")
    assert "__ldg" not in headers and "_now(" not in headers and ".nc" not in headers


def test_loads_behind_the_wait_stay_there():
    text = source("smla_paged.cuh")
    assert re.search(r"asm volatile\(\"griddepcontrol\.wait;\"", text)
    loads = re.findall(r"asm( volatile)?\(\"ld\.global(\S*)", text)
    assert loads and all(volatile and ".nc" not in kind for volatile, kind in loads)
    assert text.count("__ldg") == 1 and re.search(r"kLoads == kReadOnly\) return __ldg", text)


@pytest.mark.parametrize("name", sorted(DEPENDENTS))
def test_dependents_wait_before_they_read(name):
    text = source(name)
    for kernel in DEPENDENTS[name]:
        body = text[re.search(rf"\b{kernel}\(", text).end():]
        lead = body[body.index("{") + 1:body.index("wait_for_primary();")]
        # declarations, and nothing that leaves: a grid's end has to mean the end of those before it
        assert "return" not in lead and "[" not in re.sub(r"__shared__[^;]*;", "", lead) and "load" not in lead
        assert f"launch_dependent({kernel}" in text


@pytest.mark.parametrize("name", ["paged_merge_kernel", "paged_merge_pair_kernel"])
def test_merges_read_partials_past_the_read_only_path(name):
    body = attend_functions()[name]
    assert "__ldg" not in body and "_now(" not in body and "return" not in body[:body.index("wait_for_primary();")]

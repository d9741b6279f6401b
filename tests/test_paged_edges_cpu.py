"""Edges of the paged cache's host checks."""

import ctypes

import pytest

import sparse_mla_decode_csr_gb300 as smla
from test_paged_cpu import attend_params


@pytest.mark.parametrize("scale", [3e38, -3e38, 2.4e38])
def test_attend_refuses_a_scale_that_overflows_in_log2_units(scale):
    # 2.4e38 log2(e) is beyond the largest f32, 3.40e38: an infinite factor would turn
    # scores of zero into NaN
    assert smla.lib.smla_paged_attend(ctypes.byref(attend_params(sm_scale=scale)), None, 0, None) == -2


@pytest.mark.parametrize("scale", [2.3e38, -2.3e38, 1e-45, 0.0])
def test_attend_takes_every_scale_that_does_not(scale):
    # (a batch without rows: the checks alone)
    p = attend_params(sm_scale=scale)
    p.batch.n_rows = 0
    assert smla.lib.smla_paged_attend(ctypes.byref(p), None, 0, None) == 0

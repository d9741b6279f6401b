"""_smla.so takes well-formed calls only: whatever else it is given it answers with False,
without raising, so that the checks in Python name the fault."""

import pytest
import torch

from sparse_mla_decode_csr_gb300 import _native

CALLS = {"write": 8, "read": 8, "append": 14, "tree": 7, "attend": 14, "accept": 9}


@pytest.mark.parametrize("name", sorted(CALLS))
def test_arguments_of_any_kind_are_refused(name):
    call, n = getattr(_native, name), CALLS[name]
    host = torch.zeros(3, 4)
    for args in ([], [None] * n, [0] * n, ["x"] * n, [host] * n, [host] * (n - 1), [host] * (n + 1), [object()] * n,
                 [torch.zeros(2, 2).to_sparse()] * n, [torch.zeros(2, device="meta")] * n, [float("nan")] * n):
        assert call(*args) is False


def test_a_flag_that_raises_is_refused():
    class Odd:
        def __bool__(self):
            raise ValueError("no truth value")

        def __float__(self):
            raise ValueError("no number")

    assert _native.append(*[Odd()] * 14) is False and _native.attend(*[Odd()] * 14) is False

"""What the calls in Python make of the answers of _smla.so."""

import pytest
import torch

import sparse_mla_decode_csr_gb300 as smla

Z = torch.zeros(1)
CALLS = {
    "write": lambda: smla.smla_paged_write(Z, Z, Z, Z, Z, Z),
    "read": lambda: smla.smla_paged_read(Z, Z, Z, Z, Z, Z),
    "append": lambda: smla.smla_paged_append(Z, Z, Z, Z, Z, Z, Z),
    "tree": lambda: smla.smla_paged_tree(Z, Z, Z, Z, Z),
    "attend": lambda: smla.smla_paged_attend(Z, Z, Z, Z, Z, 1.0, None, Z, Z),
    "attend_tree": lambda: smla.smla_paged_attend_tree(Z, Z, Z, Z, Z, Z, 1.0, None, Z, Z),
    "accept": lambda: smla.smla_paged_accept(Z, Z, Z, Z, Z, Z),
}


@pytest.mark.parametrize("name", sorted(CALLS))
def test_answers_of_the_native_calls(name, monkeypatch):
    asked = []

    def answers(value):
        def native(*args):
            asked.append(value)
            return value
        monkeypatch.setattr(smla._native, name.replace("_tree", ""), native)

    answers(True)
    assert CALLS[name]() is None  # made
    answers(-8)  # SMLA_ERR_LAUNCH: not made again, where the checks would refuse these tensors
    with pytest.raises(smla.SmlaError) as e:
        CALLS[name]()
    assert e.value.code == -8 and f"smla_paged_{name}" in str(e.value)
    answers(False)
    with pytest.raises(smla.SmlaError) as e:
        CALLS[name]()
    assert e.value.code == smla.SMLA_ERR_SHAPE and asked == [True, -8, False]

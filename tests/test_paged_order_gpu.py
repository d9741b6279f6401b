"""What the paged calls leave to an order: units of the pair kernel that end faster than its
ring turns."""

import numpy as np
import pytest
import torch

from test_paged_gpu import Batch, attend, check
from test_paged_tree_gpu import random_trees, tree_attend, tree_check, words_of

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("heads,tokens", [(128, 1), (100, 1), (16, 8)])
@pytest.mark.parametrize("longest", [64, 150])
def test_many_units_of_one_tile_for_each_worker(heads, tokens, longest):
    # row tiles over few positions: a worker of the pair kernel has six of them and more, the
    # first of them often of a single key tile
    r = np.random.default_rng(heads + longest)
    lens = [(tokens, int(n)) for n in r.integers(tokens, longest + 1, 520)]
    c = Batch(lens, 16)
    q, sk, out, lse, st = attend(c, heads, sink=True)
    check(c, q, out, lse, 1 / 24, sk, True)
    assert st == 0
    _, sets = random_trees(c, 3)
    q, sk, out, lse, st = tree_attend(c, heads, words_of(sets, 1), sink=True)
    tree_check(c, q, sets, out, lse, 1 / 24, sk)
    assert st == 0

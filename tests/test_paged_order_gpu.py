"""What the paged calls leave to an order: units of the pair kernel that end faster than its
ring turns; steps whose calls read what the call before wrote."""

import numpy as np
import pytest
import torch

import sparse_mla_decode_csr_gb300 as smla
from test_paged_append_gpu import FREQ, inputs
from test_paged_gpu import DEV, Batch, attend, check
from test_paged_tree_gpu import random_trees, tree_attend, tree_check, words_of

pytestmark = pytest.mark.gpu
I32 = torch.int32


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


def lengths_in_place(n_seqs, nodes, steps):
    """Steps over drafted trees whose accepts write the lengths in place, the next calls reading
    them there: tree, append, accept; the last accepted token written again by tree and append;
    the next tree's nodes added."""
    c = Batch([(nodes, 40 + 3 * b + nodes) for b in range(n_seqs)], 16, spare_pages=0)
    pages = -(-int(c.seq_lens.max() + steps * nodes) // 16)
    table = torch.randperm(n_seqs * pages, generator=c.g).to(I32).view(n_seqs, pages)
    d = dict(kv0=torch.zeros(n_seqs * pages, 16, 656, dtype=torch.uint8), table=table, cu=c.cu,
             one=torch.arange(n_seqs + 1, dtype=I32), sl0=c.seq_lens, roots=torch.full((n_seqs,), -1, dtype=I32))
    r = np.random.default_rng(nodes)
    sl, want = c.seq_lens.numpy().astype(np.int64).copy(), []
    for k in range(steps):
        parents, sets = random_trees(c, 100 * nodes + k)
        path = torch.full((n_seqs, 8), -1, dtype=I32)
        past, new = sl - nodes, np.zeros(n_seqs, np.int64)
        for b in range(n_seqs):
            keep = sorted(max(sets[b * nodes:(b + 1) * nodes], key=len))[:int(r.integers(1, 9))]
            path[b, :len(keep)] = torch.tensor(keep, dtype=I32)
            new[b] = past[b] + len(keep)
        lat, rope, q = inputs(c, 2, "bf16", seed=k)
        d[f"parents{k}"], d[f"path{k}"], d[f"lat{k}"], d[f"rope{k}"], d[f"q{k}"] = parents, path, lat, rope, q
        want.append((np.repeat(past, nodes) + [len(s) - 1 for s in sets], new - 1, new))
        sl = new + nodes
    d = {k: v.to(DEV) for k, v in d.items()}
    turns = smla.smla_rotation_turns(FREQ)

    def run(apart):
        """All steps; `apart`: each call by itself, with lengths of its own."""
        kv, sl, got = d["kv0"].clone(), d["sl0"].clone(), []

        def behind(t):
            if not apart:
                return t
            torch.cuda.synchronize()
            return t.clone()

        for k in range(steps):
            pos, pos1 = torch.zeros(n_seqs * nodes, dtype=I32, device=DEV), torch.zeros(n_seqs, dtype=I32, device=DEV)
            q_out, q1 = torch.zeros_like(d[f"q{k}"]), torch.zeros_like(d[f"q{k}"][:n_seqs])
            lat, rope, q = d[f"lat{k}"], d[f"rope{k}"], d[f"q{k}"]
            smla.smla_paged_tree(d[f"parents{k}"], d["cu"], sl, None, pos)
            sl, p = behind(sl), behind(pos)
            smla.smla_paged_append(lat, rope, kv, d["table"], d["cu"], sl, turns, q_rope=q, q_out=q_out, positions=p)
            new = torch.zeros_like(sl) if apart else sl
            smla.smla_paged_accept(kv, d["table"], d["cu"], behind(sl), d[f"path{k}"], new)
            sl = behind(new)
            smla.smla_paged_tree(d["roots"], d["one"], sl, None, pos1)
            smla.smla_paged_append(lat[:n_seqs] * 2, rope[:n_seqs], kv, d["table"], d["one"], behind(sl), turns,
                                   q_rope=q[:n_seqs], q_out=q1, positions=behind(pos1))
            sl = behind(sl)
            got.append([pos, pos1, q_out, q1, kv.clone(), sl.clone()])
            if apart:
                torch.cuda.synchronize()
                sl = sl + nodes
            else:
                sl.add_(nodes)
        return got

    return run, want


@pytest.mark.parametrize("n_seqs,nodes", [(1, 5), (64, 9), (300, 3), (5, 200)])
def test_lengths_that_an_accept_wrote_in_place_are_read_behind_it(n_seqs, nodes):
    run, want = lengths_in_place(n_seqs, nodes, 6)
    apart = run(True)
    torch.cuda.synchronize()
    for (pos, pos1, *_, sl), (p, p1, new) in zip(apart, want):
        assert pos.tolist() == p.tolist() and pos1.tolist() == p1.tolist() and sl.tolist() == new.tolist()

    def same(got):
        torch.cuda.synchronize()
        for k, (a, b) in enumerate(zip(got, apart)):
            for x, y in zip(a, b):
                assert torch.equal(x, y), k

    same(run(False))
    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        got = run(False)
    for _ in range(3):
        for x in [y for g in got for y in g]:
            x.fill_(0)
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            graph.replay()
        same(got)

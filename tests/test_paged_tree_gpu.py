"""Trees of drafted tokens on the GPU against plain 64-bit evaluations: masks and
positions, attention by masks in each kernel, accepted paths, and a verification step
of all of them."""

import numpy as np
import pytest
import torch

import oracle
import sparse_mla_decode_csr_gb300 as smla
from smla_testlib import allowance, bits
from test_paged_append_gpu import FREQ, check_append, check_rotated, inputs
from test_paged_gpu import DEV, REC, Batch, gen, unpack

pytestmark = pytest.mark.gpu
I32 = torch.int32


def words_of(sets, words):
    """Mask int32 [rows, words] of sets of nodes."""
    m = np.zeros((len(sets), max(words, 1)), np.uint32)
    for r, nodes in enumerate(sets):
        for j in nodes:
            if j // 32 < words:
                m[r, j // 32] |= np.uint32(1 << (j % 32))
    return torch.from_numpy(m[:, :words].view(np.int32))


def random_trees(c, seed, deep=0.5):
    """Parents by row, and the sets of ancestors (with the node itself) by row."""
    r = np.random.default_rng(seed)
    parents, sets = torch.full((c.rows,), -7, dtype=I32), [set() for _ in range(c.rows)]
    for b, (n, _) in enumerate(c.lens):
        for i in range(n):
            row = int(c.cu[b]) + i
            p = i - 1 if r.random() < deep else int(r.integers(-1, i)) if i else -1
            parents[row] = p if p >= 0 else -int(r.integers(1, 5))
            sets[row] = {i} | (sets[row - i + p] if p >= 0 else set())
    return parents, sets


def run_tree(c, parents, words, *, mask=True, positions=True, pad=0):
    buf = torch.full((c.rows, words + pad), 0x55555555, dtype=I32, device=DEV)
    pos = torch.full((c.rows,), -99, dtype=I32, device=DEV)
    status = torch.zeros(1, dtype=I32, device=DEV)
    _, cu, sl = c.dev()
    smla.smla_paged_tree(parents.to(DEV), cu, sl, buf[:, :words] if mask else None, pos if positions else None,
                         status=status)
    return buf.cpu(), pos.cpu(), int(status)


TREES = [
    # lens, words, pad
    ([(1, 1)], 1, 0), ([(60, 500)] * 5, 2, 0), ([(5, 9), (0, 4), (1, 70), (33, 33), (64, 64), (65, 90)], 3, 1),
    ([(500, 700), (129, 129)], 16, 2), ([(1000, 1000)], 32, 0), ([(7, 3), (2, 0)], 1, 0), ([(3, 10)] * 300, 1, 0),
    ([(2500, 2600), (2048, 2048), (40, 50)], 79, 1),  # more nodes than shared memory takes, more words than a round
]


@pytest.mark.parametrize("lens,words,pad", TREES)
@pytest.mark.parametrize("deep", [0.0, 0.5, 1.0])
def test_masks_and_positions(lens, words, pad, deep):
    c = Batch(lens, 16, front=1, behind=2)
    parents, sets = random_trees(c, 7, deep)
    mask, pos, st = run_tree(c, parents, words, pad=pad)
    want = words_of(sets, words)
    rows = [r for r, _, _ in c.positions()]
    assert torch.equal(mask[rows, :words], want[rows])
    depth = {r: len(sets[r]) - 1 for r in rows}
    first = {r: s - n for b, (n, s) in enumerate(c.lens) for r in range(int(c.cu[b]), int(c.cu[b]) + n)}
    assert all(int(pos[r]) == first[r] + depth[r] for r in rows)
    others = np.setdiff1d(np.arange(c.rows), rows)
    assert (mask[others] == 0x55555555).all() and (pos[others] == -99).all() and (mask[:, words:] == 0x55555555).all()
    assert st == 0
    only_mask = run_tree(c, parents, words, positions=False)
    only_pos = run_tree(c, parents, words, mask=False)
    assert torch.equal(only_mask[0], mask[:, :words]) and (only_mask[1] == -99).all()
    assert torch.equal(only_pos[1], pos) and (only_pos[0] == 0x55555555).all() and only_pos[2] == 0


def test_parents_that_are_no_lower_nodes_are_roots():
    c = Batch([(6, 20), (4, 4)], 16)
    parents = torch.tensor([0, 0, 5, 2, 2 ** 31 - 1, -(2 ** 31), -1, 1, 0, 2], dtype=I32)
    mask, pos, st = run_tree(c, parents, 1)
    sets = [{0}, {0, 1}, {2}, {2, 3}, {4}, {5}, {0}, {1}, {0, 2}, {0, 2, 3}]
    assert torch.equal(mask, words_of(sets, 1))
    assert pos.tolist() == [14, 15, 14, 15, 14, 14, 0, 0, 1, 2]
    assert st == smla.STATUS_INDEX_OOB


def test_nodes_behind_the_words_are_left_out_and_flagged():
    c = Batch([(70, 100)], 16)
    parents, sets = random_trees(c, 2, 0.8)
    mask, pos, st = run_tree(c, parents, 1)
    assert torch.equal(mask, words_of(sets, 1)) and st == smla.STATUS_INDEX_OOB
    assert pos.tolist() == [29 + len(s) for s in sets]


# ---- attention by masks ----


def tree_reference(c, q, sets, sm_scale, sink, causal=False, operand_rel=0.0):
    idx, ptr, rows = [], [0], []
    for r, b, p in c.positions():
        n, s = c.lens[b]
        idx += [c.slot(b, t) for t in range(max(s - n, 0))]
        idx += [c.slot(b, s - n + j) for j in sorted(sets[r]) if j < n and s - n + j >= 0 and not (causal and s - n + j > p)]
        ptr.append(len(idx))
        rows.append(r)
    idx, ptr = np.array(idx, np.int32), np.array(ptr, np.int32)
    qq = q.double().numpy()[rows]
    sk = None if sink is None else sink.double().numpy()
    out, lse, _ = oracle.sparse_mla_decode(qq, c.rec, idx, ptr, None, sm_scale, sk)
    return rows, out, lse, allowance(qq, c.rec, idx, ptr, None, sm_scale, sk, operand_rel=operand_rel)


def tree_check(c, q, sets, out, lse, sm_scale, sink, causal=False, operand_rel=0.0):
    """The bounds of smla_paged_attend's tests: its roundings (see check there)."""
    rows, ref, ref_lse, (a_out, a_lse) = tree_reference(c, q, sets, sm_scale, sink, causal, operand_rel)
    got, got_lse = out.double().cpu().numpy(), lse.double().cpu().numpy()
    assert np.isfinite(got[rows]).all()
    err = np.abs(got[rows] - ref) - (a_out + 2.0 ** -8 * np.abs(ref) + 1e-30)
    assert err.max(initial=-1) <= 0, f"out exceeds its bound by {err.max():.3g} at {np.unravel_index(err.argmax(), err.shape)}"
    assert np.array_equal(np.isneginf(got_lse[rows]), np.isneginf(ref_lse))
    fin = np.isfinite(ref_lse)
    e = np.abs(got_lse[rows][fin] - ref_lse[fin]) - (a_lse[fin] + 2.0 ** -18 * (1 + np.abs(ref_lse[fin]).max(initial=0)))
    assert e.max(initial=-1) <= 0, f"lse exceeds its bound by {e.max():.3g}"
    others = np.setdiff1d(np.arange(c.rows), rows)
    assert (got[others] == 7.0).all() and (got_lse[others] == 7.0).all()


def tree_attend(c, heads, mask, *, sink=False, causal=False, sm_scale=1 / 24, q=None, kv=None, seed=5, **kw):
    if q is None:
        q = torch.randn(c.rows, heads, 576, generator=gen(seed)).to(torch.bfloat16)
    sk = torch.randn(heads, generator=gen(seed + 1)) if sink else None
    out = torch.full((c.rows, heads, 512), 7.0, dtype=torch.bfloat16, device=DEV)
    lse = torch.full((c.rows, heads), 7.0, device=DEV)
    status = torch.zeros(1, dtype=I32, device=DEV)
    smla.smla_paged_attend_tree(q.to(DEV), c.cache() if kv is None else kv, *c.dev(), mask.to(DEV), sm_scale,
                                None if sk is None else sk.to(DEV), out, lse, causal=causal, status=status, **kw)
    torch.cuda.synchronize()
    return q, sk, out, lse, int(status)


EMPTY = [(0, 0)] * 60  # lowers the mean number of rows: the kernels of few rows
# lens by the kernel that serves them with the heads beside them
KERNELS = {
    "few": (16, [(1, 95), (3, 97), (2, 192), (5, 5), (1, 1), (7, 700), (40, 130)] + EMPTY),
    "few_1": (1, [(33, 33), (70, 500), (17, 1200), (100, 160)] + EMPTY),
    "narrow32": (30, [(3, 200), (9, 150), (1, 64), (5, 333), (35, 64)] + EMPTY),
    "narrow64": (64, [(1, 200), (7, 150), (2, 64), (33, 97)] + EMPTY),
    "narrow64_7": (7, [(9, 200), (7, 150), (2, 64), (10, 77)]),
    "pair": (16, [(60, 300), (9, 9), (17, 200), (0, 50), (33, 140), (2, 64)]),
    "pair_128": (128, [(5, 90), (34, 70)]),
    "pair_7": (7, [(130, 400), (64, 128), (65, 129)]),
}


@pytest.mark.parametrize("page", [1, 20, 64])
@pytest.mark.parametrize("kernel", sorted(KERNELS))
def test_attend_trees(kernel, page):
    heads, lens = KERNELS[kernel]
    c = Batch(lens, page, front=1, behind=2, page_pad=16)
    _, sets = random_trees(c, 11)
    most = max(n for n, _ in lens)
    q, sk, out, lse, st = tree_attend(c, heads, words_of(sets, -(-most // 32)), sink=True)
    tree_check(c, q, sets, out, lse, 1 / 24, sk)
    assert st == 0


@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("kernel", sorted(KERNELS))
def test_attend_any_masks(kernel, causal):
    # bits drawn at random: later nodes, rows that do not see themselves, rows that see
    # nothing but the history, bits behind the sequence's rows
    heads, lens = KERNELS[kernel]
    c = Batch(lens, 16, behind=1)
    r = np.random.default_rng(4)
    words = -(-max(n for n, _ in lens) // 32)
    density = r.choice([0.0, 0.1, 0.5, 1.0], c.rows)
    sets = [set(np.nonzero(r.random(words * 32) < d)[0].tolist()) for d in density]
    q, sk, out, lse, _ = tree_attend(c, heads, words_of(sets, words), causal=causal, sink=causal)
    tree_check(c, q, sets, out, lse, 1 / 24, sk, causal)


@pytest.mark.parametrize("heads", [16, 30, 64, 128])
def test_no_words_and_too_few(heads):
    # without words a row sees the history alone, and nothing where there is none
    c = Batch([(3, 100), (2, 2), (40, 90)] + (EMPTY if heads < 128 else []), 16)
    for words in (0, 1):
        sets = [set(range(40)) for _ in range(c.rows)]
        q, sk, out, lse, _ = tree_attend(c, heads, words_of(sets, words), sink=True)
        tree_check(c, q, [{j for j in s if j < 32 * words} for s in sets], out, lse, 1 / 24, sk)
        if words == 0:
            assert (out[3:5] == 0).all() and torch.isneginf(lse[3:5]).all()


@pytest.mark.parametrize("heads", [16, 30, 64, 128])
def test_a_mask_of_all_lower_nodes_is_the_causal_edge(heads):
    c = Batch([(9, 300), (1, 64), (40, 41)] + (EMPTY if heads < 128 else []), 16)
    sets = [set() for _ in range(c.rows)]
    for r, b, p in c.positions():
        sets[r] = set(range(p - (c.lens[b][1] - c.lens[b][0]) + 1))
    q = torch.randn(c.rows, heads, 576, generator=gen(5)).to(torch.bfloat16)
    want = torch.empty(c.rows, heads, 512, dtype=torch.bfloat16, device=DEV)
    want_lse = torch.empty(c.rows, heads, device=DEV)
    smla.smla_paged_attend(q.to(DEV), c.cache(), *c.dev(), 1 / 24, None, want, want_lse)
    # the same schedule (causal) gives the same bits
    _, _, out, lse, _ = tree_attend(c, heads, words_of(sets, 2), q=q, causal=True)
    assert torch.equal(out, want) and torch.equal(lse, want_lse)
    _, _, out, lse, _ = tree_attend(c, heads, words_of(sets, 2), q=q)
    tree_check(c, q, sets, out, lse, 1 / 24, None)
    full = torch.full((c.rows, 2), -1, dtype=I32)
    smla.smla_paged_attend(q.to(DEV), c.cache(), *c.dev(), 1 / 24, None, want, want_lse, causal=False)
    _, _, out, lse, _ = tree_attend(c, heads, full, q=q)
    assert torch.equal(out, want) and torch.equal(lse, want_lse)


@pytest.mark.parametrize("heads,lens", [(16, [(33, 9000)]), (64, [(3, 5000), (70, 400), (1, 2500)]), (16, [(1, 9000)] + EMPTY),
                                        (64, [(1, 4000), (1, 3000)])])
def test_long_histories_are_split(heads, lens):
    c = Batch(lens, 64)
    _, sets = random_trees(c, 3)
    q, sk, out, lse, _ = tree_attend(c, heads, words_of(sets, 3), sink=True)
    tree_check(c, q, sets, out, lse, 1 / 24, sk)


@pytest.mark.parametrize("heads", [16, 128])
def test_rows_before_the_start_and_pages_that_are_not_there(heads):
    c = Batch([(6, 3), (4, 0), (3, 70), (9, 40), (5, 64)] + (EMPTY if heads == 16 else []), 16)
    c.table[2, :] = -1
    c.table[3, 1] = -1
    c.seq_lens[4], c.lens[4] = 16 * c.table.shape[1] + 3, (5, 16 * c.table.shape[1] + 3)  # the last three nodes past the table
    c.table[4] = c.table[4, 0]
    _, sets = random_trees(c, 9)
    q, sk, out, lse, st = tree_attend(c, heads, words_of(sets, 1), sink=True)
    tree_check(c, q, sets, out, lse, 1 / 24, sk)
    assert st == smla.STATUS_INDEX_OOB


@pytest.mark.parametrize("kernel", ["few", "narrow32", "narrow64", "pair"])
def test_hidden_nodes_never_reach_a_row(kernel):
    heads = {"few": 16, "narrow32": 30, "narrow64": 64, "pair": 128}[kernel]
    c = Batch([(6, 75)] + (EMPTY if kernel != "pair" else []), 16)
    sets = [{0}, {0, 1}, {0, 2}, {0, 1, 3}, {0, 2, 4}, {5}]
    mask = words_of(sets, 1)
    q, _, want, want_lse, _ = tree_attend(c, heads, mask)
    c.rec[c.slot(0, 70), 7] = 0x7F                                                             # node 1: a NaN code
    c.rec[c.slot(0, 73), 528:530] = np.array([0x7F80], np.uint16).view(np.uint8)               # node 4: infinite rope
    c.rec[c.slot(0, 74), 512:516] = np.array([np.inf], np.float32).view(np.uint8)              # node 5: infinite scale
    _, _, out, lse, _ = tree_attend(c, heads, mask, q=q)
    clean = [0, 2]
    assert torch.equal(out[clean], want[clean]) and torch.equal(lse[clean], want_lse[clean])
    for bad in (1, 3, 5):
        assert torch.isnan(out[bad].float()).all() and torch.isnan(lse[bad]).all()
    assert not torch.equal(lse[4], want_lse[4])


@pytest.mark.parametrize("heads", [16, 64, 128])
def test_sharp_scores_and_odd_scales(heads):
    c = Batch([(6, 700), (40, 150)] + (EMPTY if heads == 16 else []), 64, std=3.0)
    _, sets = random_trees(c, 5)
    for scale in (1.0, -0.3, 0.0):
        q, sk, out, lse, _ = tree_attend(c, heads, words_of(sets, 2), sm_scale=scale, sink=True)
        tree_check(c, q, sets, out, lse, scale, sk)


def test_strided_tensors_workspace_and_no_lse():
    c = Batch([(7, 90), (35, 60)], 16)
    _, sets = random_trees(c, 6)
    qb = torch.randn(c.rows, 12, 600, generator=gen(1)).to(torch.bfloat16).to(DEV)
    ob = torch.full((c.rows, 12, 520), 3.0, dtype=torch.bfloat16, device=DEV)
    mb = torch.full((c.rows, 5), -1, dtype=I32, device=DEV)
    mb[:, 1:3] = words_of(sets, 2).to(DEV)
    q, out, lse = qb[:, ::2, 8:584], ob[:, 1::2, :512], torch.empty(c.rows, 6, device=DEV)
    n = smla.smla_paged_attend_workspace_size(c.rows, 6, 2, 16, c.table.shape[1])
    ws = torch.full((n + 4096,), 0xAB, dtype=torch.uint8, device=DEV)
    for s in (lse, None):
        smla.smla_paged_attend_tree(q, c.cache(), *c.dev(), mb[:, 1:3], 1 / 24, None, out, s, workspace_tensor=ws[:n])
    tree_check(c, q.cpu(), sets, out, lse, 1 / 24, None)
    assert (ob[:, ::2] == 3.0).all() and (ob[:, :, 512:] == 3.0).all() and (ws[n:] == 0xAB).all()
    with pytest.raises(smla.SmlaError) as e:
        smla.smla_paged_attend_tree(q, c.cache(), *c.dev(), mb[:, 1:3], 1 / 24, None, out, lse, workspace_tensor=ws[:n - 256])
    assert e.value.code == smla.SMLA_ERR_WORKSPACE


@pytest.mark.parametrize("seed", range(12))
def test_trees_drawn_at_random(seed):
    r = np.random.default_rng(300 + seed)
    heads = int(r.choice([1, 3, 7, 16, 18, 33, 40, 64, 90, 128]))
    most = max(1, 1600 // heads)
    lens = [(int(r.integers(0, most)), int(r.integers(0, 500))) for _ in range(int(r.integers(1, 7)))]
    lens += [(1 + most // 3, 300)] + [(0, 0)] * int(r.choice([0, 50]))
    c = Batch(lens, int(r.choice([1, 5, 16, 24, 64, 100])), seed=seed, front=int(r.integers(0, 3)),
              behind=int(r.integers(0, 3)), page_pad=48)
    c.table[torch.rand(c.table.shape, generator=gen(seed)) < 0.08] = -1
    _, sets = random_trees(c, seed, r.random())
    words = max(0, -(-max(n for n, _ in lens) // 32) - int(r.integers(0, 2)))
    q, sk, out, lse, _ = tree_attend(c, heads, words_of(sets, words), sink=bool(seed % 2))
    tree_check(c, q, [{j for j in s if j < 32 * words} for s in sets], out, lse, 1 / 24, sk)


@pytest.mark.parametrize("heads", [16, 128])
def test_a_wait_that_runs_out_sets_the_status(heads):
    c = Batch([(1, 500), (4, 900)] + (EMPTY if heads == 16 else []), 64)
    _, sets = random_trees(c, 1)
    mask = words_of(sets, 1)
    try:
        smla.smla_set_wait_limit(20_000_000, stall_first_wait=True)
        *_, st = tree_attend(c, heads, mask)
        assert st & smla.STATUS_TIMEOUT
    finally:
        smla.smla_set_wait_limit(0)
    q, sk, out, lse, st = tree_attend(c, heads, mask)
    assert st == 0
    tree_check(c, q, sets, out, lse, 1 / 24, sk)


# ---- accepted paths ----


def accepted(c, b, path):
    """The path's nodes up to the first that ends it, and whether that one is flagged."""
    good, last = [], -1
    for j in path:
        if j < 0:
            return good, False
        if j >= c.lens[b][0] or j <= last:
            return good, True
        good.append(j)
        last = j
    return good, False


def accept_check(c, path, pad=0, alias=False):
    """Runs smla_paged_accept on every sequence's path and compares all bytes."""
    kv, (table, cu, sl) = c.cache(), c.dev()
    width = max([len(p) for p in path] + [1])
    p = torch.full((len(path), width + pad), -1, dtype=I32)
    for b, x in enumerate(path):
        p[b, :len(x)] = torch.tensor(x, dtype=I32)
        p[b, width:] = 0
    status = torch.zeros(1, dtype=I32, device=DEV)
    new = sl if alias else torch.full((len(path),), -99, dtype=I32, device=DEV)
    smla.smla_paged_accept(kv, table, cu, sl, p[:, :width].to(DEV) if not pad else p.to(DEV)[:, :width], new, status=status)
    rec, lens, flagged = c.rec.copy(), [], False
    for b, x in enumerate(path):
        n, s = c.lens[b]
        good, odd = accepted(c, b, x)
        flagged |= odd
        for i, j in enumerate(good):
            src, dst = c.slot(b, s - n + j), c.slot(b, s - n + i)
            if src >= 0 and dst >= 0:
                rec[dst] = c.rec[src]
        lens.append(max(s - n + len(good), 0))
    assert np.array_equal(c.buf.cpu()[:, :c.page * REC].reshape(-1, REC).numpy(), rec)
    assert (c.buf[:, c.page * REC:] == 0xEE).all()
    assert new.tolist() == lens
    return int(status), flagged


@pytest.mark.parametrize("page", [1, 16, 48])
@pytest.mark.parametrize("pad,alias", [(0, False), (3, True)])
def test_accept(page, pad, alias):
    c = Batch([(60, 500), (8, 8), (1, 70), (0, 33), (33, 100), (300, 400), (5, 9)], page, page_pad=16, front=1)
    r = np.random.default_rng(page)
    path = [sorted(r.choice(60, 7, replace=False).tolist()), list(range(8)), [0], [], [32],
            sorted(r.choice(300, 150, replace=False).tolist()), []]
    st, flagged = accept_check(c, path, pad, alias)
    assert st == 0 and not flagged


def test_accept_paths_of_any_length_and_shift():
    for n, lens in ((31, 31), (32, 32), (33, 33), (64, 64), (65, 65), (200, 100), (200, 199)):
        c = Batch([(n, 300)] * 3, 16)
        assert accept_check(c, [list(range(n))[:lens], list(range(n - lens, n)), [n - 1]]) == (0, False)


def test_accept_ends_at_entries_that_are_no_path():
    c = Batch([(9, 40)] * 6, 16)
    assert accept_check(c, [[1, 3, 3, 4], [2, 9, 8], [5, 4], [0, 2, -1, 4], [8, 2 ** 31 - 1], [-(2 ** 31), 1]])[0] == smla.STATUS_INDEX_OOB
    assert accept_check(c, [[1, 3, -1, 4]] + [[-1]] * 5)[0] == 0


def test_accept_where_records_are_masked():
    c = Batch([(12, 5), (20, 40), (6, 60)], 16)
    c.table[1, 1], c.table[2, -1] = -1, -1
    c.seq_lens[2], c.lens[2] = 16 * c.table.shape[1] + 2, (6, 16 * c.table.shape[1] + 2)
    c.table[2, :] = torch.arange(c.table.shape[1], dtype=I32)
    c.table[1, 0], c.table[1, 2], c.table[0, 0] = 4, 5, 6
    c.n_pages = max(c.n_pages, 7)
    st, _ = accept_check(c, [[3, 9, 11], [1, 8, 18], [1, 3, 5]])
    assert st == smla.STATUS_INDEX_OOB


def test_accept_without_steps_rows_or_sequences():
    c = Batch([(4, 20), (0, 7)], 16)
    kv, (table, cu, sl) = c.cache(), c.dev()
    new = torch.zeros(2, dtype=I32, device=DEV)
    smla.smla_paged_accept(kv, table, cu, sl, torch.zeros(2, 0, dtype=I32, device=DEV), new)
    assert new.tolist() == [16, 7]
    smla.smla_paged_accept(kv, table, torch.zeros(3, dtype=I32, device=DEV), sl, torch.zeros(2, 4, dtype=I32, device=DEV), new,
                           n_rows=0)
    assert new.tolist() == [20, 7]
    z = torch.zeros(0, dtype=I32, device=DEV)
    smla.smla_paged_accept(kv, z.view(0, 0), torch.zeros(1, dtype=I32, device=DEV), z, z.view(0, 3), z)
    assert np.array_equal(kv.view(-1, REC).cpu().numpy(), c.rec)


# ---- a verification step ----


def step(s, stream=None):
    smla.smla_paged_tree(s["parents"], s["cu"], s["sl"], s["mask"], s["pos"], stream, status=s["status"])
    smla.smla_paged_append(s["lat"], s["rope"], s["kv"], s["table"], s["cu"], s["sl"], s["turns"], stream, q_rope=s["q_rope"],
                           q_out=s["q"][..., 512:], positions=s["pos"], status=s["status"])
    smla.smla_paged_attend_tree(s["q"], s["kv"], s["table"], s["cu"], s["sl"], s["mask"], 1 / 24, None, s["out"], s["lse"],
                                stream, status=s["status"])
    smla.smla_paged_accept(s["kv"], s["table"], s["cu"], s["sl"], s["path"], s["new"], stream, status=s["status"])


def step_state(c, heads, seed):
    lat, rope, q_rope = inputs(c, heads, "bf16", seed)
    lat = torch.randn(c.rows, 512, generator=gen(seed)).to(torch.bfloat16)
    table, cu, sl = c.dev()
    words = -(-max(n for n, _ in c.lens) // 32)
    n_seqs = len(c.lens)
    s = dict(lat=lat.to(DEV), rope=rope.to(DEV), q_rope=q_rope.to(DEV), kv=c.cache(), table=table, cu=cu, sl=sl,
             turns=smla.smla_rotation_turns(FREQ), mask=torch.zeros(c.rows, words, dtype=I32, device=DEV),
             pos=torch.zeros(c.rows, dtype=I32, device=DEV), new=torch.zeros(n_seqs, dtype=I32, device=DEV),
             q=torch.randn(c.rows, heads, 576, generator=gen(seed + 1)).to(torch.bfloat16).to(DEV),
             out=torch.full((c.rows, heads, 512), 7.0, dtype=torch.bfloat16, device=DEV),
             lse=torch.full((c.rows, heads), 7.0, device=DEV), status=torch.zeros(1, dtype=I32, device=DEV),
             parents=torch.zeros(c.rows, dtype=I32, device=DEV), path=torch.full((n_seqs, 6), -1, dtype=I32, device=DEV))
    new_trees(c, s, seed)
    return s


def new_trees(c, s, seed):
    parents, c.sets = random_trees(c, seed)
    s["parents"].copy_(parents)
    c.path = []
    for b, (n, _) in enumerate(c.lens):
        deepest = max((c.sets[int(c.cu[b]) + i] for i in range(n)), key=len, default=set())
        c.path.append(sorted(deepest)[:6])
        s["path"][b] = torch.tensor(c.path[b] + [-1] * (6 - len(c.path[b])), dtype=I32)


def check_step(c, s):
    """Every call's outputs, each against its definition on what the calls before it left."""
    first = {b: k - n for b, (n, k) in enumerate(c.lens)}
    where = {r: (b, p) for r, b, p in c.positions()}
    pos = [first[where[r][0]] + len(c.sets[r]) - 1 for r in range(c.rows)]
    assert s["pos"].tolist() == pos
    assert torch.equal(s["mask"].cpu(), words_of(c.sets, s["mask"].shape[1]))
    check_rotated(s["q"][..., 512:], s["q_rope"].cpu(), pos, "q")
    # the records as appended: undo the moves from the nodes that were not overwritten
    now = s["kv"].reshape(-1, REC).cpu().numpy().copy()
    lat, rope = s["lat"].cpu(), s["rope"].cpu()
    fresh = c.kv_ref.clone()
    smla.smla_paged_append(s["lat"], s["rope"], fresh, s["table"], s["cu"], s["sl"], s["turns"], positions=s["pos"])
    before = c.rec
    c.buf = fresh.view(fresh.shape[0], -1)
    check_append(c, lat, rope, c.buf, before, pos)
    c.rec = fresh.reshape(-1, REC).cpu().numpy()
    tree_check(c, s["q"].cpu(), c.sets, s["out"], s["lse"], 1 / 24, None)
    want = c.rec.copy()
    for b, path in enumerate(c.path):
        for i, j in enumerate(path):
            want[c.slot(b, first[b] + i)] = c.rec[c.slot(b, first[b] + j)]
    assert np.array_equal(now, want)
    assert s["new"].tolist() == [first[b] + len(c.path[b]) for b in range(len(c.lens))]
    c.rec = before
    assert int(s["status"]) == 0


@pytest.mark.parametrize("heads,lens", [(16, [(30, 400), (7, 60), (33, 200)]), (40, [(1, 300), (2, 20), (1, 1)]),
                                        (16, [(1, 300), (2, 20)]), (128, [(12, 90), (5, 5)])])
def test_a_verification_step(heads, lens):
    c = Batch(lens, 16)
    s = step_state(c, heads, 21)
    c.kv_ref = s["kv"].clone()
    step(s)
    check_step(c, s)


def test_steps_in_two_replayed_graphs_and_on_other_streams():
    work = []
    for i in range(2):
        c = Batch([(20, 300), (9, 100)], 16, seed=i)
        s = step_state(c, 16, 30 + i)
        c.kv_ref = s["kv"].clone()
        step(s)  # (loads the kernels)
        torch.cuda.synchronize()
        graph, stream = torch.cuda.CUDAGraph(), torch.cuda.Stream()
        with torch.cuda.graph(graph, stream=stream):
            step(s)
        work.append((c, s, graph, stream))
    for lens in ([(20, 300), (9, 100)], [(12, 200), (17, 97)]):
        for i, (c, s, graph, stream) in enumerate(work):
            c.lens = lens
            c.cu = torch.tensor([0, lens[0][0], sum(n for n, _ in lens)], dtype=I32)
            c.seq_lens = torch.tensor([k for _, k in lens], dtype=I32)
            s["cu"].copy_(c.cu), s["sl"].copy_(c.seq_lens)
            s["kv"].copy_(c.kv_ref)
            s["out"].fill_(7.0)
            new_trees(c, s, 40 + i + lens[0][0])
        torch.cuda.synchronize()
        for c, s, graph, stream in work:
            with torch.cuda.stream(stream):
                graph.replay()
        torch.cuda.synchronize()
        for c, s, *_ in work:
            check_step(c, s)
    # the same calls, one step a stream given by hand
    streams = [torch.cuda.Stream() for _ in work]
    outs = [s["out"].clone() for _, s, *_ in work]
    for c, s, *_ in work:
        s["kv"].copy_(c.kv_ref)
    torch.cuda.synchronize()
    for (c, s, *_), st in zip(work, streams):
        step(s, st)
    torch.cuda.synchronize()
    for (c, s, *_), want in zip(work, outs):
        assert torch.equal(s["out"], want)
        check_step(c, s)


def test_tokens_after_a_step_attend_over_what_was_accepted():
    # the accepted path's records are those that plain decoding writes: the same rows
    # appended one after the other give the same bytes, and the next token the same output
    c = Batch([(12, 100), (8, 50)], 16)
    s = step_state(c, 16, 50)
    plain = s["kv"].clone()
    step(s)
    rows = [int(c.cu[b]) + j for b in range(2) for j in c.path[b]]
    cu = torch.tensor([0, len(c.path[0]), len(rows)], dtype=I32, device=DEV)
    smla.smla_paged_append(s["lat"][rows], s["rope"][rows], plain, s["table"], cu, s["new"], s["turns"])
    a, b = s["kv"].view(-1, REC).cpu().numpy(), plain.view(-1, REC).cpu().numpy()
    for q in range(2):
        kept = [c.slot(q, p) for p in range(int(s["new"][q]))]
        assert np.array_equal(a[kept], b[kept])
    outs = []
    for kv in (s["kv"], plain):
        out, lse = torch.empty(2, 16, 512, dtype=torch.bfloat16, device=DEV), torch.empty(2, 16, device=DEV)
        smla.smla_paged_attend(s["q"][:2], kv, s["table"], torch.tensor([0, 1, 2], dtype=I32, device=DEV), s["new"], 1 / 24,
                               None, out, lse)
        outs.append((out, lse))
    assert torch.equal(outs[0][0], outs[1][0]) and torch.equal(outs[0][1], outs[1][1])


# ---- the two ways into the library ----


def test_calls_through_the_checks_in_python_give_the_same():
    # (a stream given by hand goes through them; without one _smla.so makes the call)
    states = []
    for stream in (None, torch.cuda.current_stream()):
        c = Batch([(20, 300), (9, 100), (0, 7)], 16)
        s = step_state(c, 16, 60)
        step(s, stream)
        lat, rope = torch.empty(c.rows, 512, device=DEV), torch.empty(c.rows, 64, device=DEV)
        smla.smla_paged_read(s["kv"], s["table"], s["cu"], s["sl"], lat, rope, stream)
        smla.smla_paged_write(lat, rope, s["kv"], s["table"], s["cu"], s["sl"], stream)
        out, lse = torch.empty_like(s["out"]), torch.empty_like(s["lse"])
        smla.smla_paged_attend(s["q"], s["kv"], s["table"], s["cu"], s["sl"], 1 / 24, None, out, lse, stream)
        torch.cuda.synchronize()
        states.append([s[k] for k in ("mask", "pos", "q", "kv", "out", "lse", "new")] + [lat, rope, out, lse])
    for a, b in zip(*states):
        assert torch.equal(a, b)


def test_well_formed_calls_are_taken_and_others_are_not():
    native = smla._native
    c = Batch([(5, 40), (3, 9)], 16)
    s = step_state(c, 4, 61)
    batch = (s["kv"], s["table"], s["cu"], s["sl"])
    tree = (s["parents"], s["cu"], s["sl"], s["mask"], s["pos"])
    append = (*batch, s["lat"], s["rope"], s["turns"], s["q_rope"], s["q"][..., 512:], s["pos"], True, 1.0)
    attend = (*batch, s["q"], 1 / 24, None, s["out"], s["lse"], True)
    calls = [(native.write, (*batch, s["lat"], s["rope"])), (native.read, (*batch, s["lat"].clone(), s["rope"].clone())),
             (native.append, append), (native.tree, tree), (native.accept, (*batch, s["path"], s["new"], c.rows))]
    for call, args in calls:
        assert call(*args, None, None) is True and call(*args, None, s["status"]) is True
        assert call(*args, torch.cuda.current_stream(), None) is False  # a stream by hand
        assert call(*args, None, s["lse"]) is False                     # a status that is none
        for i, x in enumerate(args):
            if torch.is_tensor(x):
                assert call(*args[:i], x.cpu(), *args[i + 1:], None, None) is False
                assert call(*args[:i], x.double(), *args[i + 1:], None, None) is False
                wide = torch.zeros(*x.shape[:-1], 2 * x.shape[-1], dtype=x.dtype, device=DEV)[..., ::2]
                # (the stride of a dimension of one element, the mask's words here, says nothing)
                assert call(*args[:i], wide, *args[i + 1:], None, None) is (x.shape[-1] == 1)
    for mask in (None, s["mask"]):
        assert native.attend(*attend, None, None, None, mask) is True
        assert native.attend(*attend, torch.cuda.current_stream(), None, None, mask) is False
        for i, x in enumerate(attend):
            if torch.is_tensor(x):
                assert native.attend(*attend[:i], x.cpu(), *attend[i + 1:], None, None, None, mask) is False
                assert native.attend(*attend[:i], x.double(), *attend[i + 1:], None, None, None, mask) is False
    assert native.attend(*attend, None, None, s["lse"].t(), None) is False  # a workspace that is not contiguous
    assert native.attend(*attend, None, None, torch.zeros(256, dtype=torch.uint8, device=DEV), None) is False  # too small
    assert native.attend(*batch, s["q"], 1e40, None, s["out"], s["lse"], True, None, None, None, None) is False
    torch.cuda.synchronize()


def test_a_captured_step_behind_copies_and_joined_streams():
    # what is before a call in a graph may be a copy, or the join of two streams
    c = Batch([(20, 300), (9, 100)], 16)
    s = step_state(c, 16, 70)
    c.kv_ref = s["kv"].clone()
    step(s)
    torch.cuda.synchronize()
    pinned = {k: s[k].cpu().pin_memory() for k in ("parents", "path", "lat", "rope", "sl")}
    side, stream, graph = torch.cuda.Stream(), torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        s["parents"].copy_(pinned["parents"], non_blocking=True)
        smla.smla_paged_tree(s["parents"], s["cu"], s["sl"], s["mask"], s["pos"], status=s["status"])
        side.wait_stream(stream)
        with torch.cuda.stream(side):
            s["lat"].copy_(pinned["lat"], non_blocking=True)
            s["rope"].copy_(pinned["rope"], non_blocking=True)
        s["kv"].copy_(c.kv_ref)
        stream.wait_stream(side)
        smla.smla_paged_append(s["lat"], s["rope"], s["kv"], s["table"], s["cu"], s["sl"], s["turns"], q_rope=s["q_rope"],
                               q_out=s["q"][..., 512:], positions=s["pos"], status=s["status"])
        s["out"].fill_(7.0)
        smla.smla_paged_attend_tree(s["q"], s["kv"], s["table"], s["cu"], s["sl"], s["mask"], 1 / 24, None, s["out"], s["lse"],
                                    status=s["status"])
        s["path"].copy_(pinned["path"], non_blocking=True)
        smla.smla_paged_accept(s["kv"], s["table"], s["cu"], s["sl"], s["path"], s["new"], status=s["status"])
    for seed in (70, 71):
        new_trees(c, s, seed)
        pinned["parents"].copy_(s["parents"].cpu())
        pinned["path"].copy_(s["path"].cpu())
        for k in ("mask", "pos", "parents", "path", "lat", "rope", "lse", "new"):
            s[k].fill_(0)
        torch.cuda.synchronize()
        for _ in range(2):
            graph.replay()
        torch.cuda.synchronize()
        check_step(c, s)


@pytest.mark.parametrize("kernel", ["few", "narrow32", "narrow64", "pair", "pair_128"])
def test_many_launches_at_once_give_the_same_bits(kernel):
    # cold and warm caches, three streams, two batches of unlike shapes beside each other
    heads, lens = KERNELS[kernel]
    work = []
    for seed, part in ((1, lens), (2, lens[:3] + [(3, 1500)] + (EMPTY if (0, 0) in lens else []))):
        c = Batch(part, 16, seed=seed)
        _, sets = random_trees(c, seed)
        mask = words_of(sets, -(-max(n for n, _ in part) // 32)).to(DEV)
        q, _, out, lse, _ = tree_attend(c, heads, mask.cpu())
        work.append((c, q.to(DEV), mask, c.cache(), c.dev(), out, lse))
    flush = torch.empty(256 << 20, dtype=torch.uint8, device=DEV)
    streams = [torch.cuda.Stream() for _ in range(3)]
    torch.cuda.synchronize()
    got = []
    for i in range(18):
        c, q, mask, kv, tabs, out, lse = work[i % 2]
        with torch.cuda.stream(streams[i % 3]):
            if i % 4 == 0:
                flush.fill_(i)
            o, z = torch.full_like(out, 7.0), torch.full_like(lse, 7.0)
            smla.smla_paged_attend_tree(q, kv, *tabs, mask, 1 / 24, None, o, z)
            got.append((o, z, out, lse))
    torch.cuda.synchronize()
    for o, z, out, lse in got:
        assert torch.equal(o, out) and torch.equal(z, lse)


def test_calls_without_pages_or_table():
    c = Batch([(3, 9)], 16)
    s = step_state(c, 16, 80)
    for kv, table in ((torch.empty(0, 16, REC, dtype=torch.uint8, device=DEV), torch.zeros(1, 3, dtype=I32, device=DEV)),
                      (torch.zeros(2, 16, REC, dtype=torch.uint8, device=DEV), torch.zeros(1, 0, dtype=I32, device=DEV))):
        s["kv"], s["table"] = kv, table
        s["status"].zero_()
        s["path"][0] = torch.tensor([0, 2, -1, -1, -1, -1], dtype=I32)
        step(s)
        assert int(s["status"]) == smla.STATUS_INDEX_OOB
        pos = [6 + len(x) - 1 for x in c.sets]
        assert s["pos"].tolist() == pos and s["new"].tolist() == [8]
        check_rotated(s["q"][..., 512:], s["q_rope"].cpu(), pos)
        assert (s["out"] == 0).all() and torch.isneginf(s["lse"]).all() and (s["kv"] == 0).all()


def test_lengths_and_boundaries_that_say_nothing_sensible():
    # negative lengths count as zero, boundaries are clamped or name rows twice: every access stays
    # inside the tensors, and rows of no sequence stay as they are
    c = Batch([(4, 40), (3, 30), (2, 2)], 16, behind=4)
    s = step_state(c, 16, 81)
    for cu, lens in (([0, 4, 7, 9], [-5, -2 ** 31, 0]), ([-7, 4, 4, 1000], [40, 30, 2]), ([0, 6, 3, 9], [40, 30, 2]),
                     ([13, 13, 0, 0], [40, 30, 2]), ([5, 5, 5, 5], [2 ** 31 - 1] * 3), ([0, 4, 7, 9], [2 ** 31 - 1, 7, 2 ** 30])):
        s["cu"].copy_(torch.tensor(cu, dtype=I32))
        s["sl"].copy_(torch.tensor(lens, dtype=I32))
        for k in ("mask", "pos"):
            s[k].fill_(0)
        step(s)
        step(s, torch.cuda.current_stream())
    torch.cuda.synchronize()
    s["cu"].copy_(torch.tensor([5, 5, 5, 5], dtype=I32))
    s["out"].fill_(7.0), s["mask"].fill_(7), s["pos"].fill_(7)
    before = s["kv"].clone()
    step(s)
    assert (s["out"] == 7.0).all() and (s["mask"] == 7).all() and (s["pos"] == 7).all() and torch.equal(s["kv"], before)

"""Cases of the operators of a drafted-token tree over the paged fp8_ds_mla cache:
the tree's masks and positions, new records with their position rotation,
attention of the tree's nodes, and the accepted path's records moved up.

The cache is uint8 [n_pages, page_size, 656] (a record: 512 E4M3 latent values,
four f32 power-of-two scales of 128 values each, 64 bf16 rope values).  Sequence
b owns the token rows cu_rows[b] .. cu_rows[b + 1], its last row sits at position
seq_lens[b] - 1, and position p lives in page block_table[b, p // page_size] at
offset p % page_size.  The rows of a sequence are the nodes of its tree, a parent
before its children; `past` is the position of the first one.

  tree    parents [rows] (a node's index, -1: a root) -> mask int32 [rows, words]
          (bit j % 32 of word j / 32: node j is the row itself or an ancestor),
          positions [rows] = past + depth
  append  latent [rows, 512], rope [rows, 64] -> records, the rope rotated by its
          position; q_rope [rows, heads, 64] rotated into q (bf16)
  attend  q [rows, heads, 576] -> out [rows, heads, 512], lse [rows, heads] over the
          history and the nodes in the row's mask
  accept  path [seqs, width] (nodes of the accepted path, -1 behind it): records of
          the path's nodes to positions past, past + 1, ..., and the new lengths
  step    the four together, as a verification step calls them
"""

import math
import random

import torch

own = False

LATENT, ROPE, QK, RECORD = 512, 64, 576, 656
SM_SCALE = 1.0 / math.sqrt(QK)
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
SIZES = {"bf16": 2, "f16": 2, "f32": 4}


def _case(name, op, seqs, rows, ctx, *, heads=0, page=64, ragged=True, depth=8, sink=False, dtype="bf16",
          interleaved=True, tree=True):
    return {"name": name, "op": op, "seqs": seqs, "rows": rows, "ctx": ctx, "heads": heads, "page": page,
            "ragged": ragged, "depth": depth, "sink": sink, "dtype": dtype, "interleaved": interleaved, "tree": tree}


def listed():
    return [
        # a serving batch's trees of 60 drafted tokens: masks and positions before the step
        _case("tree_64x60", "tree", 64, 60, 2000, ragged=False),
        # few wide and deep trees of odd sizes
        _case("tree_7x500", "tree", 7, 500, 1000, depth=40),
        # a serving step's new tokens, one a user, with their queries
        _case("append_step_64x16", "append", 64, 1, 2048, heads=16, tree=False),
        # the rows of drafted trees, rotated by depth, many heads
        _case("append_tree_32x60x128", "append", 32, 60, 2000, heads=128, page=16),
        # chunks of prompts written at once, from f32 activations, pairs of halves, odd pages
        _case("append_chunk_8x2048x16_f32", "append", 8, 2048, 1000, heads=16, page=48, dtype="f32",
              interleaved=False, tree=False),
        # one user's tree over a short history: latency of the call
        _case("attend_tree_1x60x16_c500", "attend", 1, 60, 500, heads=16, ragged=False),
        # a batch of small trees over long histories
        _case("attend_tree_64x4x16_c4096", "attend", 64, 4, 4096, heads=16, depth=3, sink=True),
        # a batch of full trees, small pages
        _case("attend_tree_32x60x64_c2000", "attend", 32, 60, 2000, heads=64, page=16, sink=True),
        # wide trees over long histories: the largest case
        _case("attend_tree_4x250x64_c16384", "attend", 4, 250, 16384, heads=64, ragged=False, depth=12),
        # the tree's records written, then the accepted path moved up
        _case("accept_64x60", "accept", 64, 60, 2000),
        # long accepted paths in odd pages
        _case("accept_7x500", "accept", 7, 500, 1000, page=48, depth=120),
        # a verification step from the parents to the new lengths
        _case("step_16x30x16_c4000", "step", 16, 30, 4000, heads=16, sink=True),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["tree", "append", "attend", "attend", "accept", "step"])
    seqs = _log_int(rng, 1, 64)
    common = {"page": rng.choice([1, 16, 48, 64, 100, 128]), "ragged": rng.random() < 0.75,
              "interleaved": rng.random() < 0.5, "sink": rng.random() < 0.5}
    if op in ("tree", "accept"):
        return dict(_case("", op, seqs, _log_int(rng, 1, 500), _log_int(rng, 1, 2000), **common,
                          depth=_log_int(rng, 1, 120)), name="")
    heads = rng.choice([1, 7, 16, 40, 64, 128])
    if op == "append":
        tree = rng.random() < 0.5
        rows = _log_int(rng, 1, 500 if tree else 2048)
        rows = max(1, min(rows, 262_144 // (seqs * heads)))
        return _case("", op, seqs, rows, _log_int(rng, 1, 4096), heads=heads, **common, tree=tree,
                     dtype=rng.choice(["bf16", "f16", "f32"]))
    rows, ctx = _log_int(rng, 1, 250), _log_int(rng, 1, 16384)
    ctx = max(1, min(ctx, 260_000 // seqs))
    # no more scores than the largest listed case has
    rows = max(1, min(rows, int(1.0e9 / (seqs * heads * (ctx + rows))), 122_880 // (seqs * heads)))
    return _case("", op, seqs, rows, ctx, heads=heads, **common, depth=_log_int(rng, 1, 20))


def _lengths(case):
    """(token rows, sequence length) of each sequence: sizes of the case, not of the seed."""
    r = random.Random("%(seqs)d-%(rows)d-%(ctx)d-%(page)d" % case)
    got = []
    for _ in range(case["seqs"]):
        n, c = case["rows"], case["ctx"]
        if case["ragged"]:
            n, c = r.randint((n + 3) // 4, n), r.randint(c // 2, c)
        got.append((n, n + c))
    return got


def _words(case):
    return -(-case["rows"] // 32)


def work(case):
    lens, op = _lengths(case), case["op"]
    rows, keys, heads, e = sum(n for n, _ in lens), sum(s for _, s in lens), case["heads"], SIZES[case["dtype"]]
    # (a path may hold every depth of its tree; half of it on average)
    moved = sum(min(n, case["depth"]) for n, _ in lens) // 2
    per = {"tree": rows * (8 + 4 * _words(case)),
           "append": rows * (QK * e + RECORD + heads * ROPE * (e + 2)) + (4 * rows if case["tree"] else 0),
           "attend": keys * RECORD + rows * (heads * (2 * QK + 2 * LATENT + 4) + 4 * _words(case)),
           "accept": rows * (QK * e + RECORD) + moved * 2 * RECORD}
    # each row sees its history and at most `depth` nodes
    seen = sum(n * (s - n + min(n, (case["depth"] + 1) // 2)) for n, s in lens)
    flops = {"tree": 0, "append": rows * (1 + heads) * ROPE * 3, "attend": 2 * seen * heads * (QK + LATENT),
             "accept": rows * ROPE * 3}
    if op == "step":
        return {"bytes": per["tree"] + per["append"] + per["attend"] + moved * 2 * RECORD,
                "flops": flops["append"] + flops["attend"]}
    return {"bytes": per[op], "flops": flops[op]}


def _trees(lens, depth, rng):
    """Parents of trees in the order of their nodes, no deeper than `depth`, and an
    accepted path of each: from a root towards a deep node, seldom all the way."""
    parents, paths = [], []
    for n, _ in lens:
        tree, level = [], []
        for i in range(n):
            # a node hangs on a late one more often than on an early one, in deep trees most often
            p = min(i, int((i + 1) * rng.random() ** (8 / (8 + depth)))) - 1
            if p >= 0 and level[p] + 1 >= depth:
                p = -1
            tree.append(p)
            level.append(0 if p < 0 else level[p] + 1)
        at, path = max((rng.randrange(n) for _ in range(4)), key=lambda i: level[i]), []
        while at >= 0:
            path.insert(0, at)
            at = tree[at]
        parents.append(tree)
        paths.append(path[:rng.randint(1, len(path))] if rng.random() < 0.95 else [])
    return parents, paths


def _records(latent, rope):
    """Records [n, 656] of latent [n, 512] and rope [n, 64]: per 128 values the scale
    pow2ceil(max(amax, 1e-4) / 448), the values over it as E4M3, rope as bf16."""
    n = latent.shape[0]
    blocks = latent.double().view(n, 4, 128)
    man, exp = torch.frexp(blocks.abs().amax(2).clamp_min(1e-4) / 448.0)
    scale = torch.ldexp(torch.ones_like(man), exp - (man == 0.5).to(exp.dtype))
    code = (blocks / scale[..., None]).float().clamp(-448.0, 448.0).to(torch.float8_e4m3fn)
    return torch.cat([code.view(torch.uint8).view(n, LATENT), scale.float().view(torch.uint8).view(n, 16),
                      rope.to(torch.bfloat16).contiguous().view(torch.uint8).view(n, 128)], 1)


def prepare(case, seed):
    lens, op = _lengths(case), case["op"]
    dev, page, dtype, heads = "cuda", case["page"], TYPES[case["dtype"]], case["heads"]
    g = torch.Generator(device=dev)
    g.manual_seed(int(seed) * 1_000_003 + 29)
    rows = sum(n for n, _ in lens)
    pages = [-(-s // page) for _, s in lens]
    n_pages = sum(pages) + 3
    s = {"op": op, "lens": lens, "tree": case["tree"], "interleaved": case["interleaved"]}

    def i32(x):
        return torch.tensor(x, dtype=torch.int32, device=dev)

    def normal(*shape, std=1.0):
        return torch.randn(*shape, generator=g, device=dev) * std

    order = torch.randperm(n_pages, generator=g, device=dev).tolist()
    table, at = [], 0
    for k in pages:
        table.append(order[at:at + k] + [-1] * (max(pages) - k))
        at += k
    s["table"] = i32(table)
    ends = [0]
    for n, _ in lens:
        ends.append(ends[-1] + n)
    s["cu"] = i32(ends)
    s["seq_lens"] = i32([k for _, k in lens])
    past = [k - n for n, k in lens]
    if case["tree"]:
        parents, paths = _trees(lens, case["depth"], random.Random(int(seed) * 7919 + 11))
        s["depth"] = case["depth"]
        s["parents"] = i32([p for t in parents for p in t])
        s["mask"] = torch.zeros(rows, _words(case), dtype=torch.int32, device=dev)
        s["positions"] = torch.zeros(rows, dtype=torch.int32, device=dev)
        if op != "tree" and op != "step":  # what the tree's call has left
            mask, depth = _plain_tree(s)
            s["mask"].copy_(mask)
            s["positions"].copy_(depth)
        s["path"] = i32([p + [-1] * (case["depth"] - len(p)) for p in paths])
        s["new_lens"] = torch.zeros(len(lens), dtype=torch.int32, device=dev)
    if op == "tree":
        return s
    cache = torch.full((n_pages * page, RECORD), 0x11, dtype=torch.uint8, device=dev)
    if op in ("attend", "step"):
        for lo in range(0, cache.shape[0], 65536):
            part = cache[lo:lo + 65536]
            part.copy_(_records(normal(part.shape[0], LATENT, std=math.sqrt(2.0)), normal(part.shape[0], ROPE)))
    s["cache"] = cache.view(n_pages, page, RECORD)
    if op != "attend":
        # the new rows as a projection leaves them: latent and rope side by side
        wide = torch.cat([normal(rows, LATENT, std=math.sqrt(2.0)), normal(rows, ROPE)], 1).to(dtype)
        s["latent"], s["rope"] = wide[:, :LATENT], wide[:, LATENT:]
        s["inv_freq"] = torch.tensor([10000.0 ** (-i / 32) for i in range(32)], dtype=torch.float64, device=dev)
        if own:
            import sparse_mla_decode_csr_gb300 as smla
            s["turns"] = smla.smla_rotation_turns(s["inv_freq"])
    if op in ("append", "step"):
        s["q_rope"] = normal(rows, heads, ROPE).to(dtype)
    if op != "accept":
        s["q"] = normal(rows, heads, QK).to(torch.bfloat16)
        s["q_out"] = s["q"][..., LATENT:]
    if op in ("attend", "step"):
        s["sink"] = normal(heads) if case["sink"] else None
        s["out"] = torch.empty(rows, heads, LATENT, dtype=torch.bfloat16, device=dev)
        s["lse"] = torch.empty(rows, heads, dtype=torch.float32, device=dev)
    return s


def _fields(cache):
    """The cache's values: E4M3 latent, f32 scales, bf16 rope (views)."""
    return {"latent": cache[..., :512].view(torch.float8_e4m3fn), "scale": cache[..., 512:528].view(torch.float32),
            "rope": cache[..., 528:].view(torch.bfloat16)}


# ---- the plain forms ----


def _row_sequences(s):
    """Sequence, node index and slot position of every token row."""
    cu = s["cu"].long()
    row = torch.arange(sum(n for n, _ in s["lens"]), device=cu.device)
    seq = torch.searchsorted(cu, row, right=True) - 1
    return seq, row - cu[seq], s["seq_lens"].long()[seq] - cu[seq + 1] + row


def _slots(s, seq, position):
    """Global slot (page * page_size + offset) of positions."""
    page = s["cache"].shape[1]
    return s["table"].long()[seq, position // page] * page + position % page


def _plain_tree(s):
    seq, node, pos = _row_sequences(s)
    first = s["cu"].long()[seq]
    words = s["mask"].shape[1]
    bits = torch.zeros(node.shape[0], words * 32, dtype=torch.bool, device=node.device)
    bits.scatter_(1, node[:, None], True)
    at, depth = s["parents"].long(), torch.zeros_like(node)
    for _ in range(s["depth"] - 1):
        up = at >= 0
        depth += up
        # (a row without a next ancestor sets its own bit again)
        bits.scatter_(1, torch.where(up, at, node)[:, None], True)
        at = torch.where(up, s["parents"].long()[first + at.clamp_min(0)], at)
    weight = torch.ones(32, dtype=torch.int64, device=node.device) << torch.arange(32, device=node.device)
    mask = (bits.view(-1, words, 32) * weight).sum(2)
    mask = torch.where(mask >= 1 << 31, mask - (1 << 32), mask).to(torch.int32)
    return mask, (pos - node + depth).to(torch.int32)


def _rotated(s, x, position):
    """x [rows, ..., 64] rotated by its row's position, in f32 (angles in f64)."""
    angle = position.double()[:, None] * s["inv_freq"]
    shape = (x.shape[0],) + (1,) * (x.dim() - 2) + (32,)
    c, d = angle.cos().float().view(shape), angle.sin().float().view(shape)
    x = x.float()
    if s["interleaved"]:
        a, b = x[..., 0::2], x[..., 1::2]
        return torch.stack([a * c - b * d, a * d + b * c], -1).flatten(-2)
    a, b = x[..., :32], x[..., 32:]
    return torch.cat([a * c - b * d, a * d + b * c], -1)


def _plain_append(s):
    seq, _, pos = _row_sequences(s)
    at = s["positions"] if s["tree"] else pos
    s["cache"].view(-1, RECORD)[_slots(s, seq, pos)] = _records(s["latent"], _rotated(s, s["rope"], at))
    if "q_rope" in s:
        s["q_out"].copy_(_rotated(s, s["q_rope"], at))


def _plain_accept(s):
    seqs, width = s["path"].shape
    path = s["path"].long()
    past = s["seq_lens"].long() - (s["cu"].long()[1:] - s["cu"].long()[:-1])
    some = path >= 0
    seq = torch.arange(seqs, device=path.device)[:, None].expand(-1, width)
    source = _slots(s, seq, past[:, None] + path.clamp_min(0))
    step = torch.arange(width, device=path.device)
    # (a step behind the path's end stays on its first slot, which it does not write)
    target = _slots(s, seq, past[:, None] + torch.where(some, step, torch.zeros_like(path)))
    flat = s["cache"].view(-1, RECORD)
    flat[target[some]] = flat[source[some]]
    s["new_lens"].copy_(past + some.sum(1))


def _values(records):
    """f32 latent and rope of records [..., 656]."""
    f = _fields(records)
    lat = f["latent"].float().view(*records.shape[:-1], 4, 128) * f["scale"][..., None]
    return lat.flatten(-2), f["rope"].float()


def _plain_attend(s):
    cache, table, cu = s["cache"], s["table"], s["cu"].long()
    page, dev = cache.shape[1], cache.device
    n_seqs, heads = table.shape[0], s["q"].shape[1]
    longest, most = max(k for _, k in s["lens"]), max(n for n, _ in s["lens"])
    key = torch.arange(longest, device=dev)
    slot = table.long()[:, key // page].clamp_min(0) * page + key % page  # [seqs, keys]
    lat, rope = _values(cache.view(-1, RECORD)[slot])
    k = torch.cat([lat, rope], -1)
    # token rows padded to the widest tree
    row = cu[:-1, None] + torch.arange(most, device=dev)
    real = row < cu[1:, None]
    row = row.clamp_max(cu[-1] - 1)
    q = s["q"].float()[row]  # [seqs, most, heads, 576]
    x = torch.matmul(q.view(n_seqs, most * heads, QK), k.transpose(1, 2)).mul_(SM_SCALE)
    # key t is seen before the tree, or as a node in the row's mask
    past = (s["seq_lens"].long() - (cu[1:] - cu[:-1]))[:, None]
    node = key - past  # [seqs, keys]
    inside = (node >= 0) & (key < s["seq_lens"].long()[:, None])
    at = node.clamp(0, s["mask"].shape[1] * 32 - 1)[:, None, :].expand(-1, most, -1)
    bit = (torch.gather(s["mask"].long()[row], 2, at // 32) >> (at % 32)) & 1
    seen = (node < 0)[:, None] | (inside[:, None] & (bit != 0))
    del at, bit
    x.view(n_seqs, most, heads, longest).masked_fill_(~seen[:, :, None], -math.inf)
    m = x.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, torch.zeros_like(m), m)
    e = x.sub_(m).exp_()
    total = e.sum(-1, keepdim=True)
    lse = (m + total.log())[..., 0].view(n_seqs, most, heads)
    if s["sink"] is not None:
        total = total + (s["sink"].repeat(most)[None, :, None] - m).exp()
    out = (torch.matmul(e, lat) / total).view(n_seqs, most, heads, LATENT)
    s["out"].copy_(out[real])
    s["lse"].copy_(lse[real])


def _own_call(s, op):
    import sparse_mla_decode_csr_gb300 as smla
    batch = (s["table"], s["cu"], s["seq_lens"])
    if op == "tree":
        smla.smla_paged_tree(s["parents"], s["cu"], s["seq_lens"], s["mask"], s["positions"])
    elif op == "append":
        smla.smla_paged_append(s["latent"], s["rope"], s["cache"], *batch, s["turns"], q_rope=s.get("q_rope"),
                               q_out=s.get("q_out"), positions=s["positions"] if s["tree"] else None,
                               interleaved=s["interleaved"])
    elif op == "attend":
        smla.smla_paged_attend_tree(s["q"], s["cache"], *batch, s["mask"], SM_SCALE, s["sink"], s["out"], s["lse"])
    else:
        smla.smla_paged_accept(s["cache"], *batch, s["path"], s["new_lens"])


def _plain_call(s, op):
    if op == "tree":
        mask, positions = _plain_tree(s)
        s["mask"].copy_(mask)
        s["positions"].copy_(positions)
    else:
        {"append": _plain_append, "attend": _plain_attend, "accept": _plain_accept}[op](s)


# the calls of a case: the records are there before a path of them is accepted
CALLS = {"tree": ["tree"], "append": ["append"], "attend": ["attend"], "accept": ["append", "accept"],
         "step": ["tree", "append", "attend", "accept"]}
OUTPUTS = {"tree": ["mask", "positions"], "append": ["q_out"], "attend": ["out", "lse"], "accept": ["new_lens"]}


def run(s):
    calls = CALLS[s["op"]]
    for op in calls:
        (_own_call if own else _plain_call)(s, op)
    got = {name: s[name] for op in calls for name in OUTPUTS[op] if name in s}
    if "append" in calls:
        got.update(_fields(s["cache"]))
    return got


# ---- the definition in 64 bits, sequence by sequence ----


def _e4m3_values(dev):
    table = []
    for code in range(256):
        e, m = code >> 3 & 15, code & 7
        v = math.nan if code & 127 == 127 else m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10)
        table.append(-v if code > 127 else v)
    return torch.tensor(table, dtype=torch.float64, device=dev)


def _round_e4m3(x):
    """x in f64 to the nearest E4M3 value, ties to even, saturating."""
    _, e = torch.frexp(x)
    step = torch.exp2((e - 4).clamp_min(-9).double())
    return ((x / step).round() * step).clamp(-448.0, 448.0)


def _rotate64(x, angle, interleaved):
    """x [..., 64] in f64 times e^(i angle [32]), as complex numbers."""
    z = torch.view_as_complex(x.reshape(*x.shape[:-1], 32, 2).contiguous()) if interleaved else \
        torch.complex(x[..., :32].contiguous(), x[..., 32:].contiguous())
    z = z * torch.polar(torch.ones_like(angle), angle)
    return torch.view_as_real(z).flatten(-2) if interleaved else torch.cat([z.real, z.imag], -1)


def exact(case, seed):
    s = prepare(case, seed)
    op, dev, lens, cu = case["op"], "cuda", _lengths(case), s["cu"].tolist()
    calls, got = CALLS[op], {}
    if work(case)["flops"] > 8e12:
        return None
    ancestors = None
    if case["tree"]:
        parents, ancestors, mask, positions = s["parents"].tolist(), [], [], []
        for b, (n, length) in enumerate(lens):
            mine = []
            for i in range(n):
                p = parents[cu[b] + i]
                mine.append((mine[p] if p >= 0 else []) + [i])
                word = [0] * _words(case)
                for j in mine[i]:
                    word[j // 32] |= 1 << (j % 32)
                mask.append([w - (1 << 32) if w >> 31 else w for w in word])
                positions.append(length - n + len(mine[i]) - 1)
            ancestors.append(mine)
        if "tree" in calls:
            got["mask"] = torch.tensor(mask, device=dev)
            got["positions"] = torch.tensor(positions, device=dev)
    if op == "tree":
        return got
    page, table = case["page"], s["table"].tolist()
    slots = [torch.tensor([table[b][p // page] * page + p % page for p in range(k)], device=dev)
             for b, (_, k) in enumerate(lens)]
    # the cache's values in f64
    flat = s["cache"].view(-1, RECORD)
    code = _e4m3_values(dev)[flat[:, :LATENT].long()]
    scale = flat[:, 512:528].contiguous().view(torch.float32).double()
    rope = flat[:, 528:].contiguous().view(torch.bfloat16).double()
    q = s["q"].double() if "q" in s else None
    if "append" in calls:
        at = torch.cat([slots[b][k - n:] for b, (n, k) in enumerate(lens)])
        where = positions if case["tree"] else [k - n + i for n, k in lens for i in range(n)]
        angle = torch.tensor(where, dtype=torch.float64, device=dev)[:, None] * s["inv_freq"]
        x = s["latent"].double().reshape(-1, 4, 128)
        y = x.abs().amax(2).clamp_min(1e-4) / 448.0
        new = torch.exp2(torch.floor(torch.log2(y)) - 1)  # below y; doubled until it is not
        for _ in range(3):
            new = torch.where(new < y, 2 * new, new)
        code[at] = _round_e4m3(x / new[..., None]).flatten(1)
        scale[at] = new
        rope[at] = _rotate64(s["rope"].double(), angle, case["interleaved"])
        if "q_rope" in s:
            got["q_out"] = _rotate64(s["q_rope"].double(), angle[:, None], case["interleaved"])
            q[..., LATENT:] = got["q_out"].to(torch.bfloat16).double()
    if "attend" in calls:
        heads = case["heads"]
        got["out"] = torch.empty(cu[-1], heads, LATENT, dtype=torch.float64, device=dev)
        got["lse"] = torch.empty(cu[-1], heads, dtype=torch.float64, device=dev)
        for b, (n, length) in enumerate(lens):
            lat = code[slots[b]] * scale[slots[b]].repeat_interleave(128, 1)
            k = torch.cat([lat, rope[slots[b]].to(torch.bfloat16).double()], 1)
            sees = torch.zeros(n, length, dtype=torch.bool, device=dev)
            sees[:, :length - n] = True
            pairs = [(i, length - n + j) for i in range(n) for j in ancestors[b][i]]
            i, j = torch.tensor(pairs, device=dev).t()
            sees[i, j] = True
            few = max(1, int(2.5e8 / (heads * length)))
            for lo in range(0, n, few):
                hi = min(n, lo + few)
                z = q[cu[b] + lo:cu[b] + hi].reshape(-1, QK) @ k.t() * SM_SCALE
                z = z.view(hi - lo, heads, length).masked_fill(~sees[lo:hi, None], -math.inf)
                norm = torch.logsumexp(z, -1)
                got["lse"][cu[b] + lo:cu[b] + hi] = norm
                if s["sink"] is not None:
                    norm = torch.logaddexp(norm, s["sink"].double())
                p = torch.exp(z - norm[..., None])
                got["out"][cu[b] + lo:cu[b] + hi] = (p.view(-1, length) @ lat).view(hi - lo, heads, LATENT)
    if "accept" in calls:
        got["new_lens"] = torch.zeros(len(lens), dtype=torch.int64, device=dev)
        before = [code.clone(), scale.clone(), rope.clone()]
        for b, path in enumerate(s["path"].tolist()):
            n, length = lens[b]
            path = [i for i in path if i >= 0]
            got["new_lens"][b] = length - n + len(path)
            for i, j in enumerate(path):
                for now, then in zip((code, scale, rope), before):
                    now[slots[b][length - n + i]] = then[slots[b][length - n + j]]
    if "append" in calls:
        shape = s["cache"].shape[:2]
        got.update({"latent": code.view(*shape, LATENT), "scale": scale.view(*shape, 4), "rope": rope.view(*shape, ROPE)})
    return got

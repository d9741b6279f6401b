"""Cases of the paged-cache operators: records written into a paged fp8_ds_mla
cache, read back from it, and attention of new tokens over it.

All three share one description of a batch.  The cache is uint8
[n_pages, page_size, 656] (a record: 512 E4M3 latent values, four f32
power-of-two scales of 128 values each, 64 bf16 rope values).  Sequence b owns
the token rows cu_rows[b] .. cu_rows[b + 1] of the token tensors, and its last
row sits at position seq_lens[b] - 1; position p lives in page
block_table[b, p // page_size] at offset p % page_size.

  write   latent [rows, 512], rope [rows, 64] -> records of those positions
  read    records of those positions -> latent, rope in the outputs' type
  attend  q [rows, heads, 576] -> out [rows, heads, 512], lse [rows, heads]:
          softmax attention of a row at position p over positions 0 .. p
          (causal) or over the whole sequence, keys = 576 dims, values = the
          512 latent dims, an optional per-head sink in the denominator
"""

import math
import random

import torch

own = False

LATENT, ROPE, QK, RECORD = 512, 64, 576, 656
SM_SCALE = 1.0 / math.sqrt(QK)
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
SIZES = {"bf16": 2, "f16": 2, "f32": 4}


def _attend(name, seqs, rows, ctx, heads, page, ragged, sink, causal=True):
    return {"name": name, "op": "attend", "seqs": seqs, "rows": rows, "ctx": ctx, "heads": heads,
            "page": page, "ragged": ragged, "sink": sink, "causal": causal, "dtype": "bf16"}


def _copy(name, op, seqs, rows, ctx, page, ragged, dtype):
    return {"name": name, "op": op, "seqs": seqs, "rows": rows, "ctx": ctx, "page": page,
            "ragged": ragged, "dtype": dtype}


def listed():
    return [
        # one user, one token, a short history: latency of the call
        _attend("attend_step_1x16_c500", 1, 1, 500, 16, 64, False, False),
        # a serving step: 64 users, one token each, histories of up to 4096
        _attend("attend_step_64x16_c4096", 64, 1, 4096, 16, 64, True, True),
        # few users with long histories: the keys' axis is split
        _attend("attend_step_4x64_c16384", 4, 1, 16384, 64, 64, True, True),
        # drafted tokens being verified: five rows a user, small pages
        _attend("attend_draft_32x5x64_c2000", 32, 5, 2000, 64, 16, True, True),
        # mixed short prompts with odd lengths and odd pages
        _attend("attend_chunk_7x300x16_c5000", 7, 300, 5000, 16, 48, True, True),
        # a long prompt's chunk: the largest case
        _attend("attend_chunk_1x2048x64_c8192", 1, 2048, 8192, 64, 64, False, False),
        # the step's new records: one row a user
        _copy("write_step_64", "write", 64, 1, 2048, 64, True, "bf16"),
        # a chunk of prompts written at once
        _copy("write_chunk_8x2048", "write", 8, 2048, 1000, 64, True, "bf16"),
        # the same from f32 activations, odd pages
        _copy("write_chunk_3x5000_f32", "write", 3, 5000, 0, 48, True, "f32"),
        # a short prefix read back for an up-projection
        _copy("read_1x512", "read", 1, 512, 0, 64, False, "bf16"),
        # the histories of a whole batch read back
        _copy("read_32x4096", "read", 32, 4096, 0, 64, True, "bf16"),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["attend", "attend", "attend", "write", "read"])
    page = rng.choice([1, 16, 48, 64, 100, 128])
    ragged = rng.random() < 0.75
    if op != "attend":
        seqs, rows = _log_int(rng, 1, 64), _log_int(rng, 1, 8192)
        rows = max(1, min(rows, 100_000 // seqs))
        ctx = 0 if op == "read" else _log_int(rng, 1, 4096)
        return {"op": op, "seqs": seqs, "rows": rows, "ctx": ctx, "page": page, "ragged": ragged,
                "dtype": rng.choice(["bf16", "f16", "f32"])}
    heads = rng.choice([1, 7, 16, 40, 64, 128])
    seqs, rows, ctx = _log_int(rng, 1, 64), _log_int(rng, 1, 2048), _log_int(rng, 1, 16384)
    ctx = max(1, min(ctx, 260_000 // seqs))
    # no more scores than the largest listed case has
    rows = max(1, min(rows, int(1.2e9 / (seqs * heads * (ctx + rows)))))
    return {"op": op, "seqs": seqs, "rows": rows, "ctx": ctx, "heads": heads, "page": page, "ragged": ragged,
            "sink": rng.random() < 0.5, "causal": rng.random() < 0.8, "dtype": "bf16"}


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


def work(case):
    lens = _lengths(case)
    rows, keys = sum(n for n, _ in lens), sum(s for _, s in lens)
    if case["op"] != "attend":
        return {"bytes": rows * (RECORD + QK * SIZES[case["dtype"]]), "flops": 0}
    heads = case["heads"]
    seen = sum(n * s - (n * (n - 1) // 2 if case["causal"] else 0) for n, s in lens)
    return {"bytes": keys * RECORD + rows * heads * (2 * QK + 2 * LATENT + 4), "flops": 2 * seen * heads * (QK + LATENT)}


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
    lens = _lengths(case)
    dev, page, dtype = "cuda", case["page"], TYPES[case["dtype"]]
    g = torch.Generator(device=dev)
    g.manual_seed(int(seed) * 1_000_003 + 17)
    rows = sum(n for n, _ in lens)
    pages = [-(-s // page) for _, s in lens]
    n_pages = sum(pages) + 3
    s = {"op": case["op"], "lens": lens}
    order = torch.randperm(n_pages, generator=g, device=dev).to(torch.int32)
    table = torch.full((len(lens), max(pages)), -1, dtype=torch.int32, device=dev)
    at = 0
    for b, k in enumerate(pages):
        table[b, :k] = order[at:at + k]
        at += k
    s["table"] = table
    ends = [0]
    for n, _ in lens:
        ends.append(ends[-1] + n)
    s["cu"] = torch.tensor(ends, dtype=torch.int32, device=dev)
    s["seq_lens"] = torch.tensor([k for _, k in lens], dtype=torch.int32, device=dev)

    def normal(*shape, std=1.0):
        return torch.randn(*shape, generator=g, device=dev) * std

    if case["op"] == "write":
        s["cache"] = torch.full((n_pages, page, RECORD), 0x11, dtype=torch.uint8, device=dev)
        s["latent"] = normal(rows, LATENT, std=math.sqrt(2.0)).to(dtype)
        s["rope"] = normal(rows, ROPE).to(dtype)
        return s
    cache = torch.empty(n_pages * page, RECORD, dtype=torch.uint8, device=dev)
    for lo in range(0, cache.shape[0], 65536):
        part = cache[lo:lo + 65536]
        part.copy_(_records(normal(part.shape[0], LATENT, std=math.sqrt(2.0)), normal(part.shape[0], ROPE)))
    s["cache"] = cache.view(n_pages, page, RECORD)
    if case["op"] == "read":
        s["latent"] = torch.empty(rows, LATENT, dtype=dtype, device=dev)
        s["rope"] = torch.empty(rows, ROPE, dtype=dtype, device=dev)
        return s
    heads = case["heads"]
    s["causal"] = case["causal"]
    s["q"] = normal(rows, heads, QK).to(dtype)
    s["sink"] = normal(heads) if case["sink"] else None
    s["out"] = torch.empty(rows, heads, LATENT, dtype=dtype, device=dev)
    s["lse"] = torch.empty(rows, heads, dtype=torch.float32, device=dev)
    return s


def _fields(cache):
    """The cache's values: E4M3 latent, f32 scales, bf16 rope (views)."""
    return {"latent": cache[..., :512].view(torch.float8_e4m3fn), "scale": cache[..., 512:528].view(torch.float32),
            "rope": cache[..., 528:].view(torch.bfloat16)}


def _token_slots(s):
    """Global slot (page * page_size + offset) of every token row."""
    cu, page = s["cu"].long(), s["cache"].shape[1]
    row = torch.arange(sum(n for n, _ in s["lens"]), device=cu.device)
    seq = torch.searchsorted(cu, row, right=True) - 1
    pos = s["seq_lens"].long()[seq] - cu[seq + 1] + row
    return s["table"].long()[seq, pos // page] * page + pos % page


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
    # token rows padded to the longest chunk, chunks ending at the same place
    row = cu[1:, None] - most + torch.arange(most, device=dev)
    real = row >= cu[:-1, None]
    q = s["q"].float()[row.clamp_min(0)]  # [seqs, most, heads, 576]
    x = torch.matmul(q.view(n_seqs, most * heads, QK), k.transpose(1, 2)).mul_(SM_SCALE)
    lens = s["seq_lens"].long()[:, None]
    seen = lens - most + 1 + torch.arange(most, device=dev) if s["causal"] else lens.expand(-1, most)
    seen = seen.repeat_interleave(heads, 1)[..., None]
    x.masked_fill_(key >= seen, -math.inf)
    m = x.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, torch.zeros_like(m), m)
    e = x.sub_(m).exp_()
    total = e.sum(-1, keepdim=True)
    lse = (m + total.log())[..., 0].view(n_seqs, most, heads)
    if s["sink"] is not None:
        total = total + (s["sink"].repeat(most)[None, :, None] - m).exp()
    out = (torch.matmul(e, lat) / total).view(n_seqs, most, heads, LATENT)
    return {"out": out[real].to(s["q"].dtype), "lse": lse[real]}


def run(s):
    if own:
        import sparse_mla_decode_csr_gb300 as smla
        if s["op"] == "write":
            smla.smla_paged_write(s["latent"], s["rope"], s["cache"], s["table"], s["cu"], s["seq_lens"])
            return _fields(s["cache"])
        if s["op"] == "read":
            smla.smla_paged_read(s["cache"], s["table"], s["cu"], s["seq_lens"], s["latent"], s["rope"])
            return {"latent": s["latent"], "rope": s["rope"]}
        smla.smla_paged_attend(s["q"], s["cache"], s["table"], s["cu"], s["seq_lens"], SM_SCALE, s["sink"],
                               s["out"], s["lse"], causal=s["causal"])
        return {"out": s["out"], "lse": s["lse"]}
    if s["op"] == "write":
        s["cache"].view(-1, RECORD)[_token_slots(s)] = _records(s["latent"], s["rope"])
        return _fields(s["cache"])
    if s["op"] == "read":
        lat, rope = _values(s["cache"].view(-1, RECORD)[_token_slots(s)])
        return {"latent": lat.to(s["latent"].dtype), "rope": rope.to(s["rope"].dtype)}
    return _plain_attend(s)


# ---- the definition in 64 bits, sequence by sequence ----


def _e4m3_values(dev):
    table = []
    for code in range(256):
        e, m = code >> 3 & 15, code & 7
        v = math.nan if code & 127 == 127 else m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10)
        table.append(-v if code > 127 else v)
    return torch.tensor(table, dtype=torch.float64, device=dev)


def _keys64(records):
    """f64 [n, 576] keys of records [n, 656]."""
    v = _e4m3_values(records.device)[records[:, :512].long()]
    scale = records[:, 512:528].contiguous().view(torch.float32).double()
    rope = records[:, 528:].contiguous().view(torch.bfloat16).double()
    return torch.cat([v * scale.repeat_interleave(128, 1), rope], 1)


def _round_e4m3(x):
    """x in f64 to the nearest E4M3 value, ties to even, saturating."""
    _, e = torch.frexp(x)
    step = torch.exp2((e - 4).clamp_min(-9).double())
    return ((x / step).round() * step).clamp(-448.0, 448.0)


def exact(case, seed):
    s = prepare(case, seed)
    page, cache = case["page"], s["cache"]
    table, cu, flat = s["table"].tolist(), s["cu"].tolist(), cache.view(-1, RECORD)
    slots = [torch.tensor([table[b][p // page] * page + p % page for p in range(k)], device=cache.device)
             for b, (_, k) in enumerate(s["lens"])]
    if case["op"] == "write":
        got = {name: v.double() for name, v in _fields(cache).items()}
        at = torch.cat([slots[b][k - n:] for b, (n, k) in enumerate(s["lens"])])
        x = s["latent"].double().view(-1, 4, 128)
        y = x.abs().amax(2).clamp_min(1e-4) / 448.0
        scale = torch.exp2(torch.floor(torch.log2(y)) - 1)  # below y; doubled until it is not
        for _ in range(3):
            scale = torch.where(scale < y, 2 * scale, scale)
        got["latent"].view(-1, LATENT)[at] = _round_e4m3(x / scale[..., None]).flatten(1)
        got["scale"].view(-1, 4)[at] = scale
        got["rope"].view(-1, ROPE)[at] = s["rope"].to(torch.bfloat16).double()
        return got
    if case["op"] == "read":
        k = _keys64(torch.cat([flat[slots[b][k - n:]] for b, (n, k) in enumerate(s["lens"])]))
        return {"latent": k[:, :LATENT], "rope": k[:, LATENT:]}
    if work(case)["flops"] > 8e12:
        return None
    heads = case["heads"]
    out = torch.empty(cu[-1], heads, LATENT, dtype=torch.float64, device=cache.device)
    lse = torch.empty(cu[-1], heads, dtype=torch.float64, device=cache.device)
    for b, (n, length) in enumerate(s["lens"]):
        k = _keys64(flat[slots[b]])
        few = max(1, int(2.5e8 / (heads * length)))
        for lo in range(0, n, few):
            hi = min(n, lo + few)
            x = s["q"][cu[b] + lo:cu[b] + hi].double().view(-1, QK) @ k.t() * SM_SCALE
            x = x.view(hi - lo, heads, length)
            if case["causal"]:
                last = length - n + torch.arange(lo, hi, device=cache.device)
                x = x.masked_fill(torch.arange(length, device=cache.device) > last[:, None, None], -math.inf)
            z = torch.logsumexp(x, -1)
            lse[cu[b] + lo:cu[b] + hi] = z
            if s["sink"] is not None:
                z = torch.logaddexp(z, s["sink"].double())
            p = torch.exp(x - z[..., None])
            out[cu[b] + lo:cu[b] + hi] = (p.view(-1, length) @ k[:, :LATENT]).view(hi - lo, heads, LATENT)
    return {"out": out, "lse": lse}

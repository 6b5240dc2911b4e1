"""Cases of the paged key/value cache operators: page and slot tables, the append of new keys and values, and the
attention of new tokens over the cache.

`listed()` and `draw(rng)` give cases, `prepare(case, seed)` their inputs on the GPU, `run(state)` one pass: through
`means_clustering_amd.kvcache` where `own` is true, else in elementary torch operations in 32 bits, rounded once at
the end.  `exact(case, seed)` is the same output from the definition in 64 bits and `work(case)` the bytes and
operations that a pass cannot do without.

Lengths are given by the case (its request count, largest lengths and kind); a seed only shuffles the requests, so
that the work of a case does not depend on the seed.
"""
import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}


# ------------------------------------------------------------------------------------------------------- cases ----

def listed():
    return [
        # Page and slot tables.  A few chats in their decode step: one new token each, all latency.
        dict(name="tables_decode_8", op="tables", requests=8, ctx=2000, new=1, kind="decode", page=16),
        # A serving step with a quarter of the requests in chunked prefill, the rest decoding, some idle.
        dict(name="tables_mixed_250", op="tables", requests=250, ctx=8191, new=511, kind="mixed", page=16),
        # The largest step: thousands of requests with long contexts and ragged chunks.
        dict(name="tables_mixed_4095", op="tables", requests=4095, ctx=32767, new=255, kind="mixed", page=64),
        # Append.  One decode step of 5 requests, rows taken out of one packed projection.
        dict(name="append_decode_5", op="append", tokens=5, hq=32, hkv=8, dim=128, rot=128, style="halves",
             dtype="bf16", norm=True, page=16, packed=True),
        # A ragged chunk of a smaller model, rotation of interleaved pairs in half of the row, no norm.
        dict(name="append_chunk_1001", op="append", tokens=1001, hq=16, hkv=16, dim=64, rot=32, style="pairs",
             dtype="fp16", norm=False, page=32, packed=False),
        # A full prefill step.
        dict(name="append_prefill_16384", op="append", tokens=16384, hq=32, hkv=8, dim=128, rot=128, style="halves",
             dtype="bf16", norm=True, page=64, packed=True),
        # Attention.  One short chat in its decode step: all latency.
        dict(name="attend_decode_1", op="attend", requests=1, ctx=500, new=1, kind="decode", hq=32, hkv=8, dim=128,
             dtype="bf16", page=16, window=0, weighted=False),
        # A serving batch in decode, ragged contexts.
        dict(name="attend_decode_64", op="attend", requests=64, ctx=8191, new=1, kind="decode", hq=32, hkv=8, dim=128,
             dtype="bf16", page=16, window=0, weighted=False),
        # Two very long contexts whose older keys are K-Means centroids, weighted by their counts.
        dict(name="attend_decode_weighted_2", op="attend", requests=2, ctx=131000, new=1, kind="decode", hq=28, hkv=4,
             dim=128, dtype="fp16", page=64, window=0, weighted=True),
        # A mixed step of a small model with a sliding window: chunks, decodes and idle requests together.
        dict(name="attend_mixed_window_30", op="attend", requests=30, ctx=4095, new=301, kind="mixed", hq=16, hkv=16,
             dim=64, dtype="fp16", page=32, window=1000, weighted=False),
        # One chunk of a long prompt, with few rows against a long cache.
        dict(name="attend_chunk_509", op="attend", requests=1, ctx=30000, new=509, kind="chunk", hq=32, hkv=8, dim=128,
             dtype="bf16", page=16, window=0, weighted=False),
        # The largest: a wide chunk of a long prompt.
        dict(name="attend_chunk_8192", op="attend", requests=1, ctx=24576, new=8192, kind="chunk", hq=32, hkv=8,
             dim=128, dtype="bf16", page=64, window=0, weighted=False),
    ]


def _odd(rng, lo, hi):
    """An odd size, spread over the logarithm of [lo, hi]."""
    n = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    return max(1, min(hi, n | 1) if hi % 2 else min(hi - 1, n | 1))


def draw(rng):
    op = rng.choice(["tables", "append", "append", "attend", "attend", "attend"])
    if op == "tables":
        kind = rng.choice(["decode", "mixed", "chunk"])
        case = dict(op=op, requests=_odd(rng, 1, 4095), ctx=_odd(rng, 63, 32767),
                    new=1 if kind == "decode" else _odd(rng, 3, 1023), kind=kind, page=rng.choice([16, 32, 64, 128]))
        while work(case)["bytes"] > work(listed()[2])["bytes"]:
            case["requests"] = case["requests"] // 2 | 1
        return case
    if op == "append":
        hkv, group, dim = rng.choice([1, 2, 4, 8, 16]), rng.choice([1, 4, 7, 8]), rng.choice([64, 80, 128, 256])
        packed = rng.random() < 0.5
        if packed:
            hkv, group, dim = 8, rng.choice([4, 8]), 128
        case = dict(op=op, tokens=_odd(rng, 1, 16383), hq=hkv * group, hkv=hkv, dim=dim,
                    rot=rng.choice([dim, dim // 32 * 16]), style=rng.choice(["halves", "pairs"]),
                    dtype=rng.choice(["bf16", "fp16"]), norm=rng.random() < 0.6, page=rng.choice([16, 32, 64, 128]),
                    packed=packed)
        while work(case)["bytes"] > work(listed()[5])["bytes"]:
            case["tokens"] = case["tokens"] // 2 | 1
        return case
    kind = rng.choice(["decode", "decode", "mixed", "chunk"])
    hkv, group = rng.choice([1, 2, 4, 8]), rng.choice([1, 2, 4, 7, 8, 16])
    case = dict(op=op, requests=_odd(rng, 1, 255) if kind != "chunk" else _odd(rng, 1, 9), ctx=_odd(rng, 31, 131071),
                new=1 if kind == "decode" else _odd(rng, 3, 2047), kind=kind, hq=hkv * group, hkv=hkv,
                dim=rng.choice([64, 80, 128, 128, 256]), dtype=rng.choice(["bf16", "fp16"]),
                page=rng.choice([16, 32, 64, 128]), window=rng.choice([0, 0, 0, _odd(rng, 15, 4095)]),
                weighted=rng.random() < 0.3)
    top = work(listed()[-1])["flops"] / 4
    while work(case)["flops"] > top or _cache_bytes(case) > 8 << 30:
        k = "requests" if case["requests"] > 1 and rng.random() < 0.5 else "ctx"
        case[k] = max(case[k] // 2 | 1, 31 if k == "ctx" else 1)
        if case["ctx"] == 31 and case["requests"] == 1:
            case["new"] = case["new"] // 2 | 1
    return case


def _lengths(case):
    """(tokens in the cache, new tokens) of each request, from the case alone."""
    r = random.Random(case["requests"] * 1000003 + case["ctx"] * 1009 + case["new"])
    out = []
    for i in range(case["requests"]):
        if case["requests"] == 1:
            c = case["ctx"]
        else:
            c = case["ctx"] if i == 0 else int(case["ctx"] * math.exp(-2.8 * r.random()))
        n = case["new"]
        if case["kind"] == "mixed":
            u = r.random()
            n = r.randint(2, max(2, n)) if u < 0.25 or i == 0 else (0 if u > 0.97 else 1)
            c = 0 if 0.20 < u < 0.25 and i > 0 else c  # a prompt's first chunk
        out.append((c, n))
    return out


def _cache_bytes(case):
    return sum(c + n + case["page"] for c, n in _lengths(case)) * case["hkv"] * case["dim"] * 4


def _visible(c, n, window):
    """Query-key pairs of one request: row i sees keys max(0, c + i - window + 1) .. c + i."""
    if not window:
        return n * c + n * (n + 1) // 2
    return sum(min(c + i + 1, window) for i in range(n))


def work(case):
    if case["op"] == "tables":
        lens, p = _lengths(case), case["page"]
        total = sum(n for _, n in lens)
        taken = sum(-(-(c + n) // p) - -(-c // p) for c, n in lens)
        # lengths in; query starts, page starts, sequence lengths, positions and slots out; each new page read from
        # the free list and written to the table; the table entry under each request's first new token
        return {"bytes": 4 * (6 * len(lens) + 2 * total + 2 * taken), "flops": 4 * total}
    if case["op"] == "append":
        rows = case["tokens"] * (case["hq"] + 2 * case["hkv"])
        qk = case["tokens"] * (case["hq"] + case["hkv"])
        return {"bytes": 2 * 2 * rows * case["dim"] + case["tokens"] * (8 + 4 * case["rot"]),
                "flops": qk * (3 * case["rot"] + (4 * case["dim"] if case["norm"] else 0))}
    lens, w = _lengths(case), case["window"]
    keys = sum(min(c + n, w + n - 1) if w else c + n for c, n in lens if n)
    total = sum(n for _, n in lens)
    pairs = sum(_visible(c, n, w) for c, n in lens)
    cache = keys * case["hkv"] * (4 * case["dim"] + (4 if case["weighted"] else 0))
    return {"bytes": cache + total * case["hq"] * (4 * case["dim"] + 4) + 4 * (keys // case["page"] + 3 * len(lens)),
            "flops": 4 * case["dim"] * case["hq"] * pairs}


# ------------------------------------------------------------------------------------------------------ inputs ----

def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    host = random.Random(seed)
    st = dict(case=case)
    if case["op"] == "append":
        _prepare_append(st, case, g)
    else:
        lens = _lengths(case)
        host.shuffle(lens)
        st["lens"] = lens
        if case["op"] == "tables":
            _prepare_tables(st, case, g)
        else:
            _prepare_attend(st, case, g)
    if own:
        from means_clustering_amd import kvcache
        st["kvcache"], st["ws"] = kvcache, kvcache.Workspace("cuda")
    return st


def _ints(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def _pages(lens, page, g, spare):
    """A block table whose rows hold the pages of `lens` tokens in shuffled order, and the shuffled pages left over."""
    need = [-(-n // page) for n in lens]
    order = torch.randperm(sum(need) + spare, generator=g, device="cuda").to(torch.int32)
    return need, order


def _fill_table(need, order, width):
    """Row r of the table holds the next need[r] pages of `order`, then -1."""
    col = torch.arange(width, device="cuda")[None]
    first = torch.tensor([0] + need, device="cuda").cumsum(0)[:-1]
    have = torch.tensor(need, device="cuda")
    at = (first[:, None] + col).clamp(max=max(order.numel() - 1, 0))
    return torch.where(col < have[:, None], order[at], torch.full_like(at, -1, dtype=torch.int32))


def _prepare_tables(st, case, g):
    lens, p = st["lens"], case["page"]
    width = -(-(case["ctx"] + case["new"]) // p) + 1
    taken = sum(-(-(c + n) // p) - -(-c // p) for c, n in lens)
    need, order = _pages([c for c, _ in lens], p, g, taken + 16)
    st["block_table"] = _fill_table(need, order, width)
    st["free"] = order[sum(need):].contiguous()
    st["ctx"], st["new"] = _ints([c for c, _ in lens]), _ints([n for _, n in lens])
    # tokens that each request has seen but no longer holds (its older keys were replaced by fewer centroids)
    st["offset"] = torch.randint(0, 1000, (len(lens),), generator=g, device="cuda", dtype=torch.int32)
    st["total"] = sum(n for _, n in lens)


def _prepare_append(st, case, g):
    t, hq, hkv, d, dt = case["tokens"], case["hq"], case["hkv"], case["dim"], DTYPES[case["dtype"]]
    if case["packed"]:
        qkv = torch.randn(t, hq + 2 * hkv, d, generator=g, device="cuda").to(dt)
        st["q"], st["k"], st["v"] = qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]
    else:
        st["q"] = torch.randn(t, hq, d, generator=g, device="cuda").to(dt)
        st["k"] = torch.randn(t, hkv, d, generator=g, device="cuda").to(dt)
        st["v"] = torch.randn(t, hkv, d, generator=g, device="cuda").to(dt)
    pages = -(-t // case["page"]) + 2
    st["k_cache"] = torch.randn(pages, case["page"], hkv, d, generator=g, device="cuda").to(dt)
    st["v_cache"] = torch.randn(pages, case["page"], hkv, d, generator=g, device="cuda").to(dt)
    # the tokens fill pages in shuffled order, each page from its start
    order = torch.randperm(pages, generator=g, device="cuda")[: -(-t // case["page"])]
    at = torch.arange(t, device="cuda")
    st["slots"] = (order[at // case["page"]] * case["page"] + at % case["page"]).to(torch.int32)
    limit = 32768
    st["positions"] = ((at * 7 + int(torch.randint(0, limit, (1,), generator=g, device="cuda"))) % limit).to(torch.int32)
    angle = torch.arange(limit, device="cuda", dtype=torch.float64)[:, None] * torch.pow(
        10000.0, -torch.arange(0, case["rot"], 2, device="cuda", dtype=torch.float64) / case["rot"])[None]
    st["rope"] = torch.cat([angle.cos(), angle.sin()], dim=1).float()
    st["q_weight"] = 1 + 0.2 * torch.randn(d, generator=g, device="cuda") if case["norm"] else None
    st["k_weight"] = 1 + 0.2 * torch.randn(d, generator=g, device="cuda") if case["norm"] else None
    st["out"] = torch.empty(t, hq, d, dtype=dt, device="cuda")


def _prepare_attend(st, case, g):
    lens, p, d, dt = st["lens"], case["page"], case["dim"], DTYPES[case["dtype"]]
    hq, hkv = case["hq"], case["hkv"]
    seq, total = [c + n for c, n in lens], sum(n for _, n in lens)
    need, order = _pages(seq, p, g, 4)
    st["block_table"] = _fill_table(need, order, max(need) + 1)
    pages = order.numel()
    # normed and rotated queries and keys: scores of about unit spread after the scale, some heads sharper
    st["q"] = (torch.randn(total, hq, d, generator=g, device="cuda")
               * (0.5 + 1.5 * torch.rand(hq, 1, generator=g, device="cuda"))).to(dt)
    st["k_cache"] = torch.empty(pages, p, hkv, d, dtype=dt, device="cuda").normal_(generator=g)
    st["v_cache"] = torch.empty(pages, p, hkv, d, dtype=dt, device="cuda").normal_(generator=g)
    st["log_weight"] = None
    if case["weighted"]:
        # logarithms of cluster sizes; 1 in 20 clusters is empty
        n = torch.randint(1, 65, (pages, hkv, p), generator=g, device="cuda").float().log()
        empty = torch.rand(pages, hkv, p, generator=g, device="cuda") < 0.05
        st["log_weight"] = torch.where(empty, torch.full_like(n, -math.inf), n)
    st["query_start"] = _ints([0] + [n for _, n in lens]).cumsum(0).to(torch.int32)
    st["seq_lens"] = _ints(seq)
    st["scale"] = d ** -0.5
    st["max_new"] = max(n for _, n in lens)
    st["out"] = torch.empty(total, hq, d, dtype=dt, device="cuda")
    st["lse"] = torch.empty(total, hq, dtype=torch.float32, device="cuda")


# ------------------------------------------------------------------------------------------------------ passes ----

def run(st):
    op = st["case"]["op"]
    if own:
        return {"tables": _own_tables, "append": _own_append, "attend": _own_attend}[op](st)
    return {"tables": _plain_tables, "append": _plain_append, "attend": _plain_attend}[op](st)


def _own_tables(st):
    t = st["kvcache"].tables(st["ctx"], st["new"], st["block_table"], st["free"], st["case"]["page"], st["total"],
                             pos_offset=st["offset"])
    return {"block_table": st["block_table"], "seq_lens": t.seq_lens, "query_start": t.query_start,
            "page_start": t.page_start, "positions": t.positions, "slots": t.slots}


def _own_append(st):
    st["kvcache"].append(st["q"], st["k"], st["v"], st["k_cache"], st["v_cache"], st["slots"],
                         positions=st["positions"], rope=st["rope"], q_weight=st["q_weight"],
                         k_weight=st["k_weight"], eps=1e-6, interleaved=st["case"]["style"] == "pairs",
                         out=st["out"])
    return {"q": st["out"], "k_cache": st["k_cache"], "v_cache": st["v_cache"]}


def _own_attend(st):
    st["kvcache"].attend(st["q"], st["k_cache"], st["v_cache"], st["block_table"], st["query_start"], st["seq_lens"],
                         scale=st["scale"], window=st["case"]["window"], log_weight=st["log_weight"],
                         max_new=st["max_new"], out=st["out"], lse=st["lse"], ws=st["ws"])
    return {"out": st["out"], "lse": st["lse"]}


def _starts(n):
    return torch.cat([n.new_zeros(1), n.cumsum(0, dtype=torch.int32)])


def _plain_tables(st):
    ctx, new, free, p, table = st["ctx"], st["new"], st["free"], st["case"]["page"], st["block_table"]
    have, need = (ctx + p - 1) // p, (ctx + new + p - 1) // p
    query_start, page_start = _starts(new), _starts(need - have)
    col = torch.arange(table.shape[1], device="cuda")[None]
    taken = page_start[:-1, None] + col - have[:, None]
    fresh = torch.where(taken < free.numel(), free[taken.clamp(0, free.numel() - 1)], -1)
    table.copy_(torch.where((col >= have[:, None]) & (col < need[:, None]), fresh, table))
    # the request of each token: the number of requests that end at or before it
    ends = torch.zeros(st["total"] + 1, dtype=torch.int64, device="cuda")
    ends.index_add_(0, query_start[1:].long(), torch.ones_like(query_start[1:], dtype=torch.int64))
    req = ends.cumsum(0)[:-1]
    at = ctx[req] + torch.arange(st["total"], device="cuda", dtype=torch.int32) - query_start[req]
    slots = table[req, (at // p).long()] * p + at % p
    return {"block_table": table, "seq_lens": ctx + new, "query_start": query_start, "page_start": page_start,
            "positions": at + st["offset"][req], "slots": slots}


def _plain_rows(x, weight, rope, positions, interleaved):
    x = x.float()
    if weight is not None:
        x = x / (x.square().mean(-1, keepdim=True) + 1e-6).sqrt() * weight
    half = rope.shape[1] // 2
    cos, sin = rope[positions.long(), None, :half], rope[positions.long(), None, half:]
    if interleaved:
        a, b = x[..., 0:2 * half:2], x[..., 1:2 * half:2]
        turned = torch.stack([a * cos - b * sin, b * cos + a * sin], dim=-1).flatten(-2)
    else:
        a, b = x[..., :half], x[..., half:2 * half]
        turned = torch.cat([a * cos - b * sin, b * cos + a * sin], dim=-1)
    return torch.cat([turned, x[..., 2 * half:]], dim=-1)


def _plain_append(st):
    case, dt = st["case"], DTYPES[st["case"]["dtype"]]
    pairs, slots = case["style"] == "pairs", st["slots"].long()
    q = _plain_rows(st["q"], st["q_weight"], st["rope"], st["positions"], pairs).to(dt)
    k = _plain_rows(st["k"], st["k_weight"], st["rope"], st["positions"], pairs).to(dt)
    st["k_cache"].view(-1, case["hkv"], case["dim"])[slots] = k
    st["v_cache"].view(-1, case["hkv"], case["dim"])[slots] = st["v"]
    return {"q": q, "k_cache": st["k_cache"], "v_cache": st["v_cache"]}


def _plain_attend(st):
    case, d, p = st["case"], st["case"]["dim"], st["case"]["page"]
    hq, hkv = case["hq"], case["hkv"]
    group, dt = hq // hkv, DTYPES[case["dtype"]]
    out, lse = torch.empty_like(st["out"]), torch.empty_like(st["lse"])
    t0 = 0
    for r, (c, n) in enumerate(st["lens"]):
        if n == 0:
            continue
        # rows see keys from `lo` on at the earliest (a sliding window), in whole pages
        lo = max(0, c - case["window"] + 1) // p * p if case["window"] else 0
        pages = st["block_table"][r, lo // p:-(-(c + n) // p)].long()
        keys = c + n - lo
        k, v = st["k_cache"][pages], st["v_cache"][pages]  # [pages, page, hkv, d]
        at = torch.arange(lo, c + n, device="cuda")[None, :]
        row = torch.arange(c, c + n, device="cuda").repeat_interleave(group)[:, None]
        hidden = at > row
        if case["window"]:
            hidden = hidden | (at <= row - case["window"])
        for h in range(hkv):
            kh, vh = k[:, :, h].reshape(-1, d)[:keys].float(), v[:, :, h].reshape(-1, d)[:keys].float()
            q = st["q"][t0:t0 + n, h * group:(h + 1) * group].reshape(n * group, d).float()
            s = (q @ kh.t()) * st["scale"]
            if st["log_weight"] is not None:
                lw = st["log_weight"][pages, h].reshape(-1)[:keys]
                s = s + lw[None]
                vh = vh.masked_fill(lw[:, None] == -math.inf, 0.0)
            s = s.masked_fill(hidden, -math.inf)
            top = s.max(dim=1, keepdim=True).values
            top = torch.where(top == -math.inf, torch.zeros_like(top), top)
            e = (s - top).exp()
            z = e.sum(dim=1, keepdim=True)
            o = torch.where(z > 0, (e @ vh) / z, torch.zeros_like(z))
            out[t0:t0 + n, h * group:(h + 1) * group] = o.to(dt).view(n, group, d)
            lse[t0:t0 + n, h * group:(h + 1) * group] = (top + z.log()).view(n, group)
        t0 += n
    return {"out": out, "lse": lse}


# ------------------------------------------------------------------------------------------------------- exact ----

def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "tables":
        return None  # whole numbers
    return _exact_append(st, case) if case["op"] == "append" else _exact_attend(st, case)


def _exact_append(st, case):
    turn = case["rot"] // 2
    pos = st["positions"].long()
    # each pair of elements is a complex number, turned by cos + i sin of its token's position
    w = torch.complex(st["rope"][pos, :turn].double(), st["rope"][pos, turn:].double())[:, None]
    i = torch.arange(turn, device="cuda")
    first, second = (2 * i, 2 * i + 1) if case["style"] == "pairs" else (i, i + turn)

    def rows(x, weight):
        y = x.double()
        if weight is not None:
            y = y * torch.rsqrt((y * y).sum(-1, keepdim=True) / case["dim"] + 1e-6) * weight.double()
        z = torch.complex(y[..., first], y[..., second]) * w
        y = y.clone()
        y[..., first], y[..., second] = z.real, z.imag
        return y

    page, at = st["slots"].long() // case["page"], st["slots"].long() % case["page"]
    k_cache, v_cache = st["k_cache"].double(), st["v_cache"].double()
    k_cache[page, at] = rows(st["k"], st["k_weight"])
    v_cache[page, at] = st["v"].double()
    return {"q": rows(st["q"], st["q_weight"]), "k_cache": k_cache, "v_cache": v_cache}


def _exact_attend(st, case):
    p, group = case["page"], case["hq"] // case["hkv"]
    out = torch.zeros(st["out"].shape, dtype=torch.float64, device="cuda")
    lse = torch.full(st["lse"].shape, -math.inf, dtype=torch.float64, device="cuda")
    starts = st["query_start"].tolist()
    for r, length in enumerate(st["seq_lens"].tolist()):
        a, b = starts[r], starts[r + 1]
        if a == b:
            continue
        j = torch.arange(length, device="cuda")
        page, at = st["block_table"][r].long()[j // p], j % p
        i = torch.arange(length - (b - a), length, device="cuda")
        seen = j[None] <= i[:, None]
        if case["window"]:
            seen &= j[None] > i[:, None] - case["window"]
        for h in range(case["hq"]):
            s = st["q"][a:b, h].double() @ st["k_cache"][page, at, h // group].double().t() * st["scale"]
            if case["weighted"]:
                s += st["log_weight"][page, h // group, at].double()[None]
            s[~seen] = -math.inf
            norm = torch.logsumexp(s, dim=1)
            some = norm > -math.inf
            s -= torch.where(some, norm, torch.zeros_like(norm))[:, None]
            out[a:b, h] = s.exp() @ st["v_cache"][page, at, h // group].double()
            lse[a:b, h] = norm
    return {"out": out, "lse": lse}

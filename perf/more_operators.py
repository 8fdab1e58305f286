"""Performance cases of the operators around the paged key/value cache that
serve long conversations:

- the norm of query and key heads with the rotation by position
  (``tp3d_qk_rope``), its backward pass (``tp3d_qk_rope_bwd``) and its form for
  a server, which writes keys and values to their slots
  (``tp3d_paged_rope_store``);
- attention over the cache with a sliding window and a few first tokens that
  stay visible (``tp3d_paged_attn_window``);
- forking, giving back and compacting the cache's pages (``tp3d_paged_fork``,
  ``tp3d_paged_free``, ``tp3d_paged_compact``), and the copies these ask for
  (``tp3d_paged_copy``).

Where ``own`` is false each is computed from elementary torch operations in 32
bits, the angles of positions in 64.
"""
from __future__ import annotations

import math
import random

import torch

own = False

# the q = 2 GPT layer of this repository's benchmark has 16 heads of 128 (hidden 2048), batch 4, sequence 1024
_LAYER = {"heads": 16, "kv_heads": 16, "dim": 128}
_GROUPED = {"heads": 32, "kv_heads": 8, "dim": 128}
_BASE, _EPS = 10000.0, 1e-6
_CONTEXT = 4096  # positions that the frequencies were made for, where they are scaled


def listed():
    def turn(name, op, tokens, heads, kv_heads, dim, rotary, interleaved=False, norm=True, dtype="bf16", scaling="plain",
             factor=1.0, far=4096, page=16, heads_first=False):
        return {"name": name, "op": op, "tokens": tokens, "heads": heads, "kv_heads": kv_heads, "dim": dim, "rotary": rotary,
                "interleaved": interleaved, "norm": norm, "dtype": dtype, "scaling": scaling, "factor": factor, "far": far,
                "page": page, "heads_first": heads_first}

    def attn(name, requests, cached, fresh, singles, page, window, sinks, heads_first=False, **heads):
        return {"name": name, "op": "attn", "requests": requests, "cached": cached, "fresh": fresh, "singles": singles,
                "page": page, "window": window, "sinks": sinks, "heads_first": heads_first, **heads}

    def pages(name, op, requests, others, kv, page, kv_heads=8, dim=128, heads_first=False):
        return {"name": name, "op": op, "requests": requests, "others": others, "kv": kv, "page": page,
                "kv_heads": kv_heads, "dim": dim, "heads_first": heads_first}

    return [
        # queries and keys of one generation step of 64 requests, keys and values to the cache: latency
        turn("turn+store decode 64", "store", 64, 16, 16, 128, 128, far=16384),
        # a large prompt batch with grouped heads, frequencies scaled for a long context
        turn("turn+store prompts 16385", "store", 16385, 32, 8, 128, 128, scaling="parts", factor=8.0, far=32768, page=64,
             heads_first=True),
        # a training step in 32 bits, a part of each head turned, neighbouring columns paired, odd token count
        turn("turn f32 part 4095", "turn", 4095, 12, 4, 96, 48, interleaved=True, dtype="f32"),
        # the gradients of a training step of the layer's own shape
        turn("turn backward 4x1024", "back", 4096, 16, 16, 128, 128, far=1024),
        # one user, one token, far into a conversation: latency
        attn("window decode 1x16384", 1, 16383, 1, 1, 16, 1024, 4, **_LAYER),
        # a server's steady state: long conversations of all lengths
        attn("window decode 32x131071", 32, 131070, 1, 32, 64, 4096, 4, True, **_GROUPED),
        # the next chunk of a long prompt
        attn("window chunk 2048 over 32001", 1, 29953, 2048, 0, 64, 4096, 4, **_LAYER),
        # chunks of four prompts in one batch with twelve requests at one token each, a short window without first tokens
        attn("window mixed 16 up to 384", 16, 3700, 384, 12, 16, 511, 0, heads=32, kv_heads=8, dim=64),
        # four samples of each of two prompts: latency
        pages("fork 2 into 8", "fork", 2, 8, 1500, 16),
        # beams of a large batch over long prompts in small pages
        pages("fork 64 into 448", "fork", 64, 448, 8000, 16, kv_heads=4, dim=64),
        # all pages of the requests that end in a step, some of them shared with others
        pages("free 256", "free", 256, 64, 8192, 16),
        # a fragmented pool drawn together
        pages("compact 32x8192", "compact", 32, 0, 8192, 32, heads_first=True),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["store", "turn", "back", "decode", "decode", "chunk", "chunk", "fork", "free", "compact"])
    page = rng.choice([16, 32, 64, 128])
    first = rng.random() < 0.5
    heads, kv_heads = rng.choice([(16, 16), (8, 8), (32, 8), (16, 2), (16, 1), (12, 4), (14, 2)])
    if op in ("store", "turn", "back"):
        dim = rng.choice([64, 128] if op == "store" else [64, 80, 96, 128, 256])
        scaling = rng.choice(["plain", "linear", "base", "parts"])
        dtype = "bf16" if op == "store" else rng.choice(["bf16", "bf16", "f32"])
        most = 16385 * 48 * 128 // ((heads + kv_heads) * dim * (1 if dtype == "bf16" else 2) * (2 if op == "back" else 1))
        return {"op": op, "tokens": _log_int(rng, 1, min(16385, most)), "heads": heads, "kv_heads": kv_heads, "dim": dim,
                "rotary": dim if rng.random() < 0.5 else 16 * rng.randint(1, dim // 16),
                "interleaved": rng.random() < 0.5, "norm": rng.random() < 0.7, "dtype": dtype, "scaling": scaling,
                "factor": 1.0 if scaling == "plain" else rng.choice([2.0, 4.0, 8.0]), "far": _log_int(rng, 64, 131072),
                "page": page, "heads_first": first}
    if op in ("decode", "chunk"):
        c = {"op": "attn", "page": page, "heads_first": first, "heads": heads, "kv_heads": kv_heads,
             "dim": rng.choice([64, 128]), "window": _log_int(rng, 16, 8192), "sinks": rng.choice([0, 1, 4, 64, 200])}
        if op == "decode":
            requests = _log_int(rng, 1, 64)
            # no more cache than the largest listed case reads
            most = max(16, 32 * 4100 * 8 * 128 // (requests * kv_heads * c["dim"]) - c["sinks"])
            return c | {"requests": requests, "cached": _log_int(rng, 1, 131071), "fresh": 1, "singles": requests,
                        "window": min(c["window"], most)}
        requests = _log_int(rng, 1, 16)
        fresh = _log_int(rng, 2, 2048 // requests)
        # no more scores than the largest listed case forms
        return c | {"requests": requests, "cached": _log_int(rng, 1, 32768), "fresh": fresh,
                    "singles": rng.choice([0, requests // 2]), "window": min(c["window"], 2 ** 27 // (requests * fresh * heads))}
    requests = _log_int(rng, 1, {"fork": 64, "free": 256, "compact": 32}[op])
    return {"op": op, "requests": requests, "others": {"fork": _log_int(rng, 1, 448), "free": rng.randint(0, 64), "compact": 0}[op],
            "kv": _log_int(rng, 33, 8192), "page": page, "kv_heads": rng.choice([1, 2, 4]), "dim": rng.choice([64, 128]),
            "heads_first": first}


def _rng(case):
    return random.Random(repr(sorted((k, v) for k, v in case.items() if k != "name")))


def _lengths(case):
    """(cached, new) tokens of each request: the first has the case's largest
    sizes, the others are spread below them."""
    rng, cached, fresh = _rng(case), [], []
    for b in range(case["requests"]):
        cached.append(case["cached"] if b == 0 else rng.randint(0, case["cached"]))
        fresh.append(case["fresh"] if b == 0 else rng.randint((case["fresh"] + 1) // 2, case["fresh"]))
    for b in range(case["requests"] - case["singles"], case["requests"]):
        fresh[b] = 1
    return cached, fresh


def _kept(case):
    """Tokens in the cache of each request; the first, the longest, ends inside a page."""
    rng = _rng(case)
    kv = [case["kv"] - (case["kv"] % case["page"] == 0)]
    return kv + [rng.randint(1, kv[0]) for _ in range(case["requests"] - 1)]


def _pages(n, page):
    return -(-n // page)


def _normal(gen, *shape, dtype=torch.bfloat16):
    return torch.empty(shape, dtype=dtype, device="cuda").normal_(generator=gen)


def _pool(gen, pages, page, kv_heads, dim, heads_first):
    """A key or value pool seen as (page, token, head, column), full of what earlier requests left in it."""
    if heads_first:
        return _normal(gen, pages, kv_heads, page, dim).transpose(1, 2)
    return _normal(gen, pages, page, kv_heads, dim)


def _frequencies(case):
    """Radians per position of each pair of columns, and the factor of the turned columns."""
    r, s = case["rotary"], case["factor"]
    base = _BASE * s ** (r / (r - 2)) if case["scaling"] == "base" else _BASE
    f = base ** (-torch.arange(0, r, 2, dtype=torch.float64, device="cuda") / r)
    if case["scaling"] == "linear":
        f = f / s
    if case["scaling"] == "parts":  # pairs of less than 1 turn over the context are interpolated, of more than 32 kept
        keep = ((_CONTEXT * f / (2 * math.pi) - 1) / 31).clamp(0, 1)
        f = f * keep + f / s * (1 - keep)
        return f, 0.1 * math.log(s) + 1
    return f, 1.0


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    prep = {"store": _prepare_turn, "turn": _prepare_turn, "back": _prepare_turn, "attn": _prepare_attn}
    return {"op": case["op"], "case": case, **prep.get(case["op"], _prepare_pages)(case, gen)}


def _prepare_turn(case, gen):
    t, h, kh, d = case["tokens"], case["heads"], case["kv_heads"], case["dim"]
    dtype = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32
    # rows as the packed query/key/value product leaves them
    packed = _normal(gen, t, (h + 2 * kh) * d, dtype=dtype)
    freq, magnitude = _frequencies(case)
    s = {"q": packed[:, :h * d].view(t, h, d), "k": packed[:, h * d:(h + kh) * d].view(t, kh, d),
         "v": packed[:, (h + kh) * d:].view(t, kh, d), "freq": freq, "magnitude": magnitude,
         "positions": torch.randint(0, case["far"], (t,), dtype=torch.int32, device="cuda", generator=gen),
         "q_weight": 1 + 0.2 * _normal(gen, d, dtype=dtype) if case["norm"] else None,
         "k_weight": 1 + 0.2 * _normal(gen, d, dtype=dtype) if case["norm"] else None,
         "q_out": torch.empty(t, h, d, dtype=dtype, device="cuda")}
    if case["op"] == "store":
        pages, page = _pages(t, case["page"]) + 4, case["page"]
        # new tokens fill whole pages in a scattered page order, as a plan lays them out
        order, at = torch.randperm(pages, generator=gen, device="cuda"), torch.arange(t, device="cuda")
        s["slots"] = order[at // page] * page + at % page
        s["cache_k"], s["cache_v"] = (_pool(gen, pages, page, kh, d, case["heads_first"]) for _ in range(2))
    else:
        s["k_out"] = torch.empty(t, kh, d, dtype=dtype, device="cuda")
    if case["op"] == "back":
        s["dq_out"], s["dk_out"] = _normal(gen, t, h, d, dtype=dtype), _normal(gen, t, kh, d, dtype=dtype)
        if case["norm"]:
            s["dq_weight"], s["dk_weight"] = (torch.empty(d, dtype=dtype, device="cuda") for _ in range(2))
    return s


def _prepare_attn(case, gen):
    i32 = {"dtype": torch.int32, "device": "cuda"}
    page, requests = case["page"], case["requests"]
    window, sinks = case["window"], case["sinks"]
    h, kh, d = case["heads"], case["kv_heads"], case["dim"]
    cached, fresh = _lengths(case)
    tokens, kv = sum(fresh), [c + f for c, f in zip(cached, fresh)]
    width = _pages(max(kv), page)
    # a server gives back the pages that no window reaches any more: columns [kept, gone) of the table have none
    kept = torch.tensor([min(_pages(sinks, page), _pages(n, page)) for n in kv], device="cuda")
    gone = torch.tensor([max(min(_pages(sinks, page), _pages(n, page)), max(0, c - window + 1) // page)
                         for c, n in zip(cached, kv)], device="cuda")
    need = torch.tensor([_pages(n, page) for n in kv], device="cuda")
    cols = torch.arange(width, device="cuda")
    held = (cols < need[:, None]) & ((cols < kept[:, None]) | (cols >= gone[:, None]))
    used = int(held.sum())
    pages = used + used // 8 + 4
    order = torch.randperm(pages, generator=gen, device="cuda").to(torch.int32)
    nth = held.flatten().cumsum(0).view(requests, width) - 1
    starts = [0]
    for f in fresh:
        starts.append(starts[-1] + f)
    # queries as the packed query/key/value product leaves them; scores of standard deviation 2
    packed = _normal(gen, tokens, (h + 2 * kh) * d)
    packed[:, :h * d] *= 2
    return {"tokens": tokens, "q": packed[:, :h * d].view(tokens, h, d), "q_start": torch.tensor(starts, **i32),
            "kv_len": torch.tensor(kv, **i32), "table": torch.where(held, order[nth.clamp(min=0)], -1).to(torch.int32),
            "most_new": max(fresh), "most_kv": max(kv), "cache_k": _pool(gen, pages, page, kh, d, case["heads_first"]),
            "cache_v": _pool(gen, pages, page, kh, d, case["heads_first"]),
            "out": torch.empty(tokens, h, d, dtype=torch.bfloat16, device="cuda"),
            "lse": torch.empty(tokens, h, dtype=torch.float32, device="cuda")}


def _prepare_pages(case, gen):
    i32 = {"dtype": torch.int32, "device": "cuda"}
    op, page, n, others = case["op"], case["page"], case["requests"], case["others"]
    kv = torch.tensor(_kept(case), device="cuda")
    need = (kv + page - 1) // page
    width, used = _pages(case["kv"], page) + 2, int(need.sum())
    # a compaction finds half of the pool free; otherwise some of it is
    pages = 2 * used + 5 if op == "compact" else used + others + used // 4 + 8
    rows = n + others
    order = torch.randperm(pages, generator=gen, device="cuda").to(torch.int32)
    # the bookkeeping in one buffer: tables, owners beyond the first of each page, free list
    book = torch.empty(rows * width + 2 * pages, **i32)
    s = {"book": book, "pages": pages, "table": book[:rows * width].view(rows, width),
         "shares": book[rows * width:rows * width + pages], "free": book[rows * width + pages:],
         "free_count": torch.tensor([pages - used], **i32), "free_left": torch.zeros(1, **i32)}
    cols = torch.arange(width, device="cuda")
    first = need.cumsum(0) - need
    table = torch.where(cols < need[:, None], order[(first[:, None] + cols).clamp(max=pages - 1)], -1).to(torch.int32)
    s["table"].fill_(-1)
    s["table"][:n] = table
    s["shares"].zero_()
    s["free"].fill_(-1)
    s["free"][:pages - used] = order[used:]
    if op == "free":
        # requests n + i share the whole pages of request i; every other row ends, or gives up what lies behind its window
        of = torch.arange(others, device="cuda") % n
        common = kv[of] // page
        shared = torch.where(cols < common[:, None], table[of], -1)
        s["table"][n:] = shared
        s["shares"].add_(torch.bincount(shared[shared >= 0].long(), minlength=pages).to(torch.int32))
        held, row = torch.cat([need, common]), torch.arange(rows, device="cuda")
        s["first"] = torch.where(row % 4 == 0, 1, 0).to(torch.int32)
        s["end"] = torch.where(row % 4 == 0, held // 2, torch.where(row % 2 == 1, held, 0)).to(torch.int32)
    else:
        s["copy_from"], s["copy_to"] = (torch.full((max(others, pages // 2),), -1, **i32) for _ in range(2))
        s["copy_count"] = torch.zeros(1, **i32)
        s["cache_k"], s["cache_v"] = (_pool(gen, pages, page, case["kv_heads"], case["dim"], case["heads_first"])
                                      for _ in range(2))
    if op == "fork":
        child = torch.arange(others, device="cuda")
        s["src"], s["dst"] = (child % n).to(torch.int32), (n + child).to(torch.int32)
        s["len"] = kv[child % n].to(torch.int32)
    if op == "compact":
        s["kv_len"], s["page_map"] = kv.to(torch.int32), torch.empty(pages, **i32)
    s["book_before"] = book.clone()
    return s


def _turned(x, s):
    """x (token, head, column) in 32 bits with its first columns turned by the positions' angles."""
    c = s["case"]
    r = c["rotary"]
    angle = s["positions"].double()[:, None] * s["freq"]
    cos, sin = ((f(angle) * s["magnitude"]).float()[:, None] for f in (torch.cos, torch.sin))
    if c["interleaved"]:
        a, b = x[..., 0:r:2], x[..., 1:r:2]
        turned = torch.stack([a * cos - b * sin, a * sin + b * cos], -1).flatten(2)
    else:
        a, b = x[..., :r // 2], x[..., r // 2:r]
        turned = torch.cat([a * cos - b * sin, a * sin + b * cos], -1)
    return torch.cat([turned, x[..., r:]], -1)


def _turned_back(g, s):
    """The transposed rotation."""
    c = s["case"]
    r = c["rotary"]
    angle = s["positions"].double()[:, None] * s["freq"]
    cos, sin = ((f(angle) * s["magnitude"]).float()[:, None] for f in (torch.cos, torch.sin))
    if c["interleaved"]:
        a, b = g[..., 0:r:2], g[..., 1:r:2]
        turned = torch.stack([a * cos + b * sin, b * cos - a * sin], -1).flatten(2)
    else:
        a, b = g[..., :r // 2], g[..., r // 2:r]
        turned = torch.cat([a * cos + b * sin, b * cos - a * sin], -1)
    return torch.cat([turned, g[..., r:]], -1)


def _plain_turn(s):
    def one(x, weight):
        y = x.float()
        if weight is not None:
            y = y / (y.square().mean(-1, keepdim=True) + _EPS).sqrt() * weight.float()
        return _turned(y, s).to(x.dtype)

    q, k = one(s["q"], s["q_weight"]), one(s["k"], s["k_weight"])
    if s["op"] == "turn":
        return {"q": q, "k": k}
    at, off = s["slots"] // s["case"]["page"], s["slots"] % s["case"]["page"]
    s["cache_k"][at, off] = k
    s["cache_v"][at, off] = s["v"]
    return {"q": q, "cache_k": s["cache_k"], "cache_v": s["cache_v"]}


def _plain_back(s):
    def one(x, dy, weight):
        g = _turned_back(dy.float(), s)
        if weight is None:
            return g.to(x.dtype), None
        y, w = x.float(), weight.float()
        inv = 1 / (y.square().mean(-1, keepdim=True) + _EPS).sqrt()
        n = y * inv
        gw = g * w
        dx = inv * (gw - n * (gw * n).mean(-1, keepdim=True))
        return dx.to(x.dtype), (g * n).sum((0, 1)).to(x.dtype)

    (dq, dqw), (dk, dkw) = one(s["q"], s["dq_out"], s["q_weight"]), one(s["k"], s["dk_out"], s["k_weight"])
    return {"dq": dq, "dk": dk, "dq_weight": dqw, "dk_weight": dkw}


def _plain_attn(s):
    c = s["case"]
    h, kh, d, page, window, sinks = c["heads"], c["kv_heads"], c["dim"], c["page"], c["window"], c["sinks"]
    requests, most_new, g = c["requests"], s["most_new"], h // kh
    starts, kv = s["q_start"].long(), s["kv_len"].long()
    new = starts[1:] - starts[:-1]
    # the keys that some row sees: the first ones, then from the first row's window on; where the two meet, none twice
    lead = min(sinks, s["most_kv"])
    x = torch.arange(min(lead + window + most_new - 1, s["most_kv"]), device="cuda")
    behind = ((kv - new - window + 1).clamp(min=0) - lead).clamp(min=0)
    key = torch.where(x < lead, x, x + behind[:, None])
    there = key < kv[:, None]
    ids = s["table"].long().gather(1, (key // page).clamp(max=s["table"].shape[1] - 1)).clamp(min=0)
    k = s["cache_k"][ids, key % page].transpose(1, 2).float()
    v = s["cache_v"][ids, key % page].transpose(1, 2).float()
    j = torch.arange(most_new, device="cuda")
    rows = (starts[:-1, None] + j).clamp(max=s["tokens"] - 1)
    q = s["q"][rows].float().view(requests, most_new, kh, g, d).permute(0, 2, 3, 1, 4).reshape(requests, kh, g * most_new, d)
    score = (q @ k.transpose(2, 3) * (1.0 / math.sqrt(d))).view(requests, kh, g, most_new, -1)
    last = ((kv - new)[:, None] + j)[:, :, None]
    key = key[:, None]
    seen = there[:, None] & (key <= last) & ((key > last - window) | (key < sinks))
    score = score.masked_fill_(~seen[:, None, None], -math.inf)
    top = score.amax(-1, keepdim=True).clamp(min=-3e38)  # rows of padding may see nothing
    p = (score - top).exp()
    total = p.sum(-1, keepdim=True)
    o = (p.view(requests, kh, g * most_new, -1) @ v).view(requests, kh, g, most_new, d) / total
    lse = (top + total.log())[..., 0]
    t = torch.arange(s["tokens"], device="cuda")
    b = torch.searchsorted(starts[1:], t, right=True)
    j = t - starts[b]
    return {"out": o.permute(0, 3, 1, 2, 4)[b, j].reshape(-1, h, d).bfloat16(),
            "lse": lse.permute(0, 3, 1, 2)[b, j].reshape(-1, h)}


def _plain_copy(s):
    n = int(s["copy_count"])
    at, to = s["copy_from"][:n].long(), s["copy_to"][:n].long()
    s["cache_k"][to] = s["cache_k"][at]
    s["cache_v"][to] = s["cache_v"][at]


def _plain_fork(s):
    s["book"].copy_(s["book_before"])
    page, table, shares = s["case"]["page"], s["table"], s["shares"]
    src, dst, length = s["src"].long(), s["dst"].long(), s["len"].long()
    full, part = length // page, length % page > 0
    cols = torch.arange(table.shape[1], device="cuda")
    mine = table[src]
    whole = (cols < full[:, None]) & (mine >= 0)
    shares.index_add_(0, mine.clamp(min=0).long().flatten(), whole.flatten().int())
    nth = part.cumsum(0) - 1
    fresh = s["free"][(s["free_count"] - 1 - nth).clamp(min=0)]
    row = torch.where(cols < full[:, None], mine, table[dst])
    table[dst] = torch.where((cols == full[:, None]) & part[:, None], fresh[:, None], row)
    # the n-th copy: an extra place at the end takes what is none
    at = torch.where(part, nth, s["copy_from"].numel())
    for name, pages in (("copy_from", mine.gather(1, full[:, None].clamp(max=table.shape[1] - 1))[:, 0]), ("copy_to", fresh)):
        wide = torch.cat([s[name], s[name][:1]])
        wide[at] = pages
        s[name].copy_(wide[:-1])
    s["copy_count"].copy_(part.sum())
    s["free_left"].copy_(s["free_count"] - part.sum())
    _plain_copy(s)


def _plain_free(s):
    s["book"].copy_(s["book_before"])
    table, shares, pages = s["table"], s["shares"], s["pages"]
    cols = torch.arange(table.shape[1], device="cuda")
    gone = (cols >= s["first"][:, None]) & (cols < s["end"][:, None]) & (table >= 0)
    given = torch.zeros(pages, dtype=torch.int32, device="cuda").index_add_(0, table.clamp(min=0).long().flatten(),
                                                                            gone.flatten().int())
    free = (given > 0) & (shares < given)
    shares.copy_(torch.where(free, 0, shares - given))
    table.masked_fill_(gone, -1)
    # the highest first, so that the lowest are taken first again
    down = free.flip(0)
    at = torch.where(down, s["free_count"] + down.cumsum(0) - 1, pages)
    wide = torch.cat([s["free"], s["free"][:1]])
    wide[at] = torch.arange(pages - 1, -1, -1, dtype=torch.int32, device="cuda")
    s["free"].copy_(wide[:-1])
    s["free_left"].copy_(s["free_count"] + free.sum())


def _plain_compact(s):
    s["book"].copy_(s["book_before"])
    page, table, shares, pages = s["case"]["page"], s["table"], s["shares"], s["pages"]
    every = torch.arange(pages, dtype=torch.int32, device="cuda")
    listed_free = torch.where(every < s["free_count"], s["free"], pages).long()
    free = torch.zeros(pages + 1, dtype=torch.bool, device="cuda")
    free[listed_free] = True
    free = free[:pages]
    used = pages - s["free_count"]
    hole, mover = free & (every < used), ~free & (every >= used)
    for name, mask in (("copy_from", mover), ("copy_to", hole)):
        wide = torch.cat([s[name], s[name][:1]])
        wide[torch.where(mask, mask.cumsum(0) - 1, s[name].numel())] = every
        s[name].copy_(wide[:-1])
    s["copy_count"].copy_(hole.sum())
    nth = (mover.cumsum(0) - 1).clamp(0, s["copy_to"].numel() - 1)
    s["page_map"].copy_(torch.where(free, -1, torch.where(mover, s["copy_to"][nth], every)))
    back = (hole.cumsum(0) - 1).clamp(0, s["copy_to"].numel() - 1)
    moved = shares[s["copy_from"][back].clamp(min=0).long()]
    shares.copy_(torch.where(every >= used, 0, torch.where(hole, moved, shares)))
    cols = torch.arange(table.shape[1], device="cuda")
    held = (cols < ((s["kv_len"] + page - 1) // page)[:, None]) & (table >= 0)
    table.copy_(torch.where(held, s["page_map"][table.clamp(min=0).long()], table))
    s["free"].copy_(torch.where(every < s["free_count"], pages - 1 - every, s["free"]))
    _plain_copy(s)


def _pages_out(s):
    names = {"fork": ("table", "shares", "free_left", "copy_from", "copy_to", "copy_count", "cache_k", "cache_v"),
             "free": ("table", "shares", "free", "free_left"),
             "compact": ("table", "shares", "free", "page_map", "copy_from", "copy_to", "copy_count", "cache_k", "cache_v")}
    return {k: s[k] for k in names[s["op"]]}


_contexts = {}


def _handles(s):
    """The context, and what a program lays out once: tables of frequencies, descriptors, workspaces."""
    import tensor_transformer_layer_cube_gb300 as tp

    if "tp" in s:
        return s["tp"], s["ctx"]
    device = torch.cuda.current_device()
    if device not in _contexts:
        _contexts[device] = tp.tp3d_create(device)
    s["tp"], s["ctx"], c = tp, _contexts[device], s["case"]
    if s["op"] in ("store", "turn", "back"):
        kind = {"plain": tp.TP3D_ROPE_PLAIN, "linear": tp.TP3D_ROPE_LINEAR, "base": tp.TP3D_ROPE_BASE,
                "parts": tp.TP3D_ROPE_PARTS}[c["scaling"]]
        turns, magnitude = tp.rope_turns(c["rotary"], _BASE, kind, c["factor"], _CONTEXT)
        s["turns"] = turns.cuda()
        s["rope"] = tp.rope(s["turns"], s["q"].dtype, c["dim"], c["rotary"], interleaved=c["interleaved"],
                            magnitude=magnitude, norm=c["norm"], eps=_EPS, q_weight=s["q_weight"], k_weight=s["k_weight"])
        if s["op"] == "back":
            n = tp.tp3d_qk_rope_bwd_workspace_bytes(s["ctx"], s["rope"])
            s["workspace"] = torch.empty(n, dtype=torch.uint8, device="cuda")
    if "cache_k" in s:
        s["cache"] = tp.kv_cache(s["cache_k"], s["cache_v"])
    if s["op"] == "attn":
        s["batch"] = tp.paged_batch(s["q_start"], s["kv_len"], s["table"], s["tokens"], s["most_new"])
        n = tp.tp3d_paged_attn_workspace_bytes(s["ctx"], s["cache"], c["heads"])
        s["workspace"] = torch.empty(n, dtype=torch.uint8, device="cuda")
    if "book" in s:
        s["pool"] = tp.page_pool(c["page"], s["table"], s["shares"], s["free"])
    return s["tp"], s["ctx"]


def run(state):
    s = state
    if not own:
        if s["op"] in ("store", "turn"):
            return _plain_turn(s)
        if s["op"] == "back":
            return _plain_back(s)
        if s["op"] == "attn":
            return _plain_attn(s)
        {"fork": _plain_fork, "free": _plain_free, "compact": _plain_compact}[s["op"]](s)
        return _pages_out(s)
    tp, ctx = _handles(s)
    if s["op"] == "store":
        tp.check(tp.tp3d_paged_rope_store(ctx, s["rope"], s["cache"], s["q"], s["k"], s["v"], s["positions"], s["slots"],
                                          s["q_out"]))
        return {"q": s["q_out"], "cache_k": s["cache_k"], "cache_v": s["cache_v"]}
    if s["op"] == "turn":
        tp.check(tp.tp3d_qk_rope(ctx, s["rope"], s["q"], s["k"], s["positions"], s["q_out"], s["k_out"]))
        return {"q": s["q_out"], "k": s["k_out"]}
    if s["op"] == "back":
        tp.check(tp.tp3d_qk_rope_bwd(ctx, s["rope"], s["q"], s["k"], s["positions"], s["dq_out"], s["dk_out"], s["q_out"],
                                     s["k_out"], s.get("dq_weight"), s.get("dk_weight"), s["workspace"]))
        return {"dq": s["q_out"], "dk": s["k_out"], "dq_weight": s.get("dq_weight"), "dk_weight": s.get("dk_weight")}
    if s["op"] == "attn":
        tp.check(tp.tp3d_paged_attn_window(ctx, s["cache"], s["batch"], s["q"], s["out"], s["lse"],
                                           1.0 / math.sqrt(s["case"]["dim"]), s["case"]["window"], s["case"]["sinks"],
                                           s["workspace"]))
        return {"out": s["out"], "lse": s["lse"]}
    # a step's tables differ from the last one's; each pass begins from the same ones
    s["book"].copy_(s["book_before"])
    if s["op"] == "fork":
        tp.check(tp.tp3d_paged_fork(ctx, s["pool"], s["src"], s["dst"], s["len"], s["free_count"], s["free_left"],
                                    s["copy_from"], s["copy_to"], s["copy_count"]))
        tp.check(tp.tp3d_paged_copy(ctx, s["cache"], s["src"].numel(), s["copy_from"], s["copy_to"], s["copy_count"]))
    elif s["op"] == "free":
        tp.check(tp.tp3d_paged_free(ctx, s["pool"], s["first"], s["end"], s["free_count"], s["free_left"]))
    else:
        tp.check(tp.tp3d_paged_compact(ctx, s["pool"], s["kv_len"], s["free_count"], s["page_map"], s["copy_from"],
                                       s["copy_to"], s["copy_count"]))
        tp.check(tp.tp3d_paged_copy(ctx, s["cache"], s["pages"] // 2, s["copy_from"], s["copy_to"], s["copy_count"]))
    return _pages_out(s)


def work(case):
    op = case["op"]
    if op in ("store", "turn", "back"):
        t, h, kh, d, size = case["tokens"], case["heads"], case["kv_heads"], case["dim"], 2 if case["dtype"] == "bf16" else 4
        moved = t * (h + kh) * d * size
        if op == "back":
            return {"bytes": (3 if case["norm"] else 2) * moved + 4 * t, "flops": 20 * t * (h + kh) * d}
        extra = t * (2 * kh * d * size + 8) if op == "store" else 0
        return {"bytes": 2 * moved + extra + 4 * t, "flops": 10 * t * (h + kh) * d}
    if op == "attn":
        cached, fresh = _lengths(case)
        h, kh, d, page, window, sinks = (case[k] for k in ("heads", "kv_heads", "dim", "page", "window", "sinks"))
        keys = pairs = table = 0
        for c, f in zip(cached, fresh):
            first = max(0, c - window + 1)  # the first row's window begins here
            lead = min(sinks, first)
            keys += c + f - first + lead
            table += _pages(c + f, page) - first // page + _pages(lead, page)
            for p in range(c, c + f):
                low = max(0, p - window + 1)
                pairs += p + 1 - low + min(sinks, low)
        return {"bytes": keys * kh * d * 4 + sum(fresh) * h * (4 * d + 4) + 4 * table + 8 * case["requests"],
                "flops": 4 * d * h * pairs}
    page, kv = case["page"], _kept(case)
    rows = case["kv_heads"] * case["dim"] * page * 2 * 2  # bytes of a page, keys and values
    held = [_pages(n, page) for n in kv]
    if op == "fork":
        of = [kv[i % case["requests"]] for i in range(case["others"])]
        copies, whole = sum(1 for n in of if n % page), sum(n // page for n in of)
        return {"bytes": 2 * rows * copies + 8 * whole + 24 * len(of), "flops": 0}
    if op == "free":
        held += [kv[i % len(kv)] // page for i in range(case["others"])]
        gone = sum(max(0, n // 2 - 1) if row % 4 == 0 else n if row % 2 else 0 for row, n in enumerate(held))
        return {"bytes": 16 * gone + 8 * len(held) + 8, "flops": 0}
    used = sum(held)
    return {"bytes": 2 * rows * (used // 2) + 8 * used + 12 * (2 * used + 5), "flops": 0}


def _exact_rows(x, weight, case, s, t0, t1):
    """Norm and rotation of tokens [t0, t1) in 64 bits: complex numbers for the pairs."""
    y = x[t0:t1].double()
    if weight is not None:
        y = y * torch.rsqrt((y * y).sum(-1, keepdim=True) / case["dim"] + _EPS) * weight.double()
    r = case["rotary"]
    z = s["magnitude"] * torch.polar(torch.ones((), dtype=torch.float64, device="cuda").expand(t1 - t0, r // 2),
                                     torch.outer(s["positions"][t0:t1].double(), s["freq"]))[:, None]
    out = y.clone()
    if case["interleaved"]:
        w = torch.view_as_complex(y[..., :r].reshape(*y.shape[:2], r // 2, 2)) * z
        out[..., :r] = torch.view_as_real(w).flatten(2)
    else:
        w = torch.complex(y[..., :r // 2].contiguous(), y[..., r // 2:r].contiguous()) * z
        out[..., :r // 2], out[..., r // 2:r] = w.real, w.imag
    return out


def _exact_turn(case, s):
    t = case["tokens"]

    def whole(x, weight):
        return torch.cat([_exact_rows(x, weight, case, s, i, min(t, i + 1024)) for i in range(0, t, 1024)])

    if case["op"] == "back":
        # by differentiation of the rows above
        out = {}
        for n in ("q", "k"):
            w = s[n + "_weight"].double().requires_grad_() if case["norm"] else None
            grads = []
            for i in range(0, t, 1024):
                x = s[n].double()[i:i + 1024].requires_grad_()
                part = {"magnitude": s["magnitude"], "positions": s["positions"][i:i + 1024], "freq": s["freq"]}
                y = _exact_rows(x, w, case, part, 0, x.shape[0])
                y.backward(s["d" + n + "_out"][i:i + 1024].double())
                grads.append(x.grad)
            out["d" + n] = torch.cat(grads)
            out["d" + n + "_weight"] = w.grad if case["norm"] else None
        return out
    q, k = whole(s["q"], s["q_weight"]), whole(s["k"], s["k_weight"])
    if case["op"] == "turn":
        return {"q": q, "k": k}
    out = {"q": q}
    for name, new in (("cache_k", k), ("cache_v", s["v"].double())):
        # slot by slot: rows of a (slots, head, column) array in 64 bits
        pool = s[name].double().reshape(-1, case["kv_heads"], case["dim"])
        out[name] = pool.index_copy(0, s["slots"], new).view(s[name].shape)
    return out


def _exact_attn(case, s):
    cached, fresh = _lengths(case)
    h, kh, d, page, window, sinks = (case[k] for k in ("heads", "kv_heads", "dim", "page", "window", "sinks"))
    out = torch.zeros(s["tokens"], h, d, dtype=torch.float64, device="cuda")
    lse = torch.zeros(s["tokens"], h, dtype=torch.float64, device="cuda")
    t0 = 0
    for b, (c, f) in enumerate(zip(cached, fresh)):
        low = max(0, c - window + 1)
        keys = torch.tensor(sorted(set(range(min(sinks, c + f))) | set(range(low, c + f))), device="cuda")
        ids = s["table"][b][keys // page].long()
        rows = torch.arange(c, c + f, device="cuda")[:, None]
        hidden = (keys > rows) | ((rows - keys >= window) & (keys >= sinks))
        for g in range(kh):
            k, v = (s[n][ids, keys % page, g].double() for n in ("cache_k", "cache_v"))
            for head in range(g * (h // kh), (g + 1) * (h // kh)):
                x = torch.einsum("td,kd->tk", s["q"][t0:t0 + f, head].double(), k) / math.sqrt(d)
                x[hidden] = -math.inf
                n = torch.logsumexp(x, 1)
                lse[t0:t0 + f, head] = n
                out[t0:t0 + f, head] = torch.einsum("tk,kd->td", (x - n[:, None]).exp(), v)
        t0 += f
    return {"out": out, "lse": lse}


def _exact_pages(case, s):
    """The page contents after the copies, page by page; the whole numbers have no other value in 64 bits."""
    page, free, held = case["page"], s["free"].tolist(), s["free_count"].item()
    if case["op"] == "free":
        return None
    moves = []
    if case["op"] == "fork":
        table = s["table"].tolist()
        for src, n in zip(s["src"].tolist(), s["len"].tolist()):
            if n % page:
                held -= 1
                moves.append((table[src][n // page], free[held]))
    else:
        gone, used = set(free[:held]), s["pages"] - held
        moves = list(zip((p for p in range(used, s["pages"]) if p not in gone), sorted(p for p in gone if p < used)))
    out = {k: None for k in _pages_out(s)}
    for name in ("cache_k", "cache_v"):
        pool = s[name].double()
        for a, b in moves:
            pool[b] = pool[a]
        out[name] = pool
    return out


def exact(case, seed):
    s = prepare(case, seed)
    make = {"store": _exact_turn, "turn": _exact_turn, "back": _exact_turn, "attn": _exact_attn}
    return make.get(case["op"], _exact_pages)(case, s)

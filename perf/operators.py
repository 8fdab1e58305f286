"""Performance cases of the paged key/value cache operators.

Serving a GPT decoder layer takes three operators per step: the block tables
and slot maps of the batch (``tp3d_paged_plan``), the write of the new tokens'
keys and values into the cache (``tp3d_paged_store``) and the attention of the
new tokens over it (``tp3d_paged_attn``).  Each case is one call of one of
them.  Where ``own`` is false the operator is computed from elementary torch
operations in 32 bits.
"""
from __future__ import annotations

import math
import random

import torch

own = False

# the q = 2 GPT layer of this repository's benchmark has 16 heads of 128 (hidden 2048), batch 4, sequence 1024
_LAYER = {"heads": 16, "kv_heads": 16, "dim": 128}
_GROUPED = {"heads": 32, "kv_heads": 8, "dim": 128}


def listed():
    def attn(name, requests, cached, fresh, singles, page, heads_first=False, **heads):
        return {"name": name, "op": "attn", "requests": requests, "cached": cached, "fresh": fresh, "singles": singles,
                "page": page, "heads_first": heads_first, **heads}

    return [
        # one generation step of a busy server: every request gets one token
        {"name": "plan decode 256", "op": "plan", "requests": 256, "cached": 4095, "fresh": 1, "page": 16},
        # a batch of prompts entering an empty cache, ragged lengths
        {"name": "plan prompts 64x1024", "op": "plan", "requests": 64, "cached": 0, "fresh": 1024, "page": 16},
        # the keys and values of one generation step
        {"name": "store decode 64", "op": "store", "tokens": 64, "kv_heads": 16, "dim": 128, "page": 16,
         "heads_first": False},
        # the keys and values of a large prompt batch
        {"name": "store prompts 16385", "op": "store", "tokens": 16385, "kv_heads": 8, "dim": 128, "page": 64,
         "heads_first": True},
        # the smallest step: one user, one token, a short conversation; latency
        attn("decode 1x1023", 1, 1022, 1, 1, 16, **_LAYER),
        # a batch of conversations of all lengths, one key/value head per query head
        attn("decode 32x4096", 32, 4095, 1, 32, 16, **_LAYER),
        # a large batch with grouped heads: the steady state of a server
        attn("decode grouped 32x16384", 32, 16383, 1, 32, 64, **_GROUPED),
        # one very long document, one token at a time: the work has to be split along the keys
        attn("decode grouped 1x131071", 1, 131070, 1, 1, 128, True, **_GROUPED),
        # many short requests, one shared key/value head of 64
        attn("decode shared 128x2000", 128, 1999, 1, 128, 32, heads=16, kv_heads=1, dim=64),
        # four prompts of the layer's own training shape
        attn("prompts 4x1024", 4, 0, 1024, 0, 16, **_LAYER),
        # the next chunk of a long prompt
        attn("chunk 2048 over 6145", 1, 6145, 2048, 0, 64, **_LAYER),
        # chunks of four prompts in one batch with twelve requests at one token each
        attn("mixed 16 up to 384", 16, 3700, 384, 12, 16, heads=32, kv_heads=8, dim=64),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["plan", "store", "decode", "decode", "chunk", "chunk"])
    page = rng.choice([16, 32, 64, 128])
    if op == "plan":
        fresh = rng.choice([1, _log_int(rng, 2, 1024)])
        return {"op": "plan", "requests": _log_int(rng, 1, 256 if fresh == 1 else 64), "cached": _log_int(rng, 1, 4096) - 1,
                "fresh": fresh, "page": page}
    if op == "store":
        return {"op": "store", "tokens": _log_int(rng, 1, 16385), "kv_heads": rng.choice([1, 2, 4, 8]),
                "dim": rng.choice([64, 128]), "page": page, "heads_first": rng.random() < 0.5}
    heads, kv_heads = rng.choice([(16, 16), (8, 8), (32, 8), (16, 2), (16, 1), (12, 4), (14, 2)])
    c = {"op": "attn", "page": page, "heads_first": rng.random() < 0.5, "heads": heads, "kv_heads": kv_heads,
         "dim": rng.choice([64, 128])}
    if op == "decode":
        requests = _log_int(rng, 1, 128)
        # no more cache than the largest listed case reads
        most = min(131071, 32 * 16384 * 8 // (requests * kv_heads))
        return c | {"requests": requests, "cached": _log_int(rng, 1, most), "fresh": 1, "singles": requests}
    requests = _log_int(rng, 1, 16)
    fresh = _log_int(rng, 2, 2048 // requests)
    # no more scores than the largest listed case forms
    most = min(65536, 2 ** 28 // (requests * fresh * heads))
    return c | {"requests": requests, "cached": _log_int(rng, 1, max(1, most - fresh)), "fresh": fresh,
                "singles": rng.choice([0, requests // 2])}


def _lengths(case):
    """(cached, new) tokens of each request: the first has the case's largest
    sizes, the others are spread below them."""
    rng = random.Random(repr(sorted((k, v) for k, v in case.items() if k != "name")))
    cached, fresh = [], []
    for b in range(case["requests"]):
        cached.append(case["cached"] if b == 0 else rng.randint(0, case["cached"]))
        fresh.append(case["fresh"] if b == 0 else rng.randint((case["fresh"] + 1) // 2, case["fresh"]))
    for b in range(case["requests"] - case.get("singles", 0), case["requests"]):
        fresh[b] = 1
    return cached, fresh


def _pages(n, page):
    return -(-n // page)


def _pool(gen, pages, page, kv_heads, dim, heads_first):
    """A key or value pool seen as (page, token, head, column), full of what earlier requests left in it."""
    shape = (pages, kv_heads, page, dim) if heads_first else (pages, page, kv_heads, dim)
    p = torch.empty(shape, dtype=torch.bfloat16, device="cuda").normal_(generator=gen)
    return p.transpose(1, 2) if heads_first else p


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    i32 = {"dtype": torch.int32, "device": "cuda"}
    page = case["page"]
    if case["op"] == "store":
        t, h, d = case["tokens"], case["kv_heads"], case["dim"]
        pages = _pages(t, page) + 4
        # new tokens fill whole pages in a scattered page order, as a plan lays them out
        order = torch.randperm(pages, generator=gen, device="cuda")
        at = torch.arange(t, device="cuda")
        packed = torch.empty(t, 3 * h * d, dtype=torch.bfloat16, device="cuda").normal_(generator=gen)
        return {"op": "store", "case": case, "k": packed[:, h * d:2 * h * d].view(t, h, d),
                "v": packed[:, 2 * h * d:].view(t, h, d), "slots": order[at // page] * page + at % page,
                "cache_k": _pool(gen, pages, page, h, d, case["heads_first"]),
                "cache_v": _pool(gen, pages, page, h, d, case["heads_first"])}
    cached, fresh = _lengths(case)
    requests, tokens = case["requests"], sum(fresh)
    kv = [c + f for c, f in zip(cached, fresh)]
    width = _pages(max(kv), page)
    held = cached if case["op"] == "plan" else kv
    used, need = [_pages(n, page) for n in held], [_pages(n, page) for n in kv]
    pages = sum(need) + sum(need) // 8 + 4
    order = torch.randperm(pages, generator=gen, device="cuda").to(torch.int32)
    first = torch.tensor([sum(used[:b]) for b in range(requests)], device="cuda")
    cols = torch.arange(width, device="cuda")
    mine = cols < torch.tensor(used, device="cuda")[:, None]
    table = torch.where(mine, order[(first[:, None] + cols).clamp_(max=pages - 1)], -1).to(torch.int32)
    state = {"op": case["op"], "case": case, "tokens": tokens, "table": table}
    if case["op"] == "plan":
        state |= {"cached": torch.tensor(cached, **i32), "fresh": torch.tensor(fresh, **i32),
                  "free": order[sum(used):].clone(), "free_count": torch.tensor([pages - sum(used)], **i32),
                  "q_start": torch.empty(requests + 1, **i32), "kv_len": torch.empty(requests, **i32),
                  "slots": torch.empty(tokens, dtype=torch.int64, device="cuda"),
                  "positions": torch.empty(tokens, **i32), "free_left": torch.empty(1, **i32)}
        return state
    h, kh, d = case["heads"], case["kv_heads"], case["dim"]
    starts = [0]
    for f in fresh:
        starts.append(starts[-1] + f)
    # queries as the packed query/key/value product leaves them; scores of standard deviation 2
    packed = torch.empty(tokens, (h + 2 * kh) * d, dtype=torch.bfloat16, device="cuda").normal_(generator=gen)
    packed[:, :h * d] *= 2
    state |= {"q": packed[:, :h * d].view(tokens, h, d), "q_start": torch.tensor(starts, **i32),
              "kv_len": torch.tensor(kv, **i32), "most_new": max(fresh), "most_kv": max(kv),
              "cache_k": _pool(gen, pages, page, kh, d, case["heads_first"]),
              "cache_v": _pool(gen, pages, page, kh, d, case["heads_first"]),
              "out": torch.empty(tokens, h, d, dtype=torch.bfloat16, device="cuda"),
              "lse": torch.empty(tokens, h, dtype=torch.float32, device="cuda")}
    return state


def _plain_plan(s):
    page = s["case"]["page"]
    cached, fresh = s["cached"].long(), s["fresh"].long()
    kv = cached + fresh
    ends = fresh.cumsum(0)
    old, new = (cached + page - 1) // page, (kv + page - 1) // page
    need = new - old
    first = need.cumsum(0) - need
    j = torch.arange(s["table"].shape[1], device="cuda") - old[:, None]
    take = (j >= 0) & (j < need[:, None])
    at = (s["free_count"] - 1 - first[:, None] - j).clamp(0, s["free"].numel() - 1)
    table = torch.where(take, s["free"][at], s["table"])
    t = torch.arange(s["tokens"], device="cuda")
    b = torch.searchsorted(ends, t, right=True)
    pos = cached[b] + t - (ends - fresh)[b]
    slots = table[b, pos // page].long() * page + pos % page
    q_start = torch.cat([torch.zeros_like(ends[:1]), ends])
    return {"table": table, "q_start": q_start.int(), "kv_len": kv.int(), "slots": slots, "positions": pos.int(),
            "free_left": (s["free_count"] - need.sum()).int()}


def _plain_store(s):
    page = s["case"]["page"]
    at, off = s["slots"] // page, s["slots"] % page
    s["cache_k"][at, off] = s["k"]
    s["cache_v"][at, off] = s["v"]
    return {"cache_k": s["cache_k"], "cache_v": s["cache_v"]}


def _plain_attn(s):
    h, kh, d = s["case"]["heads"], s["case"]["kv_heads"], s["case"]["dim"]
    requests, most_new, most_kv, g = s["case"]["requests"], s["most_new"], s["most_kv"], h // kh
    starts, kv = s["q_start"].long(), s["kv_len"].long()
    new = starts[1:] - starts[:-1]
    # the cache of every request, padded to the longest: (request, head, key, column)
    pages = s["table"].clamp(min=0).long()
    k = s["cache_k"][pages].flatten(1, 2)[:, :most_kv].transpose(1, 2).float()
    v = s["cache_v"][pages].flatten(1, 2)[:, :most_kv].transpose(1, 2).float()
    # the queries, padded to the most new tokens: (request, key/value head, head of its group and token, column)
    j = torch.arange(most_new, device="cuda")
    rows = (starts[:-1, None] + j).clamp(max=s["tokens"] - 1)
    q = s["q"][rows].float().view(requests, most_new, kh, g, d).permute(0, 2, 3, 1, 4).reshape(requests, kh, g * most_new, d)
    score = (q @ k.transpose(2, 3) * (1.0 / math.sqrt(d))).view(requests, kh, g, most_new, most_kv)
    last = (kv - new)[:, None] + j
    hidden = torch.arange(most_kv, device="cuda") > last[:, :, None]
    score = score.masked_fill_(hidden[:, None, None], -math.inf)
    top = score.amax(-1, keepdim=True)
    p = (score - top).exp()
    total = p.sum(-1, keepdim=True)
    o = (p.view(requests, kh, g * most_new, most_kv) @ v).view(requests, kh, g, most_new, d) / total
    lse = (top + total.log())[..., 0]
    t = torch.arange(s["tokens"], device="cuda")
    b = torch.searchsorted(starts[1:], t, right=True)
    j = t - starts[b]
    return {"out": o.permute(0, 3, 1, 2, 4)[b, j].reshape(-1, h, d).bfloat16(),
            "lse": lse.permute(0, 3, 1, 2)[b, j].reshape(-1, h)}


_contexts = {}


def _handles(s):
    """The context, and the descriptors that a server builds once for its cache and each batch."""
    import tensor_transformer_layer_cube_gb300 as tp

    if "tp" not in s:
        device = torch.cuda.current_device()
        if device not in _contexts:
            _contexts[device] = tp.tp3d_create(device)
        s["tp"], s["ctx"] = tp, _contexts[device]
        if s["op"] != "plan":
            s["cache"] = tp.kv_cache(s["cache_k"], s["cache_v"])
        if s["op"] == "attn":
            s["batch"] = tp.paged_batch(s["q_start"], s["kv_len"], s["table"], s["tokens"], s["most_new"])
            n = tp.tp3d_paged_attn_workspace_bytes(s["ctx"], s["cache"], s["case"]["heads"])
            s["workspace"] = torch.empty(n, dtype=torch.uint8, device="cuda")
    return s["tp"], s["ctx"]


def run(state):
    s = state
    if not own:
        return {"plan": _plain_plan, "store": _plain_store, "attn": _plain_attn}[s["op"]](s)
    tp, ctx = _handles(s)
    if s["op"] == "plan":
        tp.check(tp.tp3d_paged_plan(ctx, s["case"]["page"], s["case"]["requests"], s["tokens"], s["cached"], s["fresh"],
                                    s["free"], s["free"].numel(), s["free_count"], s["table"], s["table"].shape[1],
                                    s["q_start"], s["kv_len"], s["slots"], s["positions"], s["free_left"]))
        return {k: s[k] for k in ("table", "q_start", "kv_len", "slots", "positions", "free_left")}
    if s["op"] == "store":
        tp.check(tp.tp3d_paged_store(ctx, s["cache"], s["k"], s["v"], s["slots"]))
        return {"cache_k": s["cache_k"], "cache_v": s["cache_v"]}
    tp.check(tp.tp3d_paged_attn(ctx, s["cache"], s["batch"], s["q"], s["out"], s["lse"],
                                1.0 / math.sqrt(s["case"]["dim"]), s["workspace"]))
    return {"out": s["out"], "lse": s["lse"]}


def work(case):
    if case["op"] == "store":
        moved = 2 * case["tokens"] * case["kv_heads"] * case["dim"] * 2
        return {"bytes": 2 * moved + 8 * case["tokens"], "flops": 0}
    cached, fresh = _lengths(case)
    page, tokens = case["page"], sum(fresh)
    if case["op"] == "plan":
        need = sum(_pages(c + f, page) - _pages(c, page) for c, f in zip(cached, fresh))
        partial = sum(1 for c, f in zip(cached, fresh) if c % page and f)
        return {"bytes": case["requests"] * 16 + 8 * need + 4 * partial + 12 * tokens + 12, "flops": 0}
    h, kh, d = case["heads"], case["kv_heads"], case["dim"]
    pairs = sum(f * c + f * (f + 1) // 2 for c, f in zip(cached, fresh))
    keys = sum(c + f for c, f in zip(cached, fresh))
    table = sum(_pages(c + f, page) for c, f in zip(cached, fresh))
    return {"bytes": keys * kh * d * 4 + tokens * h * (4 * d + 4) + 4 * table + 8 * case["requests"],
            "flops": 4 * d * h * pairs}


def exact(case, seed):
    s = prepare(case, seed)
    page = case["page"]
    if case["op"] == "store":
        out = {}
        for name, new in (("cache_k", s["k"]), ("cache_v", s["v"])):
            # slot by slot: rows of a (slots, head, column) array in 64 bits
            pool = s[name].double().reshape(-1, case["kv_heads"], case["dim"])
            out[name] = pool.index_copy(0, s["slots"], new.double()).view(s[name].shape)
        return out
    cached, fresh = _lengths(case)
    if case["op"] == "plan":
        table, free, left = s["table"].tolist(), s["free"].tolist(), int(s["free_count"])
        starts, slots, positions = [0], [], []
        for b, (c, f) in enumerate(zip(cached, fresh)):
            for i in range(c, c + f):
                if table[b][i // page] < 0:
                    left -= 1
                    table[b][i // page] = free[left]
                slots.append(table[b][i // page] * page + i % page)
                positions.append(i)
            starts.append(starts[-1] + f)
        i32 = torch.int32
        return {"table": torch.tensor(table, dtype=i32), "q_start": torch.tensor(starts, dtype=i32),
                "kv_len": torch.tensor([c + f for c, f in zip(cached, fresh)], dtype=i32),
                "slots": torch.tensor(slots), "positions": torch.tensor(positions, dtype=i32),
                "free_left": torch.tensor([left], dtype=i32)}
    h, kh, d = case["heads"], case["kv_heads"], case["dim"]
    out = torch.zeros(s["tokens"], h, d, dtype=torch.float64, device="cuda")
    lse = torch.zeros(s["tokens"], h, dtype=torch.float64, device="cuda")
    t0 = 0
    for b, (c, f) in enumerate(zip(cached, fresh)):
        ids = s["table"][b, :_pages(c + f, page)].long()
        future = torch.ones(f, c + f, dtype=torch.bool, device="cuda").triu(c + 1)
        for head in range(h):
            of = head // (h // kh)
            k = s["cache_k"][ids, :, of].double().reshape(-1, d)[:c + f]
            v = s["cache_v"][ids, :, of].double().reshape(-1, d)[:c + f]
            x = torch.einsum("td,kd->tk", s["q"][t0:t0 + f, head].double(), k) / math.sqrt(d)
            x[future] = -math.inf
            n = torch.logsumexp(x, 1)
            lse[t0:t0 + f, head] = n
            out[t0:t0 + f, head] = torch.einsum("tk,kd->td", (x - n[:, None]).exp(), v)
        t0 += f
    return {"out": out, "lse": lse}

"""The paged key/value cache on the GPU against the float64 oracle.

Tolerances of the attention, derived from its arithmetic (u = 2^-9, the unit
roundoff of bf16; e = 2^-24, of fp32):
- the scores are fp32 sums of d exact products, so each is off by at most
  (d + 8) e scale sum|q_c k_c| (the 8 covers the scaling and the base-2
  conversion), and a probability by twice that relatively (its own score and
  the maximum), plus 2^-20 for the exponential;
- the probabilities of the second product are rounded to bf16 (u), the output
  again (u).  So |O - want| <= u |want| + (u + s) sum p|v| with s the score
  term, times 1 + 2^-5 for products of the two and the fp32 sums;
- the log-sum-exp is off by the score term, (keys + 64) e from the running
  sum, and 2^-20 (1 + |lse|) from the logarithm and conversions.
"""
import numpy as np
import pytest
import torch

import tensor_transformer_layer_cube_gb300 as t
from oracle import paged as OP
from tests.gpu_util import assert_guards_intact, device, guarded

pytestmark = pytest.mark.gpu

U, E = 2.0 ** -9, 2.0 ** -24
EPAGES = 10


@pytest.fixture(scope="module")
def ctx():
    c = t.tp3d_create(0)
    yield c
    t.tp3d_destroy(c)


def i32(x):
    return torch.as_tensor(np.asarray(x), dtype=torch.int32).to(device())


# ------------------------------------------------------------------ plan
def run_plan(ctx, page, cached, fresh, free, free_count, table, tokens):
    requests, width = table.shape
    out = {"q_start": torch.full((requests + 1,), -7, dtype=torch.int32, device=device()),
           "kv_len": torch.full((requests,), -7, dtype=torch.int32, device=device()),
           "slots": torch.full((tokens,), -7, dtype=torch.int64, device=device()),
           "positions": torch.full((tokens,), -7, dtype=torch.int32, device=device()),
           "free_left": torch.full((1,), -7, dtype=torch.int32, device=device())}
    tab = i32(table)
    st = t.tp3d_paged_plan(ctx, page, requests, tokens, i32(cached), i32(fresh), i32(free), len(free),
                           i32([free_count]), tab, width, out["q_start"], out["kv_len"], out["slots"],
                           out["positions"], out["free_left"])
    assert st == 0
    sync = t.tp3d_sync_status(ctx)
    return {k: v.cpu().numpy() for k, v in out.items()} | {"table": tab.cpu().numpy(), "sync": sync}


def plan_case(rng, requests, page, max_cached, max_fresh, spare=3):
    cached = rng.integers(0, max_cached + 1, requests)
    fresh = rng.integers(0, max_fresh + 1, requests)
    width = max(1, int(max((c + f + page - 1) // page for c, f in zip(cached, fresh)) if requests else 1) + 1)
    held = [-(-int(c) // page) for c in cached]
    need = sum(-(-int(c + f) // page) for c, f in zip(cached, fresh)) - sum(held)
    order = rng.permutation(sum(held) + need + spare)
    table = np.full((requests, width), -1)
    at = 0
    for b, n in enumerate(held):
        table[b, :n] = order[at:at + n]
        at += n
    return cached, fresh, order[at:], table


@pytest.mark.parametrize("requests,page,max_cached,max_fresh", [
    (0, 16, 0, 0), (1, 16, 0, 1), (1, 16, 40, 0), (1, 64, 100, 333), (7, 16, 0, 50), (255, 16, 300, 1),
    (256, 32, 31, 33), (1000, 16, 64, 3), (1025, 128, 500, 7), (4097, 16, 20, 2), (16384, 16, 17, 1),
    (3, 4096, 9000, 5000)])
@pytest.mark.parametrize("pad", [0, 5])
def test_plan(ctx, requests, page, max_cached, max_fresh, pad):
    rng = np.random.default_rng(requests + page)
    cached, fresh, free, table = plan_case(rng, requests, page, max_cached, max_fresh)
    tokens = int(fresh.sum()) + pad
    got = run_plan(ctx, page, cached, fresh, free, len(free), table, tokens)
    q_start, kv, tab, slots, pos, left, fits = OP.plan(page, cached, fresh, free, len(free), table, tokens)
    assert fits and got["sync"] == 0
    np.testing.assert_array_equal(got["q_start"], q_start)
    np.testing.assert_array_equal(got["kv_len"], kv)
    np.testing.assert_array_equal(got["slots"], slots)
    np.testing.assert_array_equal(got["positions"], pos)
    np.testing.assert_array_equal(got["table"], tab)
    assert got["free_left"][0] == left


@pytest.mark.parametrize("what", ["free", "tokens", "width", "negative", "negative cached", "overflow", "count",
                                  "negative count"])
def test_plan_that_does_not_fit(ctx, what):
    rng = np.random.default_rng(5)
    page = 16
    cached, fresh, free, table = plan_case(rng, 9, page, 60, 40, spare=0)
    cached, fresh = cached.astype(np.int64), fresh.astype(np.int64)
    fresh[3] = 20
    cached, fresh, free, table = cached, fresh, np.arange(500, 600), table
    table = np.concatenate([table, np.full((9, 4), -1)], 1)
    count, tokens = len(free), int(fresh.sum())
    if what == "free":
        count = 2  # the step needs 3
    elif what == "tokens":
        tokens -= 11
    elif what == "width":
        fresh[4] = table.shape[1] * page - cached[4] + 1
        tokens = int(fresh.sum())
    elif what == "negative":
        fresh[2] = -3
    elif what == "negative cached":
        cached[2] = -1
    elif what == "overflow":
        cached[2], fresh[2] = 2 ** 31 - 1, 2 ** 31 - 1
    elif what == "count":
        count = len(free) + 1
    else:
        count = -1
    got = run_plan(ctx, page, cached, fresh, free, count, table, tokens)
    assert got["sync"] == EPAGES and t.tp3d_sync_status(ctx) == 0
    want = OP.plan(page, cached, fresh, free, min(max(count, 0), len(free)), table, tokens)
    for k, w in zip(("q_start", "kv_len", "table", "slots", "positions"), want):
        np.testing.assert_array_equal(got[k], w, err_msg=k)
    assert got["free_left"][0] == want[5]


# ------------------------------------------------------------------ pools
def pool(pages, page, kv_heads, d, heads_first=False, pad=0, fill=float("nan")):
    """A (page, token, head, column) view of a pool of stale contents; ``pad`` extra columns between rows."""
    shape = (pages, kv_heads, page, d + pad) if heads_first else (pages, page, kv_heads, d + pad)
    x = torch.full(shape, fill, dtype=torch.bfloat16, device=device())
    return (x.transpose(1, 2) if heads_first else x)[..., :d]


def values(rng, shape, std=1.0):
    return torch.from_numpy((rng.normal(size=shape) * std).astype(np.float32)).to(torch.bfloat16)


@pytest.mark.parametrize("tokens,kv_heads,d,page,heads_first,pad", [
    (1, 1, 64, 16, False, 0), (1, 16, 128, 16, True, 0), (7, 3, 64, 32, False, 8), (129, 8, 128, 64, True, 16),
    (1000, 2, 64, 16, False, 0), (2049, 5, 128, 128, True, 0)])
def test_store(ctx, tokens, kv_heads, d, page, heads_first, pad):
    rng = np.random.default_rng(tokens)
    pages = -(-tokens // page) + 3
    kp, vp = (pool(pages, page, kv_heads, d, heads_first, pad, 7.0) for _ in range(2))
    packed = values(rng, (tokens, 3 * kv_heads * d)).to(device())
    k = packed[:, kv_heads * d:2 * kv_heads * d].view(tokens, kv_heads, d)
    v = packed[:, 2 * kv_heads * d:].view(tokens, kv_heads, d)
    slots = rng.permutation(pages * page)[:tokens].astype(np.int64)
    slots[rng.random(tokens) < 0.2] = -1
    before = [x.float().cpu().numpy() for x in (kp, vp)]
    base = [x._base if x._base is not None else x for x in (kp, vp)]
    t.check(t.tp3d_paged_store(ctx, t.kv_cache(kp, vp), k, v, torch.from_numpy(slots).to(device())))
    assert t.tp3d_sync_status(ctx) == 0
    for x, b, new, whole in zip((kp, vp), before, (k, v), base):
        np.testing.assert_array_equal(x.float().cpu().numpy(), OP.store(b, new.float().cpu().numpy(), slots))
        if pad:
            assert bool((whole[..., d:] == 7.0).all())


def test_store_slot_past_the_pool(ctx):
    kp, vp = pool(2, 16, 1, 64, fill=1.0), pool(2, 16, 1, 64, fill=1.0)
    k = torch.full((3, 1, 64), 2.0, dtype=torch.bfloat16, device=device())
    slots = torch.tensor([3, 32, 2 ** 40], device=device())
    t.check(t.tp3d_paged_store(ctx, t.kv_cache(kp, vp), k, k, slots))
    assert t.tp3d_sync_status(ctx) == EPAGES and t.tp3d_sync_status(ctx) == 0
    assert bool((kp[0, 3] == 2).all()) and float(kp.float().sum()) == 64 * 33


def test_store_passes_bits_through(ctx):
    kp, vp = pool(1, 16, 1, 64, fill=0.0), pool(1, 16, 1, 64, fill=0.0)
    bits = torch.arange(16 * 64, dtype=torch.int32).mul(65).to(torch.int16).to(device()).view(16, 1, 64)
    k = bits.view(torch.bfloat16)
    t.check(t.tp3d_paged_store(ctx, t.kv_cache(kp, vp), k, k, torch.arange(15, -1, -1, device=device())))
    assert t.tp3d_sync_status(ctx) == 0
    assert torch.equal(kp.view(torch.int16)[0].flip(0), bits) and torch.equal(vp.view(torch.int16)[0].flip(0), bits)


# ------------------------------------------------------------------ attention
class Case:
    """A cache holding kv tokens per request in shuffled pages of a pool that
    is NaN everywhere else, table columns past a request's pages out of range."""

    def __init__(self, kv, new, heads, kv_heads, d, page=16, heads_first=False, pad=0, packed=True, std=1.0, seed=0,
                 extra_tokens=0, v_mean=0.0):
        rng = np.random.default_rng(seed)
        self.heads, self.kv_heads, self.d, self.page = heads, kv_heads, d, page
        self.kv, self.new = np.asarray(kv), np.asarray(new)
        requests = len(kv)
        need = [-(-max(int(n), 0) // page) for n in kv]
        width = max(max(need), 1) + 1
        pages = sum(need) + 2
        order = rng.permutation(pages)
        self.table = np.full((requests, width), 2 ** 30)
        kp, vp = pool(pages, page, kv_heads, d, heads_first, pad), pool(pages, page, kv_heads, d, heads_first, pad)
        at = 0
        for b, n in enumerate(need):
            self.table[b, :n] = order[at:at + n]
            at += n
            if kv[b] > 0:
                ids = torch.from_numpy(order[at - n:at].copy()).to(device())
                for p, mean in ((kp, 0.0), (vp, v_mean)):
                    rows = torch.full((n * page, kv_heads, d), float("nan"), dtype=torch.bfloat16)
                    rows[:kv[b]] = values(rng, (int(kv[b]), kv_heads, d)) + mean
                    p[ids] = rows.view(n, page, kv_heads, d).to(device())
        self.kp, self.vp = kp, vp
        self.q_start = np.concatenate([[0], np.cumsum(self.new)])
        self.tokens = int(self.q_start[-1]) + extra_tokens
        w = heads + 2 * kv_heads if packed else heads
        x = values(rng, (max(self.tokens, 1), w * d), std).to(device())
        self.q = x[:self.tokens, :heads * d].view(self.tokens, heads, d)
        self.cache = t.kv_cache(kp, vp)
        self.dev = (i32(self.q_start), i32(self.kv), i32(self.table))
        self.scale = d ** -0.5

    def batch(self, max_new=None):
        return t.paged_batch(*self.dev, self.tokens, int(max(self.new)) if max_new is None else max_new)

    def run(self, ctx, max_new=None, o=None, lse=True, stream=None):
        o = torch.full(self.q.shape, float("nan"), dtype=torch.bfloat16, device=device()) if o is None else o
        l = torch.full(self.q.shape[:2], float("nan"), device=device()) if lse else None
        n = t.tp3d_paged_attn_workspace_bytes(ctx, self.cache, self.heads)
        self.ws = torch.empty(n, dtype=torch.uint8, device=device())
        if stream is not None:
            stream.wait_stream(torch.cuda.current_stream())
        t.check(t.tp3d_paged_attn(ctx, self.cache, self.batch(max_new), self.q, o, l, self.scale, self.ws, stream))
        return o, l

    def want(self):
        return OP.attention(self.q.float().cpu().numpy(), self.kp.float().cpu().numpy(),
                            self.vp.float().cpu().numpy(), self.table, self.q_start, self.kv, self.scale)


def compare(c, o, l, want=None):
    wo, wl, absum, amax = c.want() if want is None else want
    n = int(c.q_start[-1])
    o, wo, wl, absum, amax = o.float().cpu().numpy().astype(np.float64)[:n], wo[:n], wl[:n], absum[:n], amax[:n]
    s = (2 * (c.d + 8) * E * amax + 2.0 ** -20)[..., None]
    tol = (U * np.abs(wo) + (U + s) * absum) * (1 + 2.0 ** -5) + 1e-30
    assert not np.isnan(o).any()
    bad = np.abs(o - wo) > tol
    assert not bad.any(), (np.argwhere(bad)[:5], o[bad][:5], wo[bad][:5])
    if l is not None:
        l = l.cpu().numpy().astype(np.float64)[:n]
        empty = np.isneginf(wl)
        assert np.array_equal(np.isneginf(l), empty)
        keys = float(max(int(x) for x in c.kv)) if len(c.kv) else 0.0
        tol = (c.d + 8) * E * amax + (keys + 64) * E + 2.0 ** -20 * (1 + np.abs(np.where(empty, 0, wl)))
        err = np.abs(np.where(empty, 0, l) - np.where(empty, 0, wl))
        assert (err <= tol).all(), (err / tol).max()


HEADS = [(1, 1), (4, 4), (8, 2), (6, 2), (14, 2), (16, 1), (48, 1), (128, 1)]


@pytest.mark.parametrize("heads,kv_heads", HEADS)
@pytest.mark.parametrize("d", [64, 128])
def test_single_tokens(ctx, heads, kv_heads, d):
    kv = [1, 2, 15, 16, 17, 63, 64, 65, 127, 128, 129, 700]
    c = Case(kv, [1] * len(kv), heads, kv_heads, d, seed=heads)
    o, l = c.run(ctx)
    assert t.tp3d_sync_status(ctx) == 0
    compare(c, o, l)


@pytest.mark.parametrize("page,heads_first,pad", [(16, True, 0), (32, False, 8), (64, True, 64), (128, False, 0),
                                                  (256, True, 0), (4096, False, 0)])
@pytest.mark.parametrize("new", [1, 5, 150])
def test_pages_and_strides(ctx, page, heads_first, pad, new):
    kv = [new, new + 1, 300, 511, 513]
    c = Case(kv, [min(new, k) for k in kv], 4, 2, 128, page, heads_first, pad, packed=new != 5, seed=page + new)
    o, l = c.run(ctx)
    assert t.tp3d_sync_status(ctx) == 0
    compare(c, o, l)


@pytest.mark.parametrize("heads,kv_heads", [(2, 2), (8, 2), (6, 2), (7, 1), (32, 1), (33, 1), (128, 1)])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("kv,new", [([130], [130]), ([257, 64], [2, 64]), ([400, 33], [131, 33]), ([65, 66], [65, 17])])
def test_chunks(ctx, heads, kv_heads, d, kv, new):
    c = Case(kv, new, heads, kv_heads, d, seed=sum(kv) + heads, v_mean=1.0)
    o, l = c.run(ctx)
    assert t.tp3d_sync_status(ctx) == 0
    compare(c, o, l)


@pytest.mark.parametrize("max_new", [None, 0, 10 ** 6])
def test_mixed_lengths_and_rows_without_keys(ctx, max_new):
    # requests with no new tokens, with more new tokens than keys (rows that see nothing), with no key at all
    kv = [500, 0, 3, 900, 77, 40, 0, 1, 260]
    new = [1, 0, 8, 300, 1, 100, 5, 1, 0]
    c = Case(kv, new, 8, 2, 64, 32, seed=4)
    o, l = c.run(ctx, max_new)
    assert t.tp3d_sync_status(ctx) == 0
    compare(c, o, l)
    n = c.q_start
    assert bool((o[n[2]:n[2] + 5] == 0).all()) and bool(torch.isneginf(l[n[2]:n[2] + 5]).all())
    assert bool((o[n[6]:n[7]] == 0).all()) and bool(torch.isneginf(l[n[6]:n[7]]).all())


def test_single_tokens_without_keys(ctx):
    c = Case([0, 20, 0], [1, 1, 1], 8, 2, 128)
    o, l = c.run(ctx)
    assert t.tp3d_sync_status(ctx) == 0
    compare(c, o, l)


@pytest.mark.parametrize("kv,new,heads,kv_heads", [
    ([9001], [1], 2, 1), ([5003], [1], 16, 16), ([4100], [130], 2, 1), ([3001, 1, 77], [1, 1, 1], 8, 8),
    ([6000], [3], 16, 1), ([2500, 2000], [129, 1], 4, 1)])
def test_work_split_along_the_keys(ctx, kv, new, heads, kv_heads):
    c = Case(kv, new, heads, kv_heads, 128, 64, seed=7)
    o, l = c.run(ctx)
    assert t.tp3d_sync_status(ctx) == 0
    compare(c, o, l)
    o2, l2 = c.run(ctx)
    assert torch.equal(o.view(torch.int16), o2.view(torch.int16)) and torch.equal(l, l2)


@pytest.mark.parametrize("new", [1, 140])
@pytest.mark.parametrize("std", [0.0, 8.0, 60.0])
def test_flat_and_sharply_peaked_scores(ctx, new, std):
    c = Case([600, 350], [new, new], 4, 1, 128, std=std, seed=9, v_mean=0.5)
    o, l = c.run(ctx)
    assert t.tp3d_sync_status(ctx) == 0
    compare(c, o, l)


@pytest.mark.parametrize("new", [1, 140])
def test_growing_scores(ctx, new):
    # the row maximum grows along the keys, by more and by less than the rescaling threshold
    c = Case([900], [new], 4, 1, 64, seed=11)
    c.q[:] = 1.0
    order = c.table[0, :-1].astype(np.int64)
    ramp = torch.linspace(-30, 30, 900).to(torch.bfloat16).to(device())
    for i, p in enumerate(order):
        n = min(16, 900 - 16 * i)
        c.kp[int(p), :n] = ramp[16 * i:16 * i + n, None, None]
    o, l = c.run(ctx)
    assert t.tp3d_sync_status(ctx) == 0
    compare(c, o, l)


@pytest.mark.parametrize("new", [1, 140])
def test_nan_and_infinite_values_stay_where_they_belong(ctx, new):
    # a NaN key and an infinite value in one head of one request: that head of that request only
    kv = [300, 300]
    c = Case(kv, [new, new], 4, 2, 64, seed=12)
    clean, _ = c.run(ctx)
    page, off = int(c.table[0, 200 // 16]), 200 % 16  # position 200 (new = 140: seen by the rows from 40 on)
    c.kp[page, off, 0] = float("nan")
    c.vp[page, off, 1] = float("inf")
    o, l = c.run(ctx)
    assert t.tp3d_sync_status(ctx) == 0
    n = c.q_start
    assert torch.equal(o[n[1]:], clean[n[1]:])
    sees = 0 if new == 1 else 40
    assert torch.equal(o[:sees], clean[:sees])
    assert bool(o[sees:n[1], :2].isnan().all())
    v = o[sees:n[1], 2:].float()
    assert bool((v.isinf() | v.isnan()).all()) and bool((c.kp[page, off, 0].isnan()).all())


def test_rows_past_the_requests_are_not_written(ctx):
    c = Case([40, 9], [3, 1], 4, 2, 64, extra_tokens=4)
    whole, flat = guarded(c.tokens * 4 * 64, torch.bfloat16)
    o = flat.view(c.tokens, 4, 64)
    o, l = c.run(ctx, o=o)
    assert t.tp3d_sync_status(ctx) == 0
    compare(c, o, l)
    assert bool(o[4:].isnan().all()) and bool(l[4:].isnan().all())
    assert_guards_intact(whole)


@pytest.mark.parametrize("new", [1, 140])
def test_strided_output_and_no_lse(ctx, new):
    c = Case([200, 333], [new, new], 6, 2, 128, seed=3)
    big = torch.full((8, c.tokens, 136), 3.0, dtype=torch.bfloat16, device=device())
    o = big.transpose(0, 1)[:, 1:7, :128]
    o, _ = c.run(ctx, o=o, lse=False)
    assert t.tp3d_sync_status(ctx) == 0
    compare(c, o, None)
    assert bool((big[0] == 3).all()) and bool((big[7] == 3).all()) and bool((big[:, :, 128:] == 3).all())


@pytest.mark.parametrize("new", [1, 140])
def test_bad_pages_and_lengths_stay_in_bounds(ctx, new):
    c = Case([300, 300], [new, new], 4, 2, 64, seed=5)
    good, _ = c.run(ctx)
    assert t.tp3d_sync_status(ctx) == 0
    for bad in (-1, c.kp.shape[0], 2 ** 31 - 1):
        table = c.table.copy()
        table[0, 3] = bad
        c.dev = (c.dev[0], c.dev[1], i32(table))
        o, _ = c.run(ctx)
        assert t.tp3d_sync_status(ctx) == EPAGES
        assert torch.equal(o[c.q_start[1]:], good[c.q_start[1]:])
    for kv in ([300, 10 ** 9], [-5, 300]):
        c.dev = (c.dev[0], i32(kv), i32(np.where(c.table > 10 ** 6, 0, c.table)))
        c.run(ctx)
        assert t.tp3d_sync_status(ctx) == EPAGES
    for qs in ([0, new, 10 ** 9], [-3, new, 2 * new], [new, 0, 2 * new]):
        c.dev = (i32(qs), i32([300, 300]), i32(c.table))
        c.run(ctx, max_new=0)
        assert t.tp3d_sync_status(ctx) == EPAGES
    assert t.tp3d_sync_status(ctx) == 0


def test_max_new_below_the_truth_is_reported(ctx):
    c = Case([300, 300], [1, 200], 4, 1, 64)
    o, l = c.run(ctx, max_new=1)
    assert t.tp3d_sync_status(ctx) == EPAGES
    wo, wl, ab, am = c.want()
    c.q_start = c.q_start[:2]
    compare(c, o, l, (wo, wl, ab, am))


def test_pool_past_32_bit_offsets(ctx):
    # pages whose element offsets pass 2^31 and 2^32; only the pages in use are written
    page, kv_heads, d = 16, 8, 128
    pages = (2 ** 32 // (page * kv_heads * d)) + 8
    kp, vp = (torch.empty(pages, page, kv_heads, d, dtype=torch.bfloat16, device=device()) for _ in range(2))
    small = Case([75], [75], 8, 8, d, page, seed=2)
    ids = [pages - 1, pages // 2 + 3, 5, pages - 9, 1]
    new = torch.tensor(ids, device=device())
    old = torch.from_numpy(small.table[0, :5].astype(np.int64)).to(device())
    kp[new], vp[new] = small.kp[old], small.vp[old]
    want = small.want()
    small.cache = t.kv_cache(kp, vp)
    for tokens in (75, 1):
        table = i32([ids + [0]])
        if tokens == 1:
            small.q, small.tokens, small.new, small.q_start = small.q[74:], 1, np.array([1]), np.array([0, 1])
            want = [x[74:] for x in want]
        small.dev = (i32(small.q_start), i32([75]), table)
        o, l = small.run(ctx)
        assert t.tp3d_sync_status(ctx) == 0
        compare(small, o, l, want)
    k = values(np.random.default_rng(1), (2, kv_heads, d)).to(device())
    slots = torch.tensor([pages * page - 1, (pages - 9) * page + 4], device=device())
    t.check(t.tp3d_paged_store(ctx, small.cache, k, k, slots))
    assert t.tp3d_sync_status(ctx) == 0
    assert torch.equal(kp[pages - 1, 15], k[0]) and torch.equal(vp[pages - 9, 4], k[1])


@pytest.mark.parametrize("new", [1, 140])
def test_other_stream_and_graph_replay(ctx, new):
    c = Case([500, 400], [new, new], 8, 2, 128, seed=6)
    want, _ = c.run(ctx)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    o, l = c.run(ctx, stream=side)
    assert t.tp3d_sync_status(ctx, side) == 0
    assert torch.equal(o, want)
    # captured once, replayed with other lengths in the same buffers
    o = torch.zeros_like(o)
    g = torch.cuda.CUDAGraph()
    batch = c.batch()
    with torch.cuda.graph(g):
        t.check(t.tp3d_paged_attn(ctx, c.cache, batch, c.q, o, l, c.scale, c.ws))
    for kv in ([500, 400], [499, 230], [new, 400]):
        c.kv = np.asarray(kv)
        c.dev[1].copy_(i32(kv))
        g.replay()
        assert t.tp3d_sync_status(ctx) == 0
        compare(c, o, l)


def test_a_step_end_to_end(ctx):
    # plan -> store -> attention over several steps, the cache filled by the operators alone
    rng = np.random.default_rng(8)
    page, requests, heads, kv_heads, d, width = 16, 5, 8, 4, 64, 12
    pages = requests * width
    kp, vp = pool(pages, page, kv_heads, d), pool(pages, page, kv_heads, d)
    cache = t.kv_cache(kp, vp)
    free = i32(rng.permutation(pages))
    count, cached, table = i32([pages]), i32([0] * requests), i32(np.full((requests, width), -1))
    have = np.zeros(requests, dtype=np.int64)
    for fresh in ([40, 1, 17, 0, 64], [1] * requests, [1] * requests, [0, 70, 1, 3, 0], [1] * requests):
        tokens = sum(fresh) + 2
        q_start, kv_len, left = i32([0] * (requests + 1)), i32([0] * requests), i32([0])
        slots = torch.zeros(tokens, dtype=torch.int64, device=device())
        pos = i32([0] * tokens)
        t.check(t.tp3d_paged_plan(ctx, page, requests, tokens, cached, i32(fresh), free, pages, count, table, width,
                                  q_start, kv_len, slots, pos, left))
        x = values(rng, (tokens, (heads + 2 * kv_heads) * d)).to(device())
        q, k, v = (y.view(tokens, -1, d) for y in x.split([heads * d, kv_heads * d, kv_heads * d], 1))
        t.check(t.tp3d_paged_store(ctx, cache, k, v, slots))
        o, l = torch.zeros(tokens, heads, d, dtype=torch.bfloat16, device=device()), torch.zeros(tokens, heads, device=device())
        ws = torch.empty(t.tp3d_paged_attn_workspace_bytes(ctx, cache, heads), dtype=torch.uint8, device=device())
        t.check(t.tp3d_paged_attn(ctx, cache, t.paged_batch(q_start, kv_len, table, tokens, max(fresh)), q, o, l,
                                  d ** -0.5, ws))
        assert t.tp3d_sync_status(ctx) == 0
        have += np.asarray(fresh)
        np.testing.assert_array_equal(kv_len.cpu().numpy(), have)
        c = Case.__new__(Case)
        c.q, c.kp, c.vp, c.table, c.d, c.scale = q, kp, vp, table.cpu().numpy(), d, d ** -0.5
        c.q_start, c.kv, c.new = q_start.cpu().numpy(), have, np.asarray(fresh)
        compare(c, o, l)
        cached, count = kv_len, left


@pytest.mark.parametrize("heads,kv_heads,new", [(4, 2, 5), (16, 2, 2), (1, 1, 16), (1, 1, 17), (8, 1, 3), (2, 2, 64)])
@pytest.mark.parametrize("d", [64, 128])
def test_short_chunks(ctx, heads, kv_heads, new, d):
    # a few tokens each, on both sides of the row count where the kernel changes; some rows see nothing
    kv = [new, 1, new + 70, 515, 2]
    c = Case(kv, [new] * 5, heads, kv_heads, d, 16, True, seed=new * heads, v_mean=0.5)
    o, l = c.run(ctx)
    assert t.tp3d_sync_status(ctx) == 0
    compare(c, o, l)


@pytest.mark.parametrize("requests", [127, 129, 385, 1000])
@pytest.mark.parametrize("long_every", [0, 7])
def test_many_requests(ctx, requests, long_every):
    # more requests than a CTA looks at in one round; some idle, some with many rows
    rng = np.random.default_rng(requests)
    kv = rng.integers(1, 40, requests)
    new = (rng.random(requests) < 0.8).astype(np.int64)
    if long_every:
        new[3::long_every] = np.minimum(kv[3::long_every], 20)
    c = Case(kv, new, 4, 1, 64, seed=requests)
    o, l = c.run(ctx)
    assert t.tp3d_sync_status(ctx) == 0
    compare(c, o, l)


@pytest.mark.parametrize("new", [3, 9, 140])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("value", [float("nan"), float("inf"), float("-inf")])
def test_values_that_are_not_finite_in_masked_places(ctx, new, d, value):
    # in the values of later tokens of the chunk: rows before them are what they are without them, bit for bit
    kv = [260, new, 333]
    c = Case(kv, [new] * 3, 4, 2, d, seed=13)
    clean, cl = c.run(ctx)
    at = [(0, 260 - new + new // 2, 0, 3), (0, 259, 1, d - 1), (1, new - 1, 0, 17), (2, 333 - new + 1, 1, 40)]
    for b, pos, head, col in at:
        c.vp[int(c.table[b, pos // 16]), pos % 16, head, col] = value
    o, l = c.run(ctx)
    assert t.tp3d_sync_status(ctx) == 0
    assert torch.equal(l, cl)
    hit = torch.zeros_like(o, dtype=torch.bool)
    for b, pos, head, col in at:
        first = int(c.q_start[b]) + pos - (kv[b] - new)  # the token at that position sees it, as all after it
        hit[first:int(c.q_start[b + 1]), 2 * head:2 * head + 2, col] = True
    assert torch.equal(o[~hit], clean[~hit])
    assert not bool(o[hit].isfinite().any())


def test_values_that_are_not_finite_in_split_work(ctx):
    # the same where the last keys are one CTA's part of a row and the first ones another's
    for new, heads, kv_heads in ((4, 4, 1), (150, 2, 1)):
        c = Case([5000], [new], heads, kv_heads, 128, 64, seed=14)
        clean, _ = c.run(ctx)
        pos = 5000 - new // 2
        c.vp[int(c.table[0, pos // 64]), pos % 64, 0, 5] = float("nan")
        o, _ = c.run(ctx)
        assert t.tp3d_sync_status(ctx) == 0
        sees = pos - (5000 - new)
        hit = torch.zeros_like(o, dtype=torch.bool)
        hit[sees:, :, 5] = True
        assert torch.equal(o[~hit], clean[~hit]) and bool(o[hit].isnan().all())


@pytest.mark.parametrize("d", [64, 128])
def test_no_store_outside_the_output(ctx, d):
    c = Case([300, 40, 1], [200, 17, 1], 4, 2, d, extra_tokens=3)
    whole, flat = guarded(c.tokens * 4 * d, torch.bfloat16)
    o, l = c.run(ctx, o=flat.view(c.tokens, 4, d))
    assert t.tp3d_sync_status(ctx) == 0
    compare(c, o, l)
    assert bool(o[218:].isnan().all()) and bool(l[218:].isnan().all())
    assert_guards_intact(whole)


# ------------------------------------------------------------------ refusals
def test_refusals(ctx):
    EINVAL, ESHAPE, EALIGN, EDTYPE, EUNSUP, EOVER = 1, 2, 3, 4, 7, 8
    c = Case([40], [1], 4, 2, 64)
    ws = torch.empty(t.tp3d_paged_attn_workspace_bytes(ctx, c.cache, 4) + 256, dtype=torch.uint8, device=device())
    o = torch.empty(c.q.shape, dtype=torch.bfloat16, device=device())
    lib = t.lib()
    import ctypes

    def attn(cache=c.cache, batch=None, heads=4, scale=1.0, q=c.q.data_ptr(), qs=(512, 64), out=o.data_ptr(),
             os_=(256, 64), lse=None, w=ws.data_ptr(), x=ctx):
        b = c.batch() if batch is None else batch
        return lib.tp3d_paged_attn(x, ctypes.byref(cache), ctypes.byref(b), heads, scale, q, t.tp3d_row_strides(*qs),
                                   out, t.tp3d_row_strides(*os_), lse, w, None)

    def cache(**kw):
        x = t.tp3d_kv_cache.from_buffer_copy(c.cache)
        for k, v in kw.items():
            setattr(x, k, v)
        return x

    def batch(**kw):
        x = c.batch()
        for k, v in kw.items():
            setattr(x, k, v)
        return x

    assert attn() == 0
    assert attn(x=None) == EINVAL and attn(q=None) == EINVAL and attn(out=None) == EINVAL and attn(w=None) == EINVAL
    assert attn(cache(k=None)) == EINVAL and attn(cache(pages=0)) == EINVAL and attn(cache(kv_heads=0)) == EINVAL
    assert attn(cache(dtype=0)) == EDTYPE
    assert attn(cache(head_dim=96)) == EUNSUP and attn(cache(page=24)) == EUNSUP and attn(cache(page=8)) == EUNSUP
    assert attn(cache(k=c.kp.data_ptr() + 2)) == EALIGN and attn(cache(token_stride=68)) == EALIGN
    assert attn(cache(page_stride=0)) == EINVAL
    assert attn(heads=3) == ESHAPE and attn(heads=0) == EINVAL and attn(cache(kv_heads=1), heads=129) == EUNSUP
    for s in (0.0, -1.0, float("nan"), float("inf")):
        assert attn(scale=s) == EINVAL
    assert attn(qs=(516, 64)) == EALIGN and attn(q=c.q.data_ptr() + 8) == EALIGN and attn(qs=(0, 64)) == EINVAL
    assert attn(os_=(256, 68)) == EALIGN and attn(w=ws.data_ptr() + 16) == EALIGN and attn(lse=ws.data_ptr() + 2) == EALIGN
    assert attn(out=c.q.data_ptr()) == EOVER and attn(out=c.kp.data_ptr()) == EOVER and attn(w=o.data_ptr()) == EOVER
    assert attn(batch=batch(requests=-1)) == EINVAL and attn(batch=batch(kv_len=None)) == EINVAL
    assert attn(batch=batch(block_table=None)) == EINVAL and attn(batch=batch(tokens=-1)) == EINVAL
    assert attn(batch=batch(requests=0)) == 0 and attn(batch=batch(tokens=0)) == 0
    assert t.tp3d_paged_attn_workspace_bytes(ctx, cache(head_dim=32), 4) == 0
    assert t.tp3d_paged_attn_workspace_bytes(ctx, c.cache, 3) == 0

    def store(cc=c.cache, n=1, k=c.q.data_ptr(), ts=512, hs=64, s=ws.data_ptr(), x=ctx):
        return lib.tp3d_paged_store(x, ctypes.byref(cc), n, k, k, ts, hs, s, None)
    ws.zero_()
    assert store(n=0) == 0 and store(n=-1) == EINVAL and store(x=None) == EINVAL and store(k=None) == EINVAL
    assert store(s=None) == EINVAL and store(s=ws.data_ptr() + 4) == EALIGN and store(ts=12) == EALIGN
    assert store(k=c.kp.data_ptr()) == EOVER and store(cache(dtype=0)) == EDTYPE and store(hs=-64) == EINVAL

    buf = torch.zeros(4096, dtype=torch.int32, device=device())
    p = [buf.data_ptr() + 256 * i for i in range(16)]

    def plan(page=16, n=2, tokens=4, cap=4, width=3, x=ctx, **kw):
        a = [p[0], p[1], p[2], cap, p[3], p[4], width, p[5], p[6], p[7], p[8], p[9]]
        for k, v in kw.items():
            a[int(k[1:])] = v
        return lib.tp3d_paged_plan(x, page, n, tokens, *a, None)
    assert plan() == 0
    assert plan(x=None) == EINVAL and plan(n=-1) == EINVAL and plan(tokens=-1) == EINVAL and plan(cap=-1) == EINVAL
    assert plan(page=17) == EUNSUP and plan(page=8192) == EUNSUP and plan(n=16385) == EUNSUP
    for i in (0, 1, 2, 4, 5, 7, 8, 9, 10, 11):
        assert plan(**{f"a{i}": None}) == EINVAL, i
    assert plan(a0=p[0] + 2) == EALIGN and plan(a9=p[7] + 4) == EALIGN
    assert plan(a8=p[0]) == EOVER and plan(a11=p[3]) == EOVER and plan(a7=p[6]) == EOVER
    t.tp3d_sync_status(ctx)
    with pytest.raises(ValueError):
        t.kv_cache(c.kp, c.vp[:1])
    with pytest.raises(ValueError):
        t.kv_cache(c.kp[..., ::2], c.vp[..., ::2])
    with pytest.raises(ValueError):
        t.paged_batch(c.dev[0], c.dev[1].long(), c.dev[2], 1)
    with pytest.raises(ValueError):
        t.tp3d_paged_attn(ctx, c.cache, c.batch(), c.q.float(), o.float(), None, 1.0, ws)
    with pytest.raises(ValueError):
        t.tp3d_paged_store(ctx, c.cache, c.q, c.q, torch.zeros(1, dtype=torch.int64, device=device()))


@pytest.mark.parametrize("kv,new,heads,d", [
    # items in two and three parts, CTAs whose range goes on behind one, and items in many parts
    ([9000, 7000, 8000], [200, 130, 256], 8, 128), ([4000, 900, 3000, 600], [700, 120, 900, 64], 12, 64),
    ([20000, 300], [64, 140], 2, 64)])
def test_order_of_arrival_does_not_change_the_result(ctx, kv, new, heads, d):
    c = Case(kv, new, heads, heads, d, 64, seed=heads)
    o, l = c.run(ctx)
    assert t.tp3d_sync_status(ctx) == 0
    compare(c, o, l)
    # long blocks beside it hold a good part of the SMs: CTAs start after the ones before them have ended
    x = torch.rand(140, 1 << 22, device=device())
    side = torch.cuda.Stream()
    for i in range(24):
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            x[:20 * (i % 8)].softmax(1)
        o2, l2 = c.run(ctx)
        assert torch.equal(o.view(torch.int16), o2.view(torch.int16)) and torch.equal(l, l2)
    assert t.tp3d_sync_status(ctx) == 0


@pytest.mark.parametrize("heads,kv_heads,new", [(4, 2, 5), (16, 2, 2), (1, 1, 16), (8, 1, 2), (14, 2, 1), (3, 3, 1)])
@pytest.mark.parametrize("d", [64, 128])
def test_few_rows_of_many_requests(ctx, heads, kv_heads, new, d):
    # enough of them for every SM; lengths at the tiles' edges, one long enough to be split
    kv = [1, 2, 15, 16, 17, 63, 64, 65, 127, 128, 129, 255, 257, 300, new, new + 1] * 10 + [6000]
    c = Case(kv, [new] * len(kv), heads, kv_heads, d, 32, seed=heads + new)
    o, l = c.run(ctx)
    assert t.tp3d_sync_status(ctx) == 0
    compare(c, o, l)
    if new == 1:
        return
    # a value that is not finite in a masked place changes the rows that see its key, and no other
    b = next(i for i, n in enumerate(kv) if n == 257)
    pos = 257 - new + new // 2
    c.vp[int(c.table[b, pos // 32]), pos % 32, kv_heads - 1, 9] = float("inf")
    got, _ = c.run(ctx)
    assert t.tp3d_sync_status(ctx) == 0
    hit = torch.zeros_like(o, dtype=torch.bool)
    group = heads // kv_heads
    hit[int(c.q_start[b]) + new // 2:int(c.q_start[b + 1]), heads - group:, 9] = True
    assert torch.equal(got[~hit], o[~hit]) and not bool(got[hit].isfinite().any())


@pytest.mark.parametrize("heads,kv_heads,new", [(8, 2, 11), (8, 2, 12), (6, 2, 16), (6, 2, 17), (32, 1, 1), (48, 1, 1),
                                                (7, 1, 5), (33, 1, 1)])
@pytest.mark.parametrize("d", [64, 128])
def test_more_rows_than_one_block(ctx, heads, kv_heads, new, d):
    # rows of a token in two blocks; on both sides of the row count where the kernel changes; split and short items
    kv = [5000, new, 300, 128, 129, 1]
    c = Case(kv, [new] * 6, heads, kv_heads, d, 64, True, seed=heads * new, v_mean=0.5)
    o, l = c.run(ctx)
    assert t.tp3d_sync_status(ctx) == 0
    compare(c, o, l)
    o2, l2 = c.run(ctx)
    assert torch.equal(o.view(torch.int16), o2.view(torch.int16)) and torch.equal(l, l2)
    if new == 1:
        return
    # a value that is not finite in a masked place changes the rows that see its key, and no other
    for b, n in ((0, 5000), (2, 300)):
        pos = n - new + new // 2
        c.vp[int(c.table[b, pos // 64]), pos % 64, kv_heads - 1, 7] = float("nan")
    got, _ = c.run(ctx)
    assert t.tp3d_sync_status(ctx) == 0
    hit = torch.zeros_like(o, dtype=torch.bool)
    for b in (0, 2):
        hit[int(c.q_start[b]) + new // 2:int(c.q_start[b + 1]), heads - heads // kv_heads:, 7] = True
    assert torch.equal(got[~hit], o[~hit]) and bool(got[hit].isnan().all())


@pytest.mark.parametrize("new", [1, 3, 90])
def test_steps_that_follow_each_other_at_once(ctx, new):
    # each call reads what the one before it writes (lengths, free count, table, slots, cache, then its output as the
    # next step's input): back to back they give what they give with the stream drained between any two
    page, requests, heads, kv_heads, d, steps = 16, 40, 4, 2, 64, 12
    width = -(-new * steps // page)
    pages, tokens = requests * width, requests * new
    fresh, order = i32([new] * requests), np.random.default_rng(new).permutation(pages)
    free = i32(order)
    x0 = values(np.random.default_rng(9), (tokens, heads, d)).to(device())

    def run(drain):
        kp, vp = pool(pages, page, kv_heads, d), pool(pages, page, kv_heads, d)
        cache = t.kv_cache(kp, vp)
        table = i32(np.full((requests, width), -1))
        lens = [i32([0] * requests) for _ in range(steps + 1)]
        left = [i32([pages]) for _ in range(steps + 1)]
        q_start, pos = i32([0] * (requests + 1)), i32([0] * tokens)
        slots = torch.full((tokens,), -1, dtype=torch.int64, device=device())
        x = [x0] + [torch.zeros_like(x0) for _ in range(steps)]
        l = [torch.zeros(tokens, heads, device=device()) for _ in range(steps)]
        ws = torch.empty(t.tp3d_paged_attn_workspace_bytes(ctx, cache, heads), dtype=torch.uint8, device=device())
        torch.cuda.synchronize()
        for i in range(steps):
            for call in (
                    lambda: t.tp3d_paged_plan(ctx, page, requests, tokens, lens[i], fresh, free, pages, left[i], table,
                                              width, q_start, lens[i + 1], slots, pos, left[i + 1]),
                    lambda: t.tp3d_paged_store(ctx, cache, x[i][:, :kv_heads], x[i][:, kv_heads:], slots),
                    lambda: t.tp3d_paged_attn(ctx, cache, t.paged_batch(q_start, lens[i + 1], table, tokens, new), x[i],
                                              x[i + 1], l[i], 1.0, ws)):
                t.check(call())
                if drain:
                    torch.cuda.synchronize()
        assert t.tp3d_sync_status(ctx) == 0
        return [table, *lens, *left, *(y.view(torch.int16) for y in x), *l]

    want = run(True)
    for _ in range(3):
        for got, w in zip(run(False), want):
            assert torch.equal(got, w)

"""The operators of a server of long conversations, one after the other as they
are used: plan, norm and rotation with the store, attention over a window,
pages given back behind it, forks, requests that end, and compaction.  Each
step's rows are held to the float64 oracle on what the requests have said so
far; tolerances are those of test_gpu_rope.py and test_gpu_paged.py."""
import numpy as np
import pytest
import torch

import tensor_transformer_layer_cube_gb300 as t
from oracle import paged as OP
from oracle import rope as OR
from tests.gpu_util import device
from tests.test_gpu_paged import compare, i32, pool, values

pytestmark = pytest.mark.gpu

E = 2.0 ** -24


@pytest.fixture(scope="module")
def ctx():
    c = t.tp3d_create(0)
    yield c
    t.tp3d_destroy(c)


class Server:
    """``rows`` requests at most over ``pages`` pages; what each request has in the cache is kept on the host, too."""

    def __init__(self, ctx, rows, pages, width, page, heads, kv_heads, d, window, sinks, inter):
        self.ctx, self.rows, self.pages, self.width, self.page = ctx, rows, pages, width, page
        self.heads, self.kv_heads, self.d, self.window, self.sinks, self.inter = heads, kv_heads, d, window, sinks, inter
        self.rng = np.random.default_rng(page + window)
        self.kp, self.vp = pool(pages, page, kv_heads, d), pool(pages, page, kv_heads, d)
        self.cache = t.kv_cache(self.kp, self.vp)
        self.table, self.shares = i32(np.full((rows, width), -1)), i32(np.zeros(pages))
        self.free = i32(self.rng.permutation(pages))
        self.pool = t.page_pool(page, self.table, self.shares, self.free)
        self.count, self.kv = i32([pages]), np.zeros(rows, dtype=np.int64)
        self.past = [np.zeros((2, 0, kv_heads, d)) for _ in range(rows)]
        self.words, self.magnitude = OR.turns(d // 2, kind="parts", factor=4.0, context=64.0)
        self.turns = torch.tensor(self.words, dtype=torch.int64).to(device())
        self.qw, self.kw = ((1 + values(self.rng, (d,)) / 4).to(torch.bfloat16).to(device()) for _ in range(2))
        self.rope = t.rope(self.turns, torch.bfloat16, d, d // 2, inter, self.magnitude, True, 1e-5, self.qw, self.kw)
        self.ws = torch.empty(t.tp3d_paged_attn_workspace_bytes(ctx, self.cache, heads), dtype=torch.uint8, device=device())

    def step(self, fresh, pad=3):
        fresh = np.asarray(fresh)
        n = int(fresh.sum())
        tokens, h, kh, d = n + pad, self.heads, self.kv_heads, self.d
        q_start, kv_len, left = i32([0] * (self.rows + 1)), i32([0] * self.rows), i32([0])
        slots, pos = torch.zeros(tokens, dtype=torch.int64, device=device()), i32([0] * tokens)
        x = values(self.rng, (tokens, (h + 2 * kh) * d)).to(device())
        q, k, v = x[:, :h * d].view(tokens, h, d), x[:, h * d:(h + kh) * d].view(tokens, kh, d), x[:, (h + kh) * d:].view(tokens, kh, d)
        q0, k0, v0 = (y.double().cpu().numpy() for y in (q, k, v))
        o = torch.full((tokens, h, d), float("nan"), dtype=torch.bfloat16, device=device())
        l = torch.full((tokens, h), float("nan"), device=device())
        t.check(t.tp3d_paged_plan(self.ctx, self.page, self.rows, tokens, i32(self.kv), i32(fresh), self.free, self.pages,
                                  self.count, self.table, self.width, q_start, kv_len, slots, pos, left))
        t.check(t.tp3d_paged_rope_store(self.ctx, self.rope, self.cache, q, k, v, pos, slots, q))
        t.check(t.tp3d_paged_attn_window(self.ctx, self.cache, t.paged_batch(q_start, kv_len, self.table, tokens, int(max(fresh))),
                                         q, o, l, d ** -0.5, self.window, self.sinks, self.ws))
        assert t.tp3d_sync_status(self.ctx) == 0
        self.count = left
        starts = np.concatenate([[0], np.cumsum(fresh)])
        where = np.concatenate([np.arange(c, c + f) for c, f in zip(self.kv, fresh)]).astype(np.int64)
        np.testing.assert_array_equal(pos.cpu().numpy()[:n], where)
        self.rotated(q[:n], q0[:n], where, self.qw)
        s = slots[:n]
        stored = [p[s // self.page, s % self.page] for p in (self.kp, self.vp)]
        self.rotated(stored[0], k0[:n], where, self.kw)
        np.testing.assert_array_equal(stored[1].double().cpu().numpy(), v0[:n])
        new = np.stack([y.double().cpu().numpy() for y in stored])
        for r in range(self.rows):
            self.past[r] = np.concatenate([self.past[r], new[:, starts[r]:starts[r + 1]]], 1)
        self.kv = self.kv + fresh
        self.attended(q, o, l, starts)

    def rotated(self, got, x, where, w):
        w = w.double().cpu().numpy()
        eps = float(np.float32(1e-5))
        want = OR.forward(x, self.words, where, self.inter, self.magnitude, True, eps, w)
        n = OR.spread(x * OR.inverse_rms(x, eps) * w, self.words, self.inter, self.magnitude)
        tol = 2.0 ** -8 * np.abs(want) + 24 * E * n
        assert (np.abs(got.double().cpu().numpy() - want) <= tol * (1 + 2.0 ** -6)).all()

    def attended(self, q, o, l, starts):
        # each request's past in pages of its own, in order
        need = [-(-int(n) // self.page) for n in self.kv]
        dense = np.zeros((2, sum(need) + 1, self.page, self.kv_heads, self.d))
        table, at = np.zeros((self.rows, max(need) + 1), dtype=np.int64), 0
        for r, n in enumerate(need):
            flat = dense[:, at:at + n].reshape(2, n * self.page, self.kv_heads, self.d)
            flat[:, :self.kv[r]] = self.past[r]
            table[r, :n] = np.arange(at, at + n)
            at += n

        class C:
            d, kv, q_start = self.d, self.kv, starts
        want = OP.attention(q.double().cpu().numpy(), *dense, table, starts, self.kv, self.d ** -0.5, self.window, self.sinks)
        compare(C, o, l, want)

    def give_back(self, first, end):
        left = i32([0])
        t.check(t.tp3d_paged_free(self.ctx, self.pool, i32(first), i32(end), self.count, left))
        self.count = left

    def behind_the_window(self):
        # the next token of a request sees nothing between its first tokens and its window
        low = np.maximum(0, self.kv - self.window + 1)
        first = np.minimum(-(-self.sinks // self.page), -(-self.kv // self.page))
        self.give_back(first, np.maximum(first, low // self.page))

    def end(self, r):
        self.give_back([0] * self.rows, [-(-int(n) // self.page) if x == r else 0 for x, n in enumerate(self.kv)])
        self.kv[r], self.past[r] = 0, self.past[r][:, :0]

    def fork(self, src, dst):
        n, left, count = len(src), i32([0]), i32([0])
        at, to = i32([0] * n), i32([0] * n)
        t.check(t.tp3d_paged_fork(self.ctx, self.pool, i32(src), i32(dst), i32(self.kv[src]), self.count, left, at, to, count))
        t.check(t.tp3d_paged_copy(self.ctx, self.cache, n, at, to, count))
        self.count = left
        for a, b in zip(src, dst):
            self.kv[b], self.past[b] = self.kv[a], self.past[a].copy()

    def compact(self):
        at, to, count, where = i32([0] * (self.pages // 2)), i32([0] * (self.pages // 2)), i32([0]), i32([0] * self.pages)
        t.check(t.tp3d_paged_compact(self.ctx, self.pool, i32(self.kv), self.count, where, at, to, count))
        t.check(t.tp3d_paged_copy(self.ctx, self.cache, self.pages // 2, at, to, count))
        used = self.pages - int(self.count)
        # whatever lies past the used pages can go
        self.kp[used:], self.vp[used:] = float("nan"), float("nan")

    def check_books(self):
        assert t.tp3d_sync_status(self.ctx) == 0
        table, shares = self.table.cpu().numpy(), self.shares.cpu().numpy()
        named = np.zeros(self.pages, dtype=np.int64)
        for r in range(self.rows):
            row = table[r, :-(-int(self.kv[r]) // self.page)]
            np.add.at(named, row[row >= 0], 1)
        free = self.free.cpu().numpy()[:int(self.count)]
        assert len(set(free)) == len(free) and not named[free].any()
        assert int((named > 0).sum()) + len(free) == self.pages  # no page is lost
        np.testing.assert_array_equal(np.where(named > 0, named - 1, 0), shares)


@pytest.mark.parametrize("page,heads,kv_heads,d,window,sinks,inter", [
    (16, 4, 2, 64, 40, 5, False), (16, 8, 1, 64, 33, 0, True), (32, 6, 2, 128, 100, 40, False)])
def test_long_conversations(ctx, page, heads, kv_heads, d, window, sinks, inter):
    s = Server(ctx, 8, 160 if page == 16 else 90, 40, page, heads, kv_heads, d, window, sinks, inter)
    s.step([120, 7, 0, 65, 33, 0, 0, 0])
    s.behind_the_window()
    s.step([1, 1, 40, 1, 1, 0, 0, 0])
    s.fork([0, 0, 3], [5, 6, 7])
    s.check_books()
    s.step([1, 1, 1, 1, 1, 1, 30, 1])
    s.behind_the_window()
    s.end(0)
    s.check_books()
    s.compact()
    s.check_books()
    s.step([17, 100, 1, 1, 0, 2, 1, 50])
    s.behind_the_window()
    s.end(3)
    s.fork([7], [3])
    s.end(7)
    s.step([1] * 8)
    s.compact()
    s.behind_the_window()
    s.step([0, 1, 1, 90, 1, 1, 1, 0])
    for r in range(8):
        s.end(r)
    s.check_books()
    assert int(s.count) == s.pages


def test_two_servers_at_once(ctx):
    # a context each, on streams of their own: what they say is what each says alone
    other = t.tp3d_create(0)
    try:
        shape = (8, 160, 40, 16, 4, 2, 64, 40, 5, False)
        alone = Server(ctx, *shape)
        pair = [Server(ctx, *shape), Server(other, *shape)]
        streams = [torch.cuda.Stream() for _ in pair]
        torch.cuda.synchronize()
        n, h, kh, d = 3000, alone.heads, alone.kv_heads, alone.d
        rng = np.random.default_rng(3)
        x = values(rng, (n, (h + kh) * d)).to(device())
        g = values(rng, (n, (h + kh) * d)).to(device())
        pos = i32(rng.integers(0, 5000, n))

        class Work:
            # gradients, whose sums share the context's words, then pages taken and given back
            def __init__(self, s):
                self.s = s
                self.q, self.k = x[:, :h * d].view(n, h, d), x[:, h * d:].view(n, kh, d)
                self.gq, self.gk = g[:, :h * d].view(n, h, d), g[:, h * d:].view(n, kh, d)
                self.dq, self.dk = torch.empty_like(self.q.contiguous()), torch.empty_like(self.k.contiguous())
                self.dw = [torch.empty(d, dtype=torch.bfloat16, device=device()) for _ in range(2)]
                self.ws = torch.empty(t.tp3d_qk_rope_bwd_workspace_bytes(s.ctx, s.rope), dtype=torch.uint8, device=device())
                self.zero, self.fresh, self.ends = i32([0] * 8), i32([80] * 8), i32([5] * 8)
                self.q_start, self.kv, self.at = i32([0] * 9), i32([0] * 8), i32([0] * 640)
                self.slots, self.left = torch.zeros(640, dtype=torch.int64, device=device()), [i32([0]) for _ in range(2)]

            def step(self, stream):
                s = self.s
                t.check(t.tp3d_qk_rope_bwd(s.ctx, s.rope, self.q, self.k, pos, self.gq, self.gk, self.dq, self.dk, *self.dw,
                                           self.ws, stream))
                t.check(t.tp3d_paged_plan(s.ctx, s.page, 8, 640, self.zero, self.fresh, s.free, s.pages, s.count, s.table,
                                          s.width, self.q_start, self.kv, self.slots, self.at, self.left[0], stream))
                t.check(t.tp3d_paged_free(s.ctx, s.pool, self.zero, self.ends, self.left[0], self.left[1], stream))

            def said(self):
                return [self.dq, self.dk, *self.dw, self.s.free, self.s.shares, self.s.table, self.left[1]]

        one, both = Work(alone), [Work(s) for s in pair]
        for _ in range(20):
            one.step(torch.cuda.current_stream())
        want = one.said()
        torch.cuda.synchronize()
        for _ in range(20):
            for w, stream in zip(both, streams):
                w.step(stream)
        torch.cuda.synchronize()
        got = [w.said() for w in both]
        for s in pair:
            assert t.tp3d_sync_status(s.ctx) == 0
        for one in got:
            for a, b in zip(one, want):
                assert torch.equal(a, b)
        assert int(want[-1]) == alone.pages
    finally:
        t.tp3d_destroy(other)

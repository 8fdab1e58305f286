"""Forking, giving back, compacting and copying the cache's pages on the GPU
against the oracle: whole numbers and copied bits, all equal."""
import numpy as np
import pytest
import torch

import tensor_transformer_layer_cube_gb300 as t
from oracle import pages as OG
from tests.gpu_util import assert_guards_intact, device, guarded
from tests.test_gpu_paged import i32

pytestmark = pytest.mark.gpu

EPAGES = 10


@pytest.fixture(scope="module")
def ctx():
    c = t.tp3d_create(0)
    yield c
    t.tp3d_destroy(c)


def host(x):
    return x.cpu().numpy().astype(np.int64)


class Book:
    """Bookkeeping between guard bands, from arrays of the host."""

    def __init__(self, page, table, shares, free, count):
        self.page, self.host = page, [np.asarray(x) for x in (table, shares, free)] + [count]
        self.whole, self.dev = [], []
        for x in self.host[:3]:
            w, flat = guarded(x.size, torch.int32)
            flat.copy_(torch.as_tensor(x.reshape(-1), dtype=torch.int32))
            self.whole.append(w)
            self.dev.append(flat.view(x.shape))
        self.table, self.shares, self.free = self.dev
        self.count, self.left = i32([count]), i32([-7])
        self.pool = t.page_pool(page, *self.dev)
        self.lists = [guarded(len(shares) // 2, torch.int32) for _ in range(2)]
        self.copies = i32([-7])

    def intact(self):
        for w in self.whole + [w for w, _ in self.lists]:
            assert_guards_intact(w)

    def fork(self, ctx, src, dst, length, stream=None):
        n = len(src)
        self.pairs = [guarded(n, torch.int32) for _ in range(2)]
        at, to = (x for _, x in self.pairs)
        t.check(t.tp3d_paged_fork(ctx, self.pool, i32(src), i32(dst), i32(length), self.count, self.left, at, to,
                                  self.copies, stream))
        return at, to

    def check_fork(self, ctx, src, dst, length):
        at, to = self.fork(ctx, src, dst, length)
        sync = t.tp3d_sync_status(ctx)
        table, shares, left, copies, fits = OG.fork(self.page, *self.host, src, dst, length)
        np.testing.assert_array_equal(host(self.table), table)
        np.testing.assert_array_equal(host(self.shares), shares)
        np.testing.assert_array_equal(host(self.free), self.host[2])
        assert int(self.left) == left and int(self.copies) == len(copies) and sync == (0 if fits else EPAGES)
        assert list(zip(host(at)[:len(copies)], host(to)[:len(copies)])) == copies
        assert bool((at[len(copies):] == -1).all()) and bool((to[len(copies):] == -1).all())  # as they were
        for w, _ in self.pairs:
            assert_guards_intact(w)
        self.intact()
        return copies

    def check_free(self, ctx, first, end):
        t.check(t.tp3d_paged_free(ctx, self.pool, i32(first), i32(end), self.count, self.left))
        sync = t.tp3d_sync_status(ctx)
        table, shares, free, left, fits = OG.give_back(*self.host, first, end)
        np.testing.assert_array_equal(host(self.table), table)
        np.testing.assert_array_equal(host(self.shares), shares)
        np.testing.assert_array_equal(host(self.free), free)
        assert int(self.left) == left and sync == (0 if fits else EPAGES)
        self.intact()

    def check_compact(self, ctx, kv):
        (_, at), (_, to) = self.lists
        page_map = i32([-9] * len(self.host[1]))
        t.check(t.tp3d_paged_compact(ctx, self.pool, i32(kv), self.count, page_map, at, to, self.copies))
        sync = t.tp3d_sync_status(ctx)
        table, shares, free, where, copies, fits = OG.compact(self.page, *self.host, kv)
        np.testing.assert_array_equal(host(self.table), table)
        np.testing.assert_array_equal(host(self.shares), shares)
        np.testing.assert_array_equal(host(self.free), free)
        np.testing.assert_array_equal(host(page_map), where)
        assert int(self.copies) == len(copies) and sync == (0 if fits else EPAGES)
        assert list(zip(host(at)[:len(copies)], host(to)[:len(copies)])) == copies
        self.intact()
        return copies


def book(rng, rows, held, page=16, spare=5, shared=False, width=None, holes=0.0):
    """Row r holds held[r] pages of a shuffled pool; with ``shared`` odd rows name the pages of the row before them; a
    part ``holes`` of the entries name none."""
    width = max(max(held, default=0), 1) + 1 if width is None else width
    pages = sum(held) + spare
    order = rng.permutation(pages)
    table, shares, at = np.full((rows, width), -1), np.zeros(pages, dtype=np.int64), 0
    for r, n in enumerate(held):
        if shared and r % 2:
            n = min(n, held[r - 1])
            table[r, :n] = table[r - 1, :n]
            for p in table[r, :n]:
                shares[p] += p >= 0
        else:
            table[r, :n] = np.where(rng.random(n) < holes, -1, order[at:at + n])
            at += n
    named = set(int(p) for p in table.ravel() if p >= 0)
    free = [int(p) for p in order if int(p) not in named]
    return Book(page, table, shares, np.array(free + [-5] * (pages - len(free))), len(free))


# ------------------------------------------------------------------ fork
@pytest.mark.parametrize("rows,forks,page,most", [(1, 0, 16, 3), (2, 1, 16, 1), (9, 4, 64, 40), (300, 130, 16, 70),
                                                  (16384, 8000, 16, 3), (40, 39, 4096, 2)])
def test_fork(ctx, rows, forks, page, most):
    rng = np.random.default_rng(rows)
    parents = rows - forks if forks < rows else 1
    held = list(rng.integers(1, most + 1, parents)) + [0] * (rows - parents)
    b = book(rng, rows, held, page, forks + 3)
    src = rng.integers(0, parents, forks)
    dst = parents + rng.permutation(rows - parents)[:forks]
    length = np.array([int(rng.integers(0, held[s] * page + 1)) for s in src], dtype=np.int64)
    if forks:
        length[::3] -= length[::3] % page  # whole pages
    b.check_fork(ctx, src, dst, length)


def test_fork_of_one_row_many_times_and_past_given_up_pages(ctx):
    rng = np.random.default_rng(2)
    b = book(rng, 60, [300] + [0] * 59, spare=80, holes=0.3)
    b.host[0][0, 77] = b.host[0][0, 299] = 3  # (named twice: shares follow)
    b.table[0, 77] = b.table[0, 299] = 3
    b.check_fork(ctx, [0] * 59, list(range(1, 60)), [299 * 16 + 1 + i % 16 for i in range(59)])


@pytest.mark.parametrize("what", ["dst twice", "dst a src", "row", "dst", "negative", "long", "page", "gone", "free",
                                  "count", "negative count"])
def test_fork_that_does_not_fit_changes_nothing(ctx, what):
    rng = np.random.default_rng(3)
    b = book(rng, 9, [5, 6, 7, 0, 0, 0, 0, 0, 0])
    src, dst, length = [0, 1, 2, 0], [3, 4, 5, 6], [80, 90, 17, 33]
    if what == "dst twice":
        dst[3] = 3
    elif what == "dst a src":
        dst[1] = 2
    elif what == "row":
        src[2] = 9
    elif what == "dst":
        dst[0] = -1
    elif what == "negative":
        length[1] = -1
    elif what == "long":
        length[1] = b.host[0].shape[1] * 16 + 1
    elif what in ("page", "gone"):
        b.host[0][1, 5] = len(b.host[1]) if what == "page" else -1
        b.table[1, 5] = int(b.host[0][1, 5])
    else:
        n = {"free": 2, "count": len(b.host[2]) + 1, "negative count": -1}[what]
        b.host[3] = n
        b.count.fill_(n)
    b.check_fork(ctx, src, dst, length)
    assert t.tp3d_sync_status(ctx) == 0


def test_fork_of_entries_past_the_pool(ctx):
    b = book(np.random.default_rng(4), 3, [5, 0, 0])
    for col, bad in ((1, len(b.host[1])), (2, 2 ** 31 - 1), (3, -2 ** 31)):
        b.host[0][0, col] = bad
        b.table[0, col] = bad
    b.check_fork(ctx, [0], [2], [70])


# ------------------------------------------------------------------ free
@pytest.mark.parametrize("rows,most,shared,pages", [(1, 1, False, 0), (7, 40, True, 0), (256, 90, True, 3), (1000, 5, False, 0),
                                                    (16384, 3, True, 0), (3, 3000, True, 0), (20, 4, False, 600000)])
def test_free(ctx, rows, most, shared, pages):
    rng = np.random.default_rng(rows)
    held = list(rng.integers(0, most + 1, rows))
    b = book(rng, rows, held, spare=5 + pages, shared=shared, holes=0.1)
    first = rng.integers(0, most + 1, rows)
    end = np.where(rng.random(rows) < 0.3, 0, rng.integers(0, b.host[0].shape[1] + 1, rows))
    b.check_free(ctx, first, end)


def test_free_of_everything_and_of_nothing(ctx):
    rng = np.random.default_rng(6)
    for rows in (0, 5):
        b = book(rng, rows, [9] * rows, shared=True)
        b.check_free(ctx, [3] * rows, [3] * rows)
        b = book(rng, rows, [9] * rows, shared=True)
        b.check_free(ctx, [0] * rows, [9] * rows)


@pytest.mark.parametrize("what", ["first", "end", "entry", "twice", "over", "full", "count", "negative count"])
def test_free_that_does_not_fit(ctx, what):
    rng = np.random.default_rng(7)
    b = book(rng, 5, [8, 8, 8, 8, 8], spare=0 if what == "full" else 5)
    first, end = [0, 2, 1, 8, 0], [8, 6, 0, 9, 3]
    if what == "first":
        first[1] = -1
    elif what == "end":
        end[1] = 2 ** 31 - 1
    elif what == "entry":
        b.host[0][0, 2] = len(b.host[1])
        b.host[0][0, 3] = 2 ** 31 - 1
    elif what == "twice":
        b.host[0][0, 2] = b.host[0][0, 5]
    elif what == "over":
        b.host[0][0, 2] = b.host[0][0, 5] = b.host[0][4, 1]
        b.host[1][b.host[0][4, 1]] = 1
    else:
        b.host[3] = {"full": len(b.host[2]) - 3, "count": len(b.host[2]) + 4, "negative count": -4}[what]
        b.count.fill_(b.host[3])
    b.table.copy_(i32(b.host[0]))
    b.shares.copy_(i32(b.host[1]))
    b.check_free(ctx, first, end)
    assert t.tp3d_sync_status(ctx) == 0
    b = book(rng, 5, [8] * 5)
    b.check_free(ctx, [0] * 5, [8] * 5)  # nothing of it is left behind


# ------------------------------------------------------------------ compact
@pytest.mark.parametrize("rows,most,spare,shared", [(1, 1, 0, False), (1, 1, 1, False), (3, 4, 9, True), (64, 90, 700, True),
                                                    (300, 9, 5, False), (16384, 2, 9000, True), (2, 3000, 1000, False),
                                                    (8, 4, 500000, False), (0, 1, 77, False)])
def test_compact(ctx, rows, most, spare, shared):
    rng = np.random.default_rng(rows + spare)
    held = list(rng.integers(1, most + 1, rows))
    b = book(rng, rows, held, spare=spare, shared=shared, holes=0.1)
    kv = [max(0, n * 16 - int(rng.integers(0, 16))) for n in held]
    b.check_compact(ctx, kv)


def test_compact_of_a_full_and_of_an_empty_pool_and_of_a_compact_one(ctx):
    rng = np.random.default_rng(8)
    b = book(rng, 4, [9] * 4, spare=0)
    assert b.host[3] == 0 and b.check_compact(ctx, [9 * 16] * 4) == []
    b = book(rng, 4, [0] * 4, spare=40)
    assert b.check_compact(ctx, [0] * 4) == []
    b = Book(16, np.arange(30).reshape(3, 10), np.zeros(50), rng.permutation(20) + 30, 20)
    b.host[2] = np.concatenate([b.host[2], np.full(30, -5)])
    b = Book(16, *b.host)
    assert b.check_compact(ctx, [160, 160, 160]) == []


@pytest.mark.parametrize("what", ["twice", "past", "negative", "count", "negative count", "length", "negative length", "entry",
                                  "free entry"])
def test_compact_that_does_not_fit(ctx, what):
    rng = np.random.default_rng(9)
    b = book(rng, 5, [8, 4, 8, 7, 8], spare=60)
    kv = [100, 64, 128, 99, 3]
    if what in ("twice", "past", "negative"):
        b.host[2][7] = {"twice": b.host[2][3], "past": len(b.host[1]), "negative": -1}[what]
    elif what == "length":
        kv[2] = b.host[0].shape[1] * 16 + 1
    elif what == "negative length":
        kv[2] = -1
    elif what == "entry":
        b.host[0][2, 3] = len(b.host[1]) + 2
    elif what == "free entry":
        used = len(b.host[1]) - b.host[3]
        b.host[0][2, 3] = max(int(p) for p in b.host[2][:b.host[3]])
        assert b.host[0][2, 3] >= used
    else:
        b.host[3] = len(b.host[1]) + 1 if what == "count" else -1
    b = Book(16, *b.host)
    b.check_compact(ctx, kv)
    assert t.tp3d_sync_status(ctx) == 0
    b = book(rng, 5, [8] * 5, spare=60)
    b.check_compact(ctx, [128] * 5)  # nothing of it is left behind


# ------------------------------------------------------------------ copy
def pools(rng, pages, page, kv_heads, d, heads_first=False, pad=0):
    shape = (pages, kv_heads, page, d + pad) if heads_first else (pages, page, kv_heads, d + pad)
    x = torch.from_numpy(rng.integers(-2 ** 15, 2 ** 15, shape).astype(np.int16)).to(device()).view(torch.bfloat16)
    return x, (x.transpose(1, 2) if heads_first else x)[..., :d]


@pytest.mark.parametrize("page,kv_heads,d,heads_first,pad", [(16, 1, 64, False, 0), (16, 8, 128, False, 0), (64, 5, 64, True, 0),
                                                             (128, 3, 128, True, 8), (32, 2, 64, False, 72),
                                                             (4096, 2, 64, True, 0)])
@pytest.mark.parametrize("given", [None, 5, 0])
def test_copy(ctx, page, kv_heads, d, heads_first, pad, given):
    rng = np.random.default_rng(page + d)
    pages, n = 40, 17
    (kw, k), (vw, v) = (pools(rng, pages, page, kv_heads, d, heads_first, pad) for _ in range(2))
    order = rng.permutation(pages)
    at, to = order[:n], order[n:2 * n]
    want = [x.clone() for x in (kw, vw)]
    done = n if given is None else given
    for w in want:
        w[torch.from_numpy(to[:done])] = w[torch.from_numpy(at[:done])]
        if pad:  # columns between the rows belong to nobody
            w[..., d:] = (kw if w is want[0] else vw)[..., d:]
    t.check(t.tp3d_paged_copy(ctx, t.kv_cache(k, v), n, i32(at), i32(to), None if given is None else i32([given])))
    assert t.tp3d_sync_status(ctx) == 0
    for x, w in zip((kw, vw), want):
        assert torch.equal(x.view(torch.int16), w.view(torch.int16))


@pytest.mark.parametrize("count", [-1, 4, 2 ** 31 - 1])
def test_copy_that_does_not_fit(ctx, count):
    rng = np.random.default_rng(5)
    (_, k), (_, v) = (pools(rng, 9, 16, 2, 64) for _ in range(2))
    before = [k.clone(), v.clone()]
    t.check(t.tp3d_paged_copy(ctx, t.kv_cache(k, v), 3, i32([1, 2, 3]), i32([4, 5, 6]), i32([count])))
    assert t.tp3d_sync_status(ctx) == EPAGES
    done = 0 if count < 0 else 3
    for x, b in zip((k, v), before):
        b[4:4 + done] = b[1:1 + done]
        assert torch.equal(x.view(torch.int16), b.view(torch.int16))
    t.check(t.tp3d_paged_copy(ctx, t.kv_cache(k, v), 4, i32([-1, 0, 9, 1]), i32([0, -5, 0, 2 ** 31 - 1])))
    assert t.tp3d_sync_status(ctx) == EPAGES and t.tp3d_sync_status(ctx) == 0
    for x, b in zip((k, v), before):
        assert torch.equal(x.view(torch.int16), b.view(torch.int16))


def test_copy_past_32_bit_offsets(ctx):
    page, kv_heads, d = 16, 8, 128
    pages = 2 ** 32 // (page * kv_heads * d) + 8
    k, v = (torch.empty(pages, page, kv_heads, d, dtype=torch.bfloat16, device=device()) for _ in range(2))
    for x, c in ((k, 3.0), (v, 4.0)):
        x[pages - 1], x[2], x[pages - 5] = c, 0, 0
    t.check(t.tp3d_paged_copy(ctx, t.kv_cache(k, v), 2, i32([pages - 1, pages - 1]), i32([2, pages - 5])))
    assert t.tp3d_sync_status(ctx) == 0
    for x, c in ((k, 3.0), (v, 4.0)):
        assert bool((x[2] == c).all()) and bool((x[pages - 5] == c).all())


# ------------------------------------------------------------------ together
def test_a_captured_life_of_pages(ctx):
    # plan, fork, copy, give back and compact, one after the other without a pause, on another stream and in a graph
    # that is replayed: each time what the oracle says
    rng = np.random.default_rng(10)
    page, rows, width, pages, requests = 16, 12, 8, 96, 5
    table, shares = i32(np.full((rows, width), -1)), i32(np.zeros(pages))
    order = rng.permutation(pages)
    free = i32(order)
    start = [x.clone() for x in (table, shares, free)]
    pool = t.page_pool(page, table, shares, free)
    cached, fresh, count = i32([0] * rows), i32([0] * rows), i32([pages])
    q_start, kv, left = i32([0] * (rows + 1)), i32([0] * rows), [i32([0]) for _ in range(3)]
    slots, pos = torch.zeros(600, dtype=torch.int64, device=device()), i32([0] * 600)
    src, dst = i32([0, 0, 1, 3]), i32([5, 6, 7, 11])
    length, first, end, used = i32([0] * 4), i32([0] * rows), i32([0] * rows), i32([0] * rows)
    lists, n = [i32([0] * 48) for _ in range(4)], [i32([0]) for _ in range(2)]
    page_map = i32([0] * pages)
    (_, k), (_, v) = (pools(rng, pages, page, 2, 64) for _ in range(2))
    k0 = k.clone()
    cache = t.kv_cache(k, v)

    def step(stream=None):
        t.check(t.tp3d_paged_plan(ctx, page, rows, 600, cached, fresh, free, pages, count, table, width, q_start, kv,
                                  slots, pos, left[0], stream))
        t.check(t.tp3d_paged_fork(ctx, pool, src, dst, length, left[0], left[1], lists[0], lists[1], n[0], stream))
        t.check(t.tp3d_paged_copy(ctx, cache, 4, lists[0], lists[1], n[0], stream))
        t.check(t.tp3d_paged_free(ctx, pool, first, end, left[1], left[2], stream))
        t.check(t.tp3d_paged_compact(ctx, pool, used, left[2], page_map, lists[2], lists[3], n[1], stream))
        t.check(t.tp3d_paged_copy(ctx, cache, 48, lists[2], lists[3], n[1], stream))

    def want(f, cut):
        tab, at = np.full((rows, width), -1), pages
        for r in range(requests):
            for c in range(-(-f[r] // page)):
                at -= 1
                tab[r, c] = order[at]
        lens = [f[0], cut, f[1], f[3]]
        tab, sh, at, copies, fits = OG.fork(page, tab, np.zeros(pages), order, at, [0, 0, 1, 3], [5, 6, 7, 11], lens)
        contents = host(k0.view(torch.int16))
        for a, b in copies:
            contents[b] = contents[a]
        have = np.array(list(f) + lens[:3] + [0] * 3 + lens[3:])
        gone = [-(-have[r] // page) if r in (0, 6, 11) else 0 for r in range(rows)]
        tab, sh, fr, at, ok = OG.give_back(tab, sh, order, at, [0] * rows, gone)
        have[[0, 6, 11]] = 0
        tab, sh, fr, where, moves, well = OG.compact(page, tab, sh, fr, at, have)
        for a, b in moves:
            contents[b] = contents[a]
        assert fits and ok and well
        return tab, sh, fr, where, contents, lens, gone, have

    def reset(f, w):
        for x, y in zip((table, shares, free), start):
            x.copy_(y)
        k.copy_(k0)
        fresh.copy_(i32(list(f) + [0] * (rows - requests)))
        length.copy_(i32(w[5]))
        end.copy_(i32(w[6]))
        used.copy_(i32(w[7]))
        torch.cuda.synchronize()

    def check(w):
        for x, y in zip((table, shares, free, page_map), w):
            np.testing.assert_array_equal(host(x), y)
        np.testing.assert_array_equal(host(k.view(torch.int16)), w[4])

    side, g = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    w = want((100, 30, 17, 128, 5), 40)
    reset((100, 30, 17, 128, 5), w)
    step(side)
    assert t.tp3d_sync_status(ctx, side) == 0
    check(w)
    with torch.cuda.graph(g):
        step()
    for f, cut in (((100, 30, 17, 128, 5), 40), ((33, 48, 1, 16, 128), 33), ((128, 0, 5, 0, 77), 1)):
        w = want(f, cut)
        reset(f, w)
        g.replay()
        assert t.tp3d_sync_status(ctx) == 0
        check(w)

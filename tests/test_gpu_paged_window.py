"""Attention over the paged cache with a sliding window and first tokens that
stay visible, against the float64 oracle.  The arithmetic is that of
test_gpu_paged.py, whose tolerances these are; keys that no row sees lie in
pages that have been given back, whose table entries name none."""
import ctypes

import numpy as np
import pytest
import torch

import tensor_transformer_layer_cube_gb300 as t
from oracle import paged as OP
from tests.gpu_util import assert_guards_intact, device, guarded
from tests.test_gpu_paged import Case, compare, i32

pytestmark = pytest.mark.gpu

EPAGES = 10


@pytest.fixture(scope="module")
def ctx():
    c = t.tp3d_create(0)
    yield c
    t.tp3d_destroy(c)


def begin(p, window):
    return max(0, p - window + 1)


class Window(Case):
    def __init__(self, kv, new, heads, kv_heads, d, window, sinks, page=16, given_back=True, **kw):
        super().__init__(kv, new, heads, kv_heads, d, page, **kw)
        self.window, self.sinks = window, sinks
        if given_back:
            for b, (n, f) in enumerate(zip(kv, new)):
                for col in range(-(-int(n) // page)):
                    if col * page >= sinks and (col + 1) * page <= begin(int(n) - int(f), window):
                        self.table[b, col] = -1
            self.dev = (*self.dev[:2], i32(self.table))

    def run(self, ctx, max_new=None, o=None, lse=True, stream=None, workspace=None):
        o = torch.full(self.q.shape, float("nan"), dtype=torch.bfloat16, device=device()) if o is None else o
        l = torch.full(self.q.shape[:2], float("nan"), device=device()) if lse else None
        n = t.tp3d_paged_attn_workspace_bytes(ctx, self.cache, self.heads)
        self.ws = torch.empty(n, dtype=torch.uint8, device=device()) if workspace is None else workspace
        if stream is not None:
            stream.wait_stream(torch.cuda.current_stream())
        t.check(t.tp3d_paged_attn_window(ctx, self.cache, self.batch(max_new), self.q, o, l, self.scale, self.window,
                                         self.sinks, self.ws, stream))
        return o, l

    def want(self):
        return OP.attention(self.q.float().cpu().numpy(), self.kp.float().cpu().numpy(), self.vp.float().cpu().numpy(),
                            self.table, self.q_start, self.kv, self.scale, self.window, self.sinks)

    def sees(self, b, pos):
        """Which new tokens of request b see the key at pos."""
        p = int(self.kv[b] - self.new[b]) + np.arange(int(self.new[b]))
        return torch.from_numpy((pos <= p) & ((pos > p - self.window) | (pos < self.sinks))).to(device())


WINDOWS = [(1, 0), (1, 3), (2, 16), (15, 0), (16, 1), (17, 5), (63, 64), (64, 0), (65, 100), (127, 4), (128, 0), (129, 130),
           (300, 4), (500, 0), (1000, 40), (10 ** 12, 0), (40, 10 ** 12)]


@pytest.mark.parametrize("window,sinks", WINDOWS)
@pytest.mark.parametrize("heads,kv_heads,d", [(1, 1, 64), (8, 2, 128), (48, 1, 64), (14, 2, 128)])
def test_single_tokens(ctx, window, sinks, heads, kv_heads, d):
    kv = [1, 2, 15, 16, 17, 63, 64, 65, 127, 128, 129, 130, 700, 1111]
    c = Window(kv, [1] * len(kv), heads, kv_heads, d, window, sinks, seed=heads)
    o, l = c.run(ctx)
    assert t.tp3d_sync_status(ctx) == 0
    compare(c, o, l)


@pytest.mark.parametrize("window,sinks", WINDOWS)
@pytest.mark.parametrize("heads,kv_heads,d,new", [(4, 2, 64, 5), (8, 1, 128, 2), (1, 1, 64, 40), (16, 4, 128, 11)])
def test_short_chunks(ctx, window, sinks, heads, kv_heads, d, new):
    # few rows, in one block of them and in several; some rows see nothing
    kv = [new, 1, new + 70, 515, 2, 900]
    c = Window(kv, [new] * 6, heads, kv_heads, d, window, sinks, 32, heads_first=True, seed=new * heads, v_mean=0.5)
    o, l = c.run(ctx)
    assert t.tp3d_sync_status(ctx) == 0
    compare(c, o, l)


@pytest.mark.parametrize("window,sinks", WINDOWS)
@pytest.mark.parametrize("heads,kv_heads,d", [(2, 2, 128), (4, 1, 64), (3, 1, 128), (33, 1, 64)])
def test_chunks(ctx, window, sinks, heads, kv_heads, d):
    # more rows than the kernel for few takes: whole and cut pairs of tiles, prompts and chunks of them
    c = Window([130, 700, 333, 900, 257, 40], [130, 129, 333, 300, 64, 50], heads, kv_heads, d, window, sinks,
               seed=window % 1000 + heads, v_mean=1.0)
    o, l = c.run(ctx)
    assert t.tp3d_sync_status(ctx) == 0
    compare(c, o, l)


@pytest.mark.parametrize("page,heads_first,pad", [(16, True, 0), (32, False, 8), (64, True, 64), (128, False, 0),
                                                  (256, True, 0), (4096, False, 0)])
@pytest.mark.parametrize("new", [1, 5, 150])
@pytest.mark.parametrize("window,sinks", [(100, 20), (77, 0), (300, 129)])
def test_pages_and_strides(ctx, page, heads_first, pad, new, window, sinks):
    kv = [new, new + 1, 300, 511, 513, 5000]
    c = Window(kv, [min(new, k) for k in kv], 4, 2, 128, window, sinks, page, heads_first=heads_first, pad=pad,
               packed=new != 5, seed=page + new)
    o, l = c.run(ctx)
    assert t.tp3d_sync_status(ctx) == 0
    compare(c, o, l)


@pytest.mark.parametrize("max_new", [None, 0, 10 ** 6])
@pytest.mark.parametrize("window,sinks", [(1, 0), (33, 2), (200, 64)])
def test_mixed_lengths_and_rows_without_keys(ctx, max_new, window, sinks):
    kv = [500, 0, 3, 900, 77, 40, 0, 1, 260]
    new = [1, 0, 8, 300, 1, 100, 5, 1, 0]
    c = Window(kv, new, 8, 2, 64, window, sinks, 32, seed=4)
    o, l = c.run(ctx, max_new)
    assert t.tp3d_sync_status(ctx) == 0
    compare(c, o, l)
    n = c.q_start
    assert bool((o[n[2]:n[2] + 5] == 0).all()) and bool(torch.isneginf(l[n[2]:n[2] + 5]).all())
    assert bool((o[n[6]:n[7]] == 0).all()) and bool(torch.isneginf(l[n[6]:n[7]]).all())


@pytest.mark.parametrize("kv,new,heads,kv_heads,window,sinks", [
    ([9001], [1], 2, 1, 6000, 4), ([20000], [1], 16, 16, 3001, 0), ([6100], [130], 2, 1, 4000, 100),
    ([8000, 1, 77], [1, 1, 1], 8, 8, 5000, 7), ([6000], [3], 16, 1, 4999, 1), ([4500, 2000], [129, 1], 4, 1, 2500, 600),
    ([5000, 4000, 3700], [200, 130, 256], 2, 2, 3000, 4)])
def test_work_split_along_the_keys(ctx, kv, new, heads, kv_heads, window, sinks):
    c = Window(kv, new, heads, kv_heads, 128, window, sinks, 64, seed=7)
    o, l = c.run(ctx)
    assert t.tp3d_sync_status(ctx) == 0
    compare(c, o, l)
    for _ in range(4):
        o2, l2 = c.run(ctx)
        assert torch.equal(o.view(torch.int16), o2.view(torch.int16)) and torch.equal(l, l2)


@pytest.mark.parametrize("kv,new,heads,kv_heads,d,window,sinks", [
    ([3000], [64], 1, 1, 128, 40, 0), ([5000], [250], 8, 2, 64, 1000, 3), ([3001], [17], 48, 1, 128, 100, 20),
    ([2500, 2000], [131, 131], 4, 2, 128, 300, 0), ([2600, 65, 0, 1900], [65, 64, 3, 1], 8, 2, 64, 513, 16),
    ([900] * 9, [33] * 9, 8, 4, 128, 127, 1), ([40000], [513], 8, 4, 64, 257, 300), ([40000], [300], 3, 1, 128, 2000, 0),
    ([9000, 8000], [200, 100], 2, 2, 128, 100, 5), ([9000, 8000], [201, 100], 2, 2, 128, 100, 5)])
@pytest.mark.parametrize("max_new", [0, 600])
def test_short_windows_over_long_contexts(ctx, kv, new, heads, kv_heads, d, window, sinks, max_new):
    # little work for each SM: about where a call of many rows moves to the kernel for few, on either side
    c = Window(kv, new, heads, kv_heads, d, window, sinks, 32, seed=len(kv) + window, v_mean=0.5)
    want = None
    for _ in range(2):
        o, l = c.run(ctx, max_new or max(new))
        assert t.tp3d_sync_status(ctx) == 0
        compare(c, o, l)
        assert want is None or (torch.equal(o, want[0]) and torch.equal(l, want[1]))
        want = o, l


@pytest.mark.parametrize("heads,kv_heads,d,new", [(16, 4, 64, 8), (16, 4, 128, 8), (4, 4, 64, 33), (28, 4, 128, 3), (4, 4, 128, 17)])
@pytest.mark.parametrize("window,sinks", [(10, 0), (100, 3), (700, 16), (1290, 5), (1400, 0)])
def test_short_chunks_of_many_requests(ctx, heads, kv_heads, d, new, window, sinks):
    # two blocks of 16 rows (the second one cut short, or none) in a call of many items, and lengths beside the limit
    rng = np.random.default_rng(new)
    kv = np.concatenate([rng.integers(0, 2000, 36), [1500, new, new + 1, 0]])
    fresh = np.minimum(kv, np.concatenate([rng.integers(0, new + 1, 36), [new, new, new, 0]]))
    c = Window(kv, fresh, heads, kv_heads, d, window, sinks, 16, seed=new + window, v_mean=0.5)
    for most in (None, 0):
        o, l = c.run(ctx, most)
        assert t.tp3d_sync_status(ctx) == 0
        compare(c, o, l)


@pytest.mark.parametrize("value", [float("nan"), float("inf"), float("-inf")])
def test_values_that_are_not_finite_in_short_windows(ctx, value):
    # blocks of 16 rows side by side: each row leaves out what it alone does not see
    c = Window([2000, 1500], [90, 40], 4, 2, 128, 60, 3, 32, seed=5)
    at = [(0, 1915), (0, 1990), (0, 2), (0, 1000), (1, 1470)]
    for n, (b, pos) in enumerate(at):
        page = int(c.table[b, pos // 32])
        if page >= 0:
            c.vp[page, pos % 32, :, 7 * n] = value
    o, l = c.run(ctx)
    assert t.tp3d_sync_status(ctx) == 0
    for b, (q0, n) in enumerate(zip(c.q_start, c.new)):
        for k, (r, pos) in enumerate(at):
            if r == b:
                sees = c.sees(b, pos)
                column = o[int(q0):int(q0) + int(n), :, 7 * k]
                assert bool((~torch.isfinite(column[sees])).all()) and bool(torch.isfinite(column[~sees]).all())
    assert bool(torch.isfinite(l).all())


@pytest.mark.parametrize("requests", [129, 1000])
@pytest.mark.parametrize("long_every", [0, 7])
def test_many_requests(ctx, requests, long_every):
    rng = np.random.default_rng(requests)
    kv = rng.integers(1, 60, requests)
    new = (rng.random(requests) < 0.8).astype(np.int64)
    if long_every:
        new[3::long_every] = np.minimum(kv[3::long_every], 20)
    c = Window(kv, new, 4, 1, 64, 21, 3, seed=requests)
    o, l = c.run(ctx)
    assert t.tp3d_sync_status(ctx) == 0
    compare(c, o, l)


@pytest.mark.parametrize("new", [1, 7, 200])
def test_a_window_that_leaves_nothing_out_is_the_attention_without(ctx, new):
    c = Window([900, 513], [new, new], 4, 2, 128, 10 ** 9, 0, seed=3, given_back=False)
    want = [torch.empty_like(c.q), torch.empty(c.q.shape[:2], device=device())]
    for c.window, c.sinks in ((901, 0), (10 ** 12, 5), (1, 900)):
        o, l = c.run(ctx)
        t.check(t.tp3d_paged_attn(ctx, c.cache, c.batch(), c.q, *want, c.scale, c.ws))
        assert t.tp3d_sync_status(ctx) == 0
        assert torch.equal(o, want[0]) and torch.equal(l, want[1])


@pytest.mark.parametrize("new", [1, 140])
@pytest.mark.parametrize("std", [0.0, 8.0, 60.0])
def test_flat_and_sharply_peaked_scores(ctx, new, std):
    c = Window([600, 350], [new, new], 4, 1, 128, 150, 9, std=std, seed=9, v_mean=0.5)
    o, l = c.run(ctx)
    assert t.tp3d_sync_status(ctx) == 0
    compare(c, o, l)


# ------------------------------------------------------------------ what a row does not see
SHAPES = [([700, 300], [1, 1], 4, 2, 64), ([700, 300], [5, 5], 4, 2, 128), ([515, 700], [24, 24], 4, 2, 64),
          ([700, 900], [140, 260], 4, 2, 64), ([1500, 300], [500, 300], 2, 2, 128)]


@pytest.mark.parametrize("kv,new,heads,kv_heads,d", SHAPES)
@pytest.mark.parametrize("window,sinks", [(1, 0), (20, 3), (100, 4), (100, 64), (129, 130), (260, 1)])
@pytest.mark.parametrize("value", [float("nan"), float("inf"), float("-inf")])
def test_values_that_are_not_finite(ctx, kv, new, heads, kv_heads, d, window, sinks, value):
    # at positions all over the request: rows that see such a value have something not finite in its column, the others
    # are what they are without it, bit for bit
    c = Window(kv, new, heads, kv_heads, d, window, sinks, seed=13, given_back=False)
    clean, cl = c.run(ctx)
    rng = np.random.default_rng(window + sinks)
    hit = torch.zeros_like(clean, dtype=torch.bool)
    g = heads // kv_heads
    for b in range(len(kv)):
        for pos in {0, 2, 3, 4, 63, 64, 129, kv[b] - 1, kv[b] - new[b], kv[b] - new[b] - 1, kv[b] - new[b] - window,
                    kv[b] - new[b] - window + 1, kv[b] - window - 1, kv[b] - window, *rng.integers(0, kv[b], 4)}:
            if pos < 0:
                continue
            head, col = int(rng.integers(kv_heads)), int(rng.integers(d))
            c.vp[int(c.table[b, pos // 16]), pos % 16, head, col] = value
            rows = hit[int(c.q_start[b]):int(c.q_start[b + 1])]
            rows[:, head * g:(head + 1) * g, col] |= c.sees(b, pos)[:, None]
    o, l = c.run(ctx)
    assert t.tp3d_sync_status(ctx) == 0
    assert torch.equal(l, cl) and torch.equal(o[~hit], clean[~hit])
    assert not bool(o[hit].isfinite().any())


@pytest.mark.parametrize("kv,new,heads,kv_heads,d", SHAPES)
@pytest.mark.parametrize("window,sinks", [(1, 0), (20, 3), (129, 64)])
def test_keys_that_are_not_finite(ctx, kv, new, heads, kv_heads, d, window, sinks):
    c = Window(kv, new, heads, kv_heads, d, window, sinks, seed=14, given_back=False)
    clean, cl = c.run(ctx)
    spoilt = 0
    for b in range(len(kv)):
        p = np.arange(kv[b] - new[b], kv[b])
        for pos in range(kv[b]):
            if pos % 7 < 2 and not ((pos <= p) & ((pos > p - window) | (pos < sinks))).any():
                c.kp[int(c.table[b, pos // 16]), pos % 16] = float("nan") if pos % 2 else float("inf")
                spoilt += 1
    o, l = c.run(ctx)
    assert t.tp3d_sync_status(ctx) == 0 and (spoilt or new[0] > 260)
    assert torch.equal(l, cl) and torch.equal(o, clean)
    # and one that some rows see
    b, pos = 1, kv[1] - new[1]
    c.kp[int(c.table[b, pos // 16]), pos % 16, 0] = float("nan")
    o, l = c.run(ctx)
    assert t.tp3d_sync_status(ctx) == 0
    hit = torch.zeros_like(l, dtype=torch.bool)
    hit[int(c.q_start[b]):, :heads // kv_heads] = c.sees(b, pos)[:, None]
    assert torch.equal(l[~hit], cl[~hit]) and torch.equal(o[~hit], clean[~hit])
    assert bool(o[hit].isnan().all())


@pytest.mark.parametrize("kv,new,heads", [(700, 1, 4), (700, 5, 4), (700, 140, 4), (9000, 1, 2), (9000, 200, 2)])
def test_rows_whose_scores_are_all_lowest(ctx, kv, new, heads):
    # every key in the window and among the first at -infinity, which leaves 0 / 0; other rows see others
    c = Window([kv, 77], [new, min(new, 70)], heads, 2, 64, 200, 3, 64, seed=new, given_back=False)
    c.q[..., 0] = c.q[..., 0].abs() + 1
    clean, cl = c.run(ctx)
    for pos in [0, 1, 2, *range(begin(kv - new, 200), kv)]:
        c.kp[int(c.table[0, pos // 64]), pos % 64, 1, 0] = -torch.inf
    o, l = c.run(ctx)
    assert t.tp3d_sync_status(ctx) == 0
    hit = torch.zeros_like(l, dtype=torch.bool)
    hit[:new, heads // 2:] = True
    assert bool(o[hit].isnan().all()) and bool(torch.isneginf(l[hit]).all())
    assert torch.equal(o[~hit], clean[~hit]) and torch.equal(l[~hit], cl[~hit])


# ------------------------------------------------------------------ pages and bounds
@pytest.mark.parametrize("new", [1, 9, 140])
def test_missing_pages_are_reported_where_they_are_needed(ctx, new):
    c = Window([900, 900], [new, new], 4, 2, 64, 200, 20, seed=5, given_back=False)
    good, _ = c.run(ctx)
    assert t.tp3d_sync_status(ctx) == 0
    low = begin(900 - new, 200)
    for col in range(0, 57):
        seen = col * 16 < 20 or (col + 1) * 16 > low
        if seen and col not in (0, 1, low // 16, 56):
            continue
        for bad in (-1, c.kp.shape[0], 2 ** 31 - 1):
            table = c.table.copy()
            table[0, col] = bad
            c.dev = (*c.dev[:2], i32(table))
            o, _ = c.run(ctx)
            assert t.tp3d_sync_status(ctx) == (EPAGES if seen else 0), (col, bad)
            assert torch.equal(o[new:], good[new:]) and (seen or torch.equal(o, good))


def test_bad_lengths_stay_in_bounds(ctx):
    for new in (1, 140):
        c = Window([300, 300], [new, new], 4, 2, 64, 100, 4, seed=5, given_back=False)
        table = np.where(c.table > 10 ** 6, 0, c.table)
        for kv in ([300, 10 ** 9], [-5, 300], [2 ** 31 - 1, -2 ** 31]):
            c.dev = (c.dev[0], i32(kv), i32(table))
            c.run(ctx)
            assert t.tp3d_sync_status(ctx) == EPAGES
        for qs in ([0, new, 10 ** 9], [-3, new, 2 * new], [new, 0, 2 * new]):
            c.dev = (i32(qs), i32([300, 300]), i32(table))
            c.run(ctx, max_new=0)
            assert t.tp3d_sync_status(ctx) == EPAGES
    assert t.tp3d_sync_status(ctx) == 0


@pytest.mark.parametrize("d", [64, 128])
def test_no_store_outside_the_output_and_the_workspace(ctx, d):
    c = Window([900, 40, 1, 5000], [200, 17, 1, 3], 4, 2, d, 300, 5, extra_tokens=3)
    whole, flat = guarded(c.tokens * 4 * d, torch.bfloat16)
    ww, ws = guarded(t.tp3d_paged_attn_workspace_bytes(ctx, c.cache, 4), torch.uint8)
    o, l = c.run(ctx, o=flat.view(c.tokens, 4, d), workspace=ws)
    assert t.tp3d_sync_status(ctx) == 0
    compare(c, o, l)
    assert bool(o[221:].isnan().all()) and bool(l[221:].isnan().all())
    assert_guards_intact(whole)
    assert_guards_intact(ww)


@pytest.mark.parametrize("new", [1, 140])
def test_other_stream_and_graph_replay(ctx, new):
    c = Window([700, 600], [new, new], 8, 2, 128, 150, 10, seed=6, given_back=False)
    want, _ = c.run(ctx)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    o, l = c.run(ctx, stream=side)
    assert t.tp3d_sync_status(ctx, side) == 0
    assert torch.equal(o, want)
    o, g, batch = torch.zeros_like(o), torch.cuda.CUDAGraph(), c.batch()
    with torch.cuda.graph(g):
        t.check(t.tp3d_paged_attn_window(ctx, c.cache, batch, c.q, o, l, c.scale, c.window, c.sinks, c.ws))
    for kv in ([700, 600], [499, 230], [new, 400]):
        c.kv = np.asarray(kv)
        c.dev[1].copy_(i32(kv))
        g.replay()
        assert t.tp3d_sync_status(ctx) == 0
        compare(c, o, l)


def test_a_wait_that_runs_out(ctx):
    # the kernel for many rows stops loading: its waits end by themselves, and the next call is whole again
    c = Window([900, 800], [200, 300], 4, 2, 128, 300, 5, seed=8)
    want, _ = c.run(ctx)
    assert t.tp3d_sync_status(ctx) == 0
    t.check(t.tp3d_set_wait_limit_ns(ctx, 20_000_000))
    try:
        for stages in (0, 1, 2, 3, 4, 5):
            t.check(t.tp3d_inject_load_stall(ctx, stages))
            c.run(ctx)
            assert t.tp3d_sync_status(ctx) in ((6,) if stages < 2 else (0, 6))
    finally:
        t.check(t.tp3d_inject_load_stall(ctx, -1))
        t.check(t.tp3d_set_wait_limit_ns(ctx, 0))
    o, _ = c.run(ctx)
    assert t.tp3d_sync_status(ctx) == 0 and torch.equal(o, want)


def test_refusals(ctx):
    c = Window([40], [1], 4, 2, 64, 8, 1, given_back=False)
    o, lib = torch.empty(c.q.shape, dtype=torch.bfloat16, device=device()), t.lib()
    ws = torch.empty(t.tp3d_paged_attn_workspace_bytes(ctx, c.cache, 4), dtype=torch.uint8, device=device())

    def attn(window=8, sinks=1, x=ctx, out=o.data_ptr(), scale=1.0):
        b = c.batch()
        return lib.tp3d_paged_attn_window(x, ctypes.byref(c.cache), ctypes.byref(b), 4, scale, window, sinks,
                                          c.q.data_ptr(), t.tp3d_row_strides(512, 64), out, t.tp3d_row_strides(256, 64),
                                          None, ws.data_ptr(), None)
    assert attn() == 0 and attn(window=2 ** 62, sinks=2 ** 62) == 0
    assert attn(window=0) == 1 and attn(window=-1) == 1 and attn(sinks=-1) == 1 and attn(x=None) == 1
    assert attn(out=c.q.data_ptr()) == 8 and attn(scale=0.0) == 1 and attn(out=None) == 1
    assert t.tp3d_sync_status(ctx) == 0
    with pytest.raises(ValueError):
        t.tp3d_paged_attn_window(ctx, c.cache, c.batch(), c.q.float(), o.float(), None, 1.0, 8, 1, ws)

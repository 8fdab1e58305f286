"""Attention over a sliding window in the kernel for many rows alone.  A call of little work goes to the kernel for few
rows whole, which depends on its requests, rows and window; so each case here has padding rows behind its requests'
(more than two windows of them, which a bound on the new tokens that says nothing cannot tell from new ones), and each
looks at which kernels its call launches.  Tolerances are those of test_gpu_paged.py, and for the probabilities
those of paged_util.py."""
import numpy as np
import pytest
import torch

import tensor_transformer_layer_cube_gb300 as t
from tests.gpu_util import device
from tests.launches import threads_of
from tests.paged_util import bound, to_bf16
from tests.test_gpu_paged import compare, i32
from tests.test_gpu_paged_window import Window, begin

pytestmark = pytest.mark.gpu

EPAGES = 10
MANY = 384  # threads of a CTA of that kernel; the one for few rows has 128 or 256


@pytest.fixture(scope="module")
def ctx():
    c = t.tp3d_create(0)
    yield c
    t.tp3d_destroy(c)


class Many(Window):
    """Requests of more than 48 rows for each key/value head; the others of a case may go to either kernel."""

    def __init__(self, kv, new, heads, kv_heads, d, window, sinks, page=16, **kw):
        super().__init__(kv, new, heads, kv_heads, d, window, sinks, page, extra_tokens=2 * window + 1, **kw)
        assert max(new) * (heads // kv_heads) > 48

    def run(self, ctx, **kw):
        o, l = super().run(ctx, max_new=0, **kw)
        n = int(self.q_start[-1])
        assert bool(o[n:].isnan().all()) and bool(l[n:].isnan().all())  # the padding's rows: as they were
        return o, l

    def launches_it(self, ctx):
        o, l = torch.empty_like(self.q), torch.empty(self.q.shape[:2], device=device())
        ws = torch.empty(t.tp3d_paged_attn_workspace_bytes(ctx, self.cache, self.heads), dtype=torch.uint8, device=device())
        batch = self.batch(0)
        return MANY in threads_of(lambda: t.check(t.tp3d_paged_attn_window(
            ctx, self.cache, batch, self.q, o, l, self.scale, self.window, self.sinks, ws)))


def test_what_a_call_of_little_work_launches(ctx):
    # the same requests and windows without the padding go to the kernel for few rows, and the results agree
    few = Window([700, 350], [140, 140], 4, 1, 128, 150, 9, seed=2)
    o, l = torch.empty_like(few.q), torch.empty(few.q.shape[:2], device=device())
    few.run(ctx)
    batch = few.batch()
    assert MANY not in threads_of(lambda: t.check(t.tp3d_paged_attn_window(
        ctx, few.cache, batch, few.q, o, l, few.scale, 150, 9, few.ws)))
    c = Many([700, 350], [140, 140], 4, 1, 128, 150, 9, seed=2)
    assert c.launches_it(ctx)
    o, l = c.run(ctx)
    assert t.tp3d_sync_status(ctx) == 0
    compare(c, o, l)


@pytest.mark.parametrize("kv,new,heads,window,sinks", [
    (700, 140, 4, 200, 3), (9000, 200, 2, 200, 3), (1500, 500, 2, 60, 0), (1000, 300, 8, 129, 130), (6100, 257, 2, 4000, 5)])
@pytest.mark.parametrize("d", [64, 128])
def test_rows_whose_scores_are_all_lowest(ctx, kv, new, heads, window, sinks, d):
    # every key in a window and among the first at -infinity, which leaves 0 / 0; other rows see others
    c = Many([kv, 77], [new, 70], heads, 2, d, window, sinks, 64, seed=new, given_back=False)
    assert c.launches_it(ctx)
    c.q[..., 0] = c.q[..., 0].abs() + 1
    clean, cl = c.run(ctx)
    # the last 40 rows see these keys and the first alone; rows before them some more
    for pos in [*range(sinks), *range(begin(kv - 40, window), kv)]:
        c.kp[int(c.table[0, pos // 64]), pos % 64, 1, 0] = -torch.inf
    o, l = c.run(ctx)
    assert t.tp3d_sync_status(ctx) == 0
    p = kv - new + np.arange(new)
    none = torch.zeros_like(l, dtype=torch.bool)
    none[:new, heads // 2:] = torch.from_numpy(p >= kv - 40).to(device())[:, None]
    own = torch.zeros_like(none)
    own[:new, heads // 2:] = True
    n = int(c.q_start[-1])
    assert bool(o[none].isnan().all()) and bool(torch.isneginf(l[none]).all())
    assert torch.equal(o[:n][~own[:n]], clean[:n][~own[:n]]) and torch.equal(l[:n][~own[:n]], cl[:n][~own[:n]])
    # the other rows of that head: what they are over the keys that are left, which is what the oracle says of them
    some = own & ~none
    if bool(some.any()):
        c.kp[..., 0] = torch.where(torch.isneginf(c.kp[..., 0]), torch.full_like(c.kp[..., 0], -2.0 ** 120), c.kp[..., 0])
        wo, wl, absum, amax = c.want()
        sees = ~none.cpu().numpy()[:n]
        got, wo = o[:n].double().cpu().numpy(), wo[:n]
        pad = ((2.0 ** -9 + 2.0 ** -9 + 2 * (d + 8) * 2.0 ** -24 * np.minimum(amax[:n], 64) + 2.0 ** -20)[..., None])
        assert not np.isnan(got[sees]).any()
        assert (np.abs(got - wo)[sees] <= ((np.abs(wo) * 2.0 ** -9 + pad * absum[:n]) * 1.04 + 1e-30)[sees]).all()


@pytest.mark.parametrize("new,heads,kv_heads", [(140, 4, 1), (300, 2, 2), (64, 16, 2)])
@pytest.mark.parametrize("std", [0.0, 8.0, 60.0])
@pytest.mark.parametrize("window,sinks", [(150, 9), (17, 0), (400, 200)])
def test_flat_and_sharply_peaked_scores(ctx, new, heads, kv_heads, std, window, sinks):
    c = Many([900, 350], [new, new], heads, kv_heads, 128, window, sinks, std=std, seed=9, v_mean=0.5)
    assert c.launches_it(ctx)
    o, l = c.run(ctx)
    assert t.tp3d_sync_status(ctx) == 0
    compare(c, o, l)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("window,sinks", [(300, 3), (700, 140), (129, 0)])
@pytest.mark.parametrize("way", ["up", "down", "steps"])
def test_scores_that_grow_and_fall_along_the_keys(ctx, d, window, sinks, way):
    # the running maximum moves in tile after tile, in none but the first, and in some rows of a warp alone
    c = Many([1700, 1100], [300, 200], 2, 2, d, window, sinks, seed=11, v_mean=0.5)
    assert c.launches_it(ctx)
    c.q[..., 0] = c.q[..., 0].abs() + 1
    if way == "steps":
        c.q[::2, :, 0] *= -1
    for b, kv in enumerate((1700, 1100)):
        for pos in range(kv):
            if c.table[b, pos // 16] >= 0:
                x = {"up": pos // 8, "down": (kv - pos) // 8, "steps": 200 * (pos // 128 % 2) - 100}[way]
                c.kp[int(c.table[b, pos // 16]), pos % 16, :, 0] = x
    o, l = c.run(ctx)
    assert t.tp3d_sync_status(ctx) == 0
    compare(c, o, l)


@pytest.mark.parametrize("kv,new,heads,kv_heads,window,sinks", [
    ([6100], [130], 2, 1, 4000, 100), ([4500, 2000], [129, 1], 4, 1, 2500, 600), ([9000, 8000], [200, 100], 2, 2, 1000, 5),
    ([5000, 4000, 3700], [200, 130, 256], 2, 2, 3001, 4)])
@pytest.mark.parametrize("d", [64, 128])
def test_work_split_along_the_keys(ctx, kv, new, heads, kv_heads, window, sinks, d):
    c = Many(kv, new, heads, kv_heads, d, window, sinks, 64, seed=7)
    assert c.launches_it(ctx)
    o, l = c.run(ctx)
    assert t.tp3d_sync_status(ctx) == 0
    compare(c, o, l)
    n = int(c.q_start[-1])
    for _ in range(4):
        o2, l2 = c.run(ctx)
        assert torch.equal(o[:n].view(torch.int16), o2[:n].view(torch.int16)) and torch.equal(l[:n], l2[:n])


# ------------------------------------------------------------------ what a row does not see
SHAPES = [([700, 300], [70, 60], 4, 2, 64), ([700, 900], [140, 260], 4, 2, 64), ([1500, 300], [500, 300], 2, 2, 128),
          ([700, 400], [129, 128], 1, 1, 128)]


@pytest.mark.parametrize("kv,new,heads,kv_heads,d", SHAPES)
@pytest.mark.parametrize("window,sinks", [(1, 0), (20, 3), (100, 64), (129, 130), (260, 1)])
@pytest.mark.parametrize("value", [float("nan"), float("inf"), float("-inf")])
def test_values_that_are_not_finite(ctx, kv, new, heads, kv_heads, d, window, sinks, value):
    c = Many(kv, new, heads, kv_heads, d, window, sinks, seed=13, given_back=False)
    assert c.launches_it(ctx)
    clean, cl = c.run(ctx)
    rng = np.random.default_rng(window + sinks)
    hit, g, n = torch.zeros_like(clean, dtype=torch.bool), heads // kv_heads, int(c.q_start[-1])
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
    o, clean, hit = o[:n], clean[:n], hit[:n]
    assert torch.equal(l[:n], cl[:n]) and torch.equal(o[~hit], clean[~hit])
    assert not bool(o[hit].isfinite().any())


@pytest.mark.parametrize("kv,new,heads,kv_heads,d", SHAPES)
@pytest.mark.parametrize("window,sinks", [(1, 0), (20, 3), (129, 64)])
def test_keys_that_are_not_finite(ctx, kv, new, heads, kv_heads, d, window, sinks):
    c = Many(kv, new, heads, kv_heads, d, window, sinks, seed=14, given_back=False)
    assert c.launches_it(ctx)
    clean, cl = c.run(ctx)
    n = int(c.q_start[-1])
    for b in range(len(kv)):
        p = np.arange(kv[b] - new[b], kv[b])
        for pos in range(kv[b]):
            if pos % 7 < 2 and not ((pos <= p) & ((pos > p - window) | (pos < sinks))).any():
                c.kp[int(c.table[b, pos // 16]), pos % 16] = float("nan") if pos % 2 else float("inf")
    o, l = c.run(ctx)
    assert t.tp3d_sync_status(ctx) == 0
    assert torch.equal(l[:n], cl[:n]) and torch.equal(o[:n], clean[:n])
    # and one that some rows see
    b, pos = 1, kv[1] - new[1]
    c.kp[int(c.table[b, pos // 16]), pos % 16, 0] = float("nan")
    o, l = c.run(ctx)
    assert t.tp3d_sync_status(ctx) == 0
    hit = torch.zeros_like(l[:n], dtype=torch.bool)
    hit[int(c.q_start[b]):, :heads // kv_heads] = c.sees(b, pos)[:, None]
    assert torch.equal(l[:n][~hit], cl[:n][~hit]) and torch.equal(o[:n][~hit], clean[:n][~hit])
    assert bool(o[:n][hit].isnan().all())


# ------------------------------------------------------------------ pages and bounds
@pytest.mark.parametrize("d,page", [(64, 16), (128, 16), (64, 128)])
def test_missing_pages_are_reported_where_they_are_needed(ctx, d, page):
    new, kv, window, sinks = 140, 900, 200, 20
    c = Many([kv, kv], [new, new], 4, 2, d, window, sinks, page, seed=5, given_back=False)
    assert c.launches_it(ctx)
    good, _ = c.run(ctx)
    assert t.tp3d_sync_status(ctx) == 0
    low, n, pages = begin(kv - new, window), 2 * new, -(-kv // page)
    for col in range(pages):
        seen = col * page < sinks or (col + 1) * page > low
        if seen and col not in (0, sinks // page, low // page, pages - 1):
            continue
        for bad in (-1, c.kp.shape[0], 2 ** 31 - 1):
            table = c.table.copy()
            table[0, col] = bad
            c.dev = (*c.dev[:2], i32(table))
            o, _ = c.run(ctx)
            assert t.tp3d_sync_status(ctx) == (EPAGES if seen else 0), (col, bad)
            assert torch.equal(o[new:n], good[new:n]) and (seen or torch.equal(o[:n], good[:n]))


def test_bad_lengths_stay_in_bounds(ctx):
    new = 140
    c = Many([300, 300], [new, new], 4, 2, 64, 100, 4, seed=5, given_back=False)
    assert c.launches_it(ctx)
    table = np.where(c.table > 10 ** 6, 0, c.table)
    for kv in ([300, 10 ** 9], [-5, 300], [2 ** 31 - 1, -2 ** 31]):
        c.dev = (c.dev[0], i32(kv), i32(table))
        Window.run(c, ctx, max_new=0)
        assert t.tp3d_sync_status(ctx) == EPAGES
    for qs in ([0, new, 10 ** 9], [-3, new, 2 * new], [new, 0, 2 * new]):
        c.dev = (i32(qs), i32([300, 300]), i32(table))
        Window.run(c, ctx, max_new=0)
        assert t.tp3d_sync_status(ctx) == EPAGES
    assert t.tp3d_sync_status(ctx) == 0


# ------------------------------------------------------------------ the probabilities' 16 bits
@pytest.mark.parametrize("many", [False, True])
@pytest.mark.parametrize("requests", [2, 40])
@pytest.mark.parametrize("kv,new,heads,kv_heads,window,sinks", [
    (130, 130, 2, 2, 40, 0), (200, 150, 6, 3, 64, 3), (300, 280, 2, 2, 33, 17), (400, 60, 2, 1, 128, 5)])
@pytest.mark.parametrize("d", [64, 128])
def test_probabilities_of_two_terms(ctx, many, requests, kv, new, heads, kv_heads, window, sinks, d):
    # elements that cancel over the keys that their row sees
    c = (Many if many else Window)([kv] * requests, [new] * requests, heads, kv_heads, d, window, sinks, std=0.05, seed=kv)
    assert not many or c.launches_it(ctx)
    rng, at = np.random.default_rng(new), []
    sees = [np.r_[0:min(sinks, max(0, p - window + 1)), max(0, p - window + 1):p + 1] for p in range(kv - new, kv)]
    for b in range(min(requests, 4)):
        q = c.q[b * new:(b + 1) * new].double().cpu().numpy()
        cols = np.arange(-(-kv // 16))[c.table[b, :-(-kv // 16)] >= 0]  # pages that are there
        ids = torch.from_numpy(c.table[b, cols]).to(device())
        k, v = np.full((kv + 15, kv_heads, d), np.nan), to_bf16(rng.normal(size=(kv + 15, kv_heads, d)))
        place = (cols[:, None] * 16 + np.arange(16)).reshape(-1)
        k[place] = c.kp[ids].flatten(0, 1).double().cpu().numpy()
        for h in range(kv_heads):
            for col in range(d):
                j, i = int(rng.integers(new)), h * (heads // kv_heads) + int(rng.integers(heads // kv_heads))
                seen = sees[j]
                s = c.scale * (k[seen, h] @ q[j, i])
                p = np.exp(s - s.max())
                p /= p.sum()
                x = v[seen, h, col]
                if len(x) < 4:
                    continue
                keys = rng.permutation(len(x))[:3]
                x[keys] = 0
                for key in keys:  # each takes what is left, up to 2^-9 of it
                    x[key] = to_bf16(-(p @ x) / p[key])
                v[seen, h, col] = x
                at.append((b * new + j, i, col))
        c.vp[ids] = torch.from_numpy(v[place]).to(torch.bfloat16).to(device()).view(len(cols), 16, kv_heads, d)
    o, _ = c.run(ctx)
    assert t.tp3d_sync_status(ctx) == 0
    n = requests * new
    want, _, absum, amax = (x[:n] for x in c.want())
    keys = np.tile(np.repeat(np.array([[float(len(x))] for x in sees]), heads, 1), (requests, 1))
    err, tol = np.abs(o[:n].double().cpu().numpy() - want), bound(want, absum, amax, keys)
    assert (err <= tol).all(), (err / tol).max()
    x = tuple(np.array(at).T)
    assert (np.abs(want[x]) <= 2.0 ** -20 * absum[x]).all()  # they do cancel

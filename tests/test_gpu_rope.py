"""The norm of query and key heads with the rotation by position on the GPU
against the float64 oracle.

Tolerances, derived from the arithmetic (u = finfo(type).eps / 2, half a step
of the output's type; e = 2^-24, of fp32, in which everything is computed):
- s = 1 / sqrt(mean x^2 + eps): the sum of squares is off by 13 e at most (8
  products and 5 additions in a row), its mean and eps add 3 e, the root halves
  that and rsqrt adds 4 e: 12 e.  n = x s w: 15 e relative.
- an angle in half turns is rounded to fp32 (2^-25 at most, pi 2^-25 < 1.6 e),
  its sine and cosine to 2 e, their product with the magnitude to 1 e: the
  factors of the rotation are off by 5 e |magnitude|.
- y_a = c n_a - s n_b: two roundings more, so |y - want| <= u |want| +
  24 e |magnitude| (|n_a| + |n_b|).
Backward: g is off by 8 e |magnitude| (|dy_a| + |dy_b|) = 8 e G.  In dx =
s (w g - n mean(w g n)) the first term is off by (12 + 8 + 4) e s |w| G, and the
second, with twice s in n and a sum of 13 steps, by 80 e s |n| mean(|w| G |n|).
dw sums T = tokens x heads terms g n, each off by 24 e G |n|, in at most T + 64
additions."""
import numpy as np
import pytest
import torch

import tensor_transformer_layer_cube_gb300 as t
from oracle import paged as OP
from oracle import rope as OR
from tests.gpu_util import assert_guards_intact, device, guarded

pytestmark = pytest.mark.gpu

E, EPAGES = 2.0 ** -24, 10
BF16, F32 = torch.bfloat16, torch.float32
FAR = [0, 1, -1, 2 ** 31 - 1, -2 ** 31, 131071, 65536, -77]


@pytest.fixture(scope="module")
def ctx():
    c = t.tp3d_create(0)
    yield c
    t.tp3d_destroy(c)


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def host(x):
    return x.double().cpu().numpy()


def random(rng, dtype, *shape):
    return torch.from_numpy(rng.normal(size=shape).astype(np.float32)).to(dtype).to(device())


class Case:
    """Rows as slices of one packed product's; positions near and far."""

    def __init__(self, tokens, heads, kv_heads, d, rot, dtype=BF16, inter=False, norm=True, weights=True, eps=1e-5,
                 kind="plain", seed=0, pad=0):
        rng = np.random.default_rng(seed + 31 * tokens + heads + d)
        self.tokens, self.heads, self.kv_heads, self.d, self.dtype, self.eps = tokens, heads, kv_heads, d, dtype, eps
        self.inter, self.norm = inter, norm
        self.packed = random(rng, dtype, max(tokens, 1), (heads + 2 * kv_heads) * d + pad)[:tokens]
        self.q = self.packed[:, :heads * d].view(tokens, heads, d)
        self.k = self.packed[:, heads * d:(heads + kv_heads) * d].view(tokens, kv_heads, d)
        self.v = self.packed[:, (heads + kv_heads) * d:(heads + 2 * kv_heads) * d].view(tokens, kv_heads, d)
        self.words, self.magnitude = OR.turns(rot, kind=kind, factor=4.0, context=4096.0) if rot else ([], 1.0)
        self.turns = torch.tensor([w - 2 ** 64 * (w >= 2 ** 63) for w in self.words], dtype=torch.int64).to(device())
        self.pos = np.resize(FAR, tokens)
        if tokens > len(FAR):
            self.pos[len(FAR):] = rng.integers(0, 40000, tokens - len(FAR))
        self.positions = torch.tensor(self.pos, dtype=torch.int32).to(device())
        self.qw, self.kw = (1 + random(rng, dtype, d) / 4 if weights and norm else None for _ in range(2))
        self.rope = t.rope(self.turns if rot else None, dtype, d, rot, inter, self.magnitude, norm, eps, self.qw, self.kw)

    def new(self, heads):
        return torch.full((self.tokens, heads, self.d), float("nan"), dtype=self.dtype, device=device())

    def kw_of(self, w):
        return dict(interleaved=self.inter, magnitude=self.magnitude, norm=self.norm, eps=np.float64(np.float32(self.eps)),
                    weight=None if w is None else host(w))

    def check(self, got, x, w):
        want = OR.forward(host(x), self.words, self.pos, **self.kw_of(w))
        n = host(x)
        if self.norm:
            n = n * OR.inverse_rms(n, self.eps) * (1 if w is None else host(w))
        tol = half_step(self.dtype) * np.abs(want) + 24 * E * OR.spread(n, self.words, self.inter, self.magnitude)
        err = np.abs(host(got) - want)
        assert not np.isnan(err).any() and (err <= tol * (1 + 2.0 ** -6) + 1e-37).all(), (err / (tol + 1e-37)).max()

    def check_back(self, got, gw, x, dy, w):
        x, dy = host(x), host(dy)
        kw = self.kw_of(w)
        dx, dw = OR.backward(x, dy, self.words, self.pos, **kw)
        g = OR.spread(dy, self.words, self.inter, self.magnitude)
        tol = 8 * E * g
        if self.norm:
            aw = np.ones(self.d) if w is None else np.abs(host(w))
            s = OR.inverse_rms(x, self.eps)
            n = np.abs(x) * s
            tol = s * (24 * E * aw * g + 80 * E * n * (aw * g * n).mean(-1, keepdims=True))
        tol = half_step(self.dtype) * np.abs(dx) + tol
        err = np.abs(host(got) - dx)
        assert not np.isnan(err).any() and (err <= tol * (1 + 2.0 ** -6) + 1e-37).all(), (err / (tol + 1e-37)).max()
        if gw is not None:
            terms = x.shape[0] * x.shape[1]
            tol = half_step(self.dtype) * np.abs(dw) + (24 + terms + 64) * E * (g * n).sum((0, 1))
            err = np.abs(host(gw) - dw)
            assert (err <= tol * (1 + 2.0 ** -6)).all(), (err / tol).max()


SHAPES = [  # tokens, heads, kv_heads, d, rotary_dim
    (1, 1, 1, 8, 0), (1, 1, 1, 16, 16), (3, 5, 1, 24, 16), (7, 16, 16, 128, 128), (33, 32, 8, 128, 64), (5, 14, 2, 64, 64),
    (130, 3, 3, 80, 80), (61, 12, 4, 96, 48), (9, 4, 2, 256, 256), (40, 2, 1, 256, 32), (600, 16, 1, 64, 32),
    (3001, 6, 2, 136, 128), (1, 128, 8, 128, 128), (64, 1, 1, 48, 48)]


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("norm", [False, True])
def test_forward(ctx, shape, dtype, inter, norm):
    c = Case(*shape, dtype, inter, norm, kind="parts" if shape[4] else "plain")
    qo, ko = c.new(c.heads), c.new(c.kv_heads)
    t.check(t.tp3d_qk_rope(ctx, c.rope, c.q, c.k, c.positions, qo, ko))
    assert t.tp3d_sync_status(ctx) == 0
    c.check(qo, c.q, c.qw)
    c.check(ko, c.k, c.kw)


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("norm", [False, True])
def test_backward(ctx, shape, dtype, inter, norm):
    c = Case(*shape, dtype, inter, norm, kind="parts" if shape[4] else "plain")
    rng = np.random.default_rng(3)
    gq, gk = random(rng, dtype, c.tokens, c.heads, c.d), random(rng, dtype, c.tokens, c.kv_heads, c.d)
    dq, dk = c.new(c.heads), c.new(c.kv_heads)
    dqw, dkw = (torch.full((c.d,), float("nan"), dtype=dtype, device=device()) if norm else None for _ in range(2))
    n = t.tp3d_qk_rope_bwd_workspace_bytes(ctx, c.rope)
    whole, ws = guarded(n, torch.uint8)
    for _ in range(2):  # the arrivals' count is where it was
        x = (c.q, c.k) if norm else (None, None)
        t.check(t.tp3d_qk_rope_bwd(ctx, c.rope, *x, c.positions, gq, gk, dq, dk, dqw, dkw, ws if norm else None))
        assert t.tp3d_sync_status(ctx) == 0
        c.check_back(dq, dqw, c.q, gq, c.qw)
        c.check_back(dk, dkw, c.k, gk, c.kw)
    assert_guards_intact(whole)


@pytest.mark.parametrize("only", ["q", "k", "none"])
def test_backward_without_some_of_the_weights_gradients(ctx, only):
    c = Case(37, 6, 3, 64, 64, weights=False)
    rng = np.random.default_rng(4)
    gq, gk = random(rng, BF16, 37, 6, 64), random(rng, BF16, 37, 3, 64)
    dq, dk = c.new(6), c.new(3)
    dw = torch.zeros(64, dtype=BF16, device=device())
    ws = torch.empty(t.tp3d_qk_rope_bwd_workspace_bytes(ctx, c.rope), dtype=torch.uint8, device=device())
    t.check(t.tp3d_qk_rope_bwd(ctx, c.rope, c.q, c.k, c.positions, gq, gk, dq, dk, dw if only == "q" else None,
                               dw if only == "k" else None, None if only == "none" else ws))
    assert t.tp3d_sync_status(ctx) == 0
    c.check_back(dq, dw if only == "q" else None, c.q, gq, None)
    c.check_back(dk, dw if only == "k" else None, c.k, gk, None)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_no_tokens(ctx, dtype):
    c = Case(0, 2, 1, 256, 256, dtype)
    t.check(t.tp3d_qk_rope(ctx, c.rope, c.q, c.k, c.positions, c.new(2), c.new(1)))
    dqw, dkw = (torch.full((256,), 7.0, dtype=dtype, device=device()) for _ in range(2))
    ws = torch.empty(t.tp3d_qk_rope_bwd_workspace_bytes(ctx, c.rope), dtype=torch.uint8, device=device())
    t.check(t.tp3d_qk_rope_bwd(ctx, c.rope, c.q, c.k, c.positions, c.q, c.k, c.new(2), c.new(1), dqw, dkw, ws))
    assert t.tp3d_sync_status(ctx) == 0 and not bool(dqw.any()) and not bool(dkw.any())


def same(a, b):
    return torch.equal(a.view(torch.int16 if a.dtype == BF16 else torch.int32),
                       b.view(torch.int16 if b.dtype == BF16 else torch.int32))


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("tokens", [3, 2000])
def test_in_place_and_nothing_outside_the_rows(ctx, dtype, tokens):
    c = Case(tokens, 6, 2, 80, 32, dtype, pad=16)
    qo, ko = c.new(6), c.new(2)
    t.check(t.tp3d_qk_rope(ctx, c.rope, c.q, c.k, c.positions, qo, ko))
    width = c.packed.shape[1]
    whole, flat = guarded(tokens * width, dtype)
    rows = flat.view(tokens, width)
    rows.copy_(c.packed)
    q, k = rows[:, :480].view(tokens, 6, 80), rows[:, 480:640].view(tokens, 2, 80)
    t.check(t.tp3d_qk_rope(ctx, c.rope, q, k, c.positions, q, k))
    assert t.tp3d_sync_status(ctx) == 0
    assert same(q, qo) and same(k, ko) and same(rows[:, 640:], c.packed[:, 640:])
    assert_guards_intact(whole)
    # gradients in place
    rng = np.random.default_rng(6)
    gq, gk = random(rng, dtype, tokens, 6, 80), random(rng, dtype, tokens, 2, 80)
    dq, dk = c.new(6), c.new(2)
    t.check(t.tp3d_qk_rope_bwd(ctx, c.rope, c.q, c.k, c.positions, gq, gk, dq, dk, None, None, None))
    t.check(t.tp3d_qk_rope_bwd(ctx, c.rope, c.q, c.k, c.positions, gq, gk, gq, gk, None, None, None))
    assert t.tp3d_sync_status(ctx) == 0
    assert same(dq, gq) and same(dk, gk)


@pytest.mark.parametrize("value", [float("nan"), float("inf"), float("-inf"), 0.0])
def test_values_that_are_not_finite_stay_in_their_rows(ctx, value):
    for norm in (False, True):
        c = Case(50, 4, 2, 64, 32, BF16, norm=norm)
        clean, other = c.new(4), c.new(2)
        t.check(t.tp3d_qk_rope(ctx, c.rope, c.q, c.k, c.positions, clean, other))
        c.q[20, 1, 3] = value
        c.q[21, 2, 40] = value  # not turned
        got, k = c.new(4), c.new(2)
        t.check(t.tp3d_qk_rope(ctx, c.rope, c.q, c.k, c.positions, got, k))
        assert t.tp3d_sync_status(ctx) == 0
        hit = torch.zeros_like(got, dtype=torch.bool)
        hit[20, 1, :] = hit[21, 2, :] = norm
        hit[20, 1, [3, 19]] = hit[21, 2, 40] = True
        assert same(k, other) and torch.equal(got[~hit], clean[~hit])
        if not norm:
            assert got[21, 2, 40].isnan() if value != value else got[21, 2, 40] == value
        elif value == 0.0:
            c.check(got, c.q, c.qw)


def test_an_infinite_value_with_the_norm(ctx):
    # 1 / sqrt(infinity) is 0: the value itself and the column that it turns against are 0 times infinity, the others 0
    c = Case(9, 2, 1, 64, 32, BF16)
    c.q[3, 1, 5] = c.q[4, 0, 60] = c.q[5, 0, 17] = float("inf")
    got, k = c.new(2), c.new(1)
    t.check(t.tp3d_qk_rope(ctx, c.rope, c.q, c.k, c.positions, got, k))
    assert t.tp3d_sync_status(ctx) == 0
    for row, cols in (((3, 1), [5, 21]), ((4, 0), [60]), ((5, 0), [17, 1])):
        want = torch.zeros(64, dtype=torch.bool, device=device())
        want[cols] = True
        assert torch.equal(got[row].isnan(), want) and bool((got[row][~want] == 0).all())
    c.check(k, c.k, c.kw)


def test_gradients_of_very_small_rows(ctx):
    # s of 10^15 and more, whose powers fp32 does not hold
    c = Case(33, 2, 2, 64, 64, F32, eps=0.0, weights=False)
    c.q *= 1e-16
    c.k *= 1e15
    rng = np.random.default_rng(11)
    gq, gk = random(rng, F32, 33, 2, 64) * 1e-10, random(rng, F32, 33, 2, 64)
    dq, dk = c.new(2), c.new(2)
    t.check(t.tp3d_qk_rope_bwd(ctx, c.rope, c.q, c.k, c.positions, gq, gk, dq, dk, None, None, None))
    assert t.tp3d_sync_status(ctx) == 0
    c.check_back(dq, None, c.q, gq, None)
    c.check_back(dk, None, c.k, gk, None)


def test_bits_of_columns_that_are_not_turned(ctx):
    c = Case(16, 2, 1, 64, 16, BF16, norm=False)
    bits = torch.arange(16 * 2 * 64, dtype=torch.int32).mul(31).to(torch.int16).to(device()).view(16, 2, 64)
    q, qo = bits.view(BF16).clone(), c.new(2)
    t.check(t.tp3d_qk_rope(ctx, c.rope, q, c.k, c.positions, qo, c.new(1)))
    assert t.tp3d_sync_status(ctx) == 0
    nan = q.isnan()
    assert torch.equal(qo[..., 16:][~nan[..., 16:]].view(torch.int16), bits[..., 16:][~nan[..., 16:]])
    assert bool(qo[..., 16:][nan[..., 16:]].isnan().all())


def test_gradients_are_the_same_each_time(ctx):
    # many CTAs add to the weights' gradients: in the same order whatever else the GPU does
    c = Case(3000, 16, 4, 128, 128, BF16)
    rng = np.random.default_rng(8)
    gq, gk = random(rng, BF16, 3000, 16, 128), random(rng, BF16, 3000, 4, 128)
    ws = torch.empty(t.tp3d_qk_rope_bwd_workspace_bytes(ctx, c.rope), dtype=torch.uint8, device=device())
    first, x, side = None, torch.rand(140, 1 << 20, device=device()), torch.cuda.Stream()
    for i in range(12):
        with torch.cuda.stream(side):
            x[:20 * (i % 7) + 1].softmax(1)
        dq, dk = c.new(16), c.new(4)
        dqw, dkw = (torch.zeros(128, dtype=BF16, device=device()) for _ in range(2))
        t.check(t.tp3d_qk_rope_bwd(ctx, c.rope, c.q, c.k, c.positions, gq, gk, dq, dk, dqw, dkw, ws))
        got = [dq, dk, dqw, dkw]
        first = first or got
        assert all(same(a, b) for a, b in zip(got, first))
    assert t.tp3d_sync_status(ctx) == 0


@pytest.mark.parametrize("tokens", [1, 37, 2500])
@pytest.mark.parametrize("page,heads_first", [(16, False), (64, True)])
@pytest.mark.parametrize("d,heads,kv_heads", [(64, 14, 2), (128, 3, 3), (128, 32, 8), (64, 1, 1)])
def test_store(ctx, tokens, page, heads_first, d, heads, kv_heads):
    rng = np.random.default_rng(tokens + d)
    c = Case(tokens, heads, kv_heads, d, d // 2 if heads == 14 else d, BF16, inter=heads == 3, norm=heads != 1)
    pages = -(-tokens // page) + 3
    shape = (pages, kv_heads, page, d) if heads_first else (pages, page, kv_heads, d)
    kp, vp = (torch.full(shape, 7.0, dtype=BF16, device=device()) for _ in range(2))
    kp, vp = (x.transpose(1, 2) if heads_first else x for x in (kp, vp))
    slots = rng.permutation(pages * page)[:tokens].astype(np.int64)
    slots[rng.random(tokens) < 0.2] = -1
    qo, ko, q2 = c.new(heads), c.new(kv_heads), c.new(heads)
    t.check(t.tp3d_qk_rope(ctx, c.rope, c.q, c.k, c.positions, qo, ko))
    want = [OP.store(host(x), host(y), slots) for x, y in ((kp, ko), (vp, c.v))]
    t.check(t.tp3d_paged_rope_store(ctx, c.rope, t.kv_cache(kp, vp), c.q, c.k, c.v, c.positions,
                                    torch.from_numpy(slots).to(device()), q2))
    assert t.tp3d_sync_status(ctx) == 0
    assert same(qo, q2)
    np.testing.assert_array_equal(host(kp), want[0])
    np.testing.assert_array_equal(host(vp), want[1])


def test_store_slot_past_the_pool(ctx):
    c = Case(3, 2, 1, 64, 64)
    kp, vp = (torch.ones(2, 16, 1, 64, dtype=BF16, device=device()) for _ in range(2))
    slots = torch.tensor([3, 32, 2 ** 40], device=device())
    q = c.q.clone()
    t.check(t.tp3d_paged_rope_store(ctx, c.rope, t.kv_cache(kp, vp), q, c.k, c.v, c.positions, slots, q))
    assert t.tp3d_sync_status(ctx) == EPAGES and t.tp3d_sync_status(ctx) == 0
    c.check(q, c.q, c.qw)
    assert torch.equal(vp[0, 3, 0], c.v[0, 0]) and float(vp.float().sum() - c.v[0].float().sum()) == 31 * 64


def test_past_32_bit_offsets(ctx):
    # rows whose element offsets pass 2^31 and 2^32
    c = Case(3, 2, 1, 64, 64)
    step = 2 ** 31 + 64
    big = torch.empty(2 * step + 256, dtype=BF16, device=device())
    q, k = big.as_strided((3, 2, 64), (step, 64, 1)), big[128:].as_strided((3, 1, 64), (step, 64, 1))
    q.copy_(c.q)
    k.copy_(c.k)
    t.check(t.tp3d_qk_rope(ctx, c.rope, q, k, c.positions, q, k))
    assert t.tp3d_sync_status(ctx) == 0
    c.check(q, c.q, c.qw)
    c.check(k, c.k, c.kw)


def test_other_stream_and_graph_replay(ctx):
    c = Case(300, 8, 2, 128, 128)
    rng = np.random.default_rng(9)
    gq, gk = random(rng, BF16, 300, 8, 128), random(rng, BF16, 300, 2, 128)
    qo, ko, dq, dk = c.new(8), c.new(2), c.new(8), c.new(2)
    dqw, dkw = (torch.zeros(128, dtype=BF16, device=device()) for _ in range(2))
    ws = torch.empty(t.tp3d_qk_rope_bwd_workspace_bytes(ctx, c.rope), dtype=torch.uint8, device=device())

    def step(stream=None):
        t.check(t.tp3d_qk_rope(ctx, c.rope, c.q, c.k, c.positions, qo, ko, stream))
        t.check(t.tp3d_qk_rope_bwd(ctx, c.rope, c.q, c.k, c.positions, gq, gk, dq, dk, dqw, dkw, ws, stream))
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    step(side)
    assert t.tp3d_sync_status(ctx, side) == 0
    c.check(qo, c.q, c.qw)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for shift in (0, 1000, -5):
        c.pos = c.pos + shift
        c.pos[:8] = shift  # (the far ones would pass 32 bits)
        c.positions.copy_(torch.tensor(c.pos, dtype=torch.int32))
        g.replay()
        assert t.tp3d_sync_status(ctx) == 0
        c.check(qo, c.q, c.qw)
        c.check(ko, c.k, c.kw)
        c.check_back(dq, dqw, c.q, gq, c.qw)
        c.check_back(dk, dkw, c.k, gk, c.kw)

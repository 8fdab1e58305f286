"""The rotation's sines and cosines on the GPU, held relative to their own values: slow columns at early positions,
where a sine is small, and rows in which one column of a pair is zero or small, where nothing else hides it.

Tolerances, derived from the arithmetic (u = finfo(type).eps / 2, half a step of the output's type; e = 2^-24, of fp32,
in which everything is computed):
- a position times a frequency is a whole number of 2^-64 turns, exact modulo one turn, and so is what is left of it
  after whole quarter turns, r.  Its halves (the lower one signed) become fp32 and are multiplied and added: fp32's
  2 pi / 2^64 is off by 0.5 e; the sum's rounding e; beyond 2^24 2^32 the upper half's conversion e and the lower one's
  nothing to speak of; else the upper half is exact, the lower no more than r, its product off by e, its conversion by
  0.5 e where there is an upper half, and by e where there is none, when the sum is exact.  So an angle t within an
  eighth of a turn is off by 3 e of itself, whatever its size;
- sin t: t's error is at most 3 e of the sine, the series' sum is rounded to e, its terms behind the first (a tenth of
  the first at most, each with four roundings) add 0.4 e and what it leaves out 0.04 e.  cos t, which is 0.7 at least:
  t's error is at most 0.8 * 3 e of it, the series adds 2 e.  Together below 5 e of the value for either;
- A = magnitude cos weight and B, of the sine: two products, 7 e (6 e with weights of 1);
- A x + B x': a product and a sum more, 9 e of |A x| + |B x'|; without the norm (weights of 1) 8 e;
- the norm: s = 1 / sqrt(mean x^2 + eps) is off by 12 e (a sum of squares by 13 e at most, mean and eps 3 e, the root
  halves that, 4 e for rsqrt), its product with the row 1 e: 22 e.
So |y - want| <= u |want| + 22 e (|c n_a| + |s n_b|), 8 e without the norm, with c and s the pair's own factors.
Backward g is off by 8 e G, G = |c dy_a| + |s dy_b|; in dx = s (w g - n mean(w g n)) the first term by (12 + 8 + 4) e
s |w| G, the second, with twice s in n and a sum of 13 steps, by 80 e s |n| mean(|w| G |n|); dw sums T = tokens x heads
terms, each off by 24 e G |n|, in at most T + 64 additions."""
import math

import numpy as np
import pytest
import torch

import tensor_transformer_layer_cube_gb300 as t
from oracle import rope as OR
from tests.gpu_util import device

pytestmark = pytest.mark.gpu

E = 2.0 ** -24
BF16, F32 = torch.bfloat16, torch.float32
POS = [0, 1, 2, 3, -1, -2, 5, 7, 100, -100, 4095, 131071, 2 ** 31 - 1, -2 ** 31]


@pytest.fixture(scope="module")
def ctx():
    c = t.tp3d_create(0)
    yield c
    t.tp3d_destroy(c)


def factors(words, positions, magnitude):
    """(cosines, sines), (token, pair): each exact relative to itself, the turns taken off as whole numbers."""
    def one(p, w):
        v = p * w % 2 ** 64
        quarters = (v + 2 ** 61) // 2 ** 62
        a = 2 * math.pi * ((v - quarters * 2 ** 62) / 2 ** 64)
        c, s = math.cos(a), math.sin(a)
        return ((c, s), (-s, c), (-c, -s), (s, -c))[quarters % 4]
    x = np.array([[one(int(p), w) for w in words] for p in positions])
    return magnitude * x[..., 0], magnitude * x[..., 1]


def turned(x, c, s, inter, back=False):
    """R x (or its transpose) and |c x_a| + |s x_b| of every column; columns that are not turned as they are."""
    a, b = OR.pairs(2 * c.shape[1], inter)
    c, s = c[:, None], (-s if back else s)[:, None]
    y, size = x.copy(), np.abs(x)
    y[..., a], y[..., b] = x[..., a] * c - x[..., b] * s, x[..., a] * s + x[..., b] * c
    size[..., a] = np.abs(x[..., a] * c) + np.abs(x[..., b] * s)
    size[..., b] = np.abs(x[..., a] * s) + np.abs(x[..., b] * c)
    return y, size


def rows(rng, heads, d, rot, inter, shape, dtype):
    """Rows of which one column of each pair is zero, or small, or neither."""
    x = rng.normal(size=(len(POS), heads, d))
    a, b = OR.pairs(rot, inter)
    x[..., {"first": b, "second": a, "small": a, "both": []}[shape]] *= 1e-6 if shape == "small" else 0.0
    return torch.from_numpy(x.astype(np.float32)).to(dtype).to(device())


def host(x):
    return x.double().cpu().numpy()


def held(got, want, tol):
    err = np.abs(host(got) - want)
    assert not np.isnan(err).any() and (err <= tol * (1 + 2.0 ** -6) + 1e-37).all(), (err / (tol + 1e-37)).max()


CASES = [  # head size, turned columns, base, kind; the slowest pairs turn by 5.6e-6, 4.4e-7, 1.4e-10, 1.1e-4 and 4.4e-5
    (16, 16, 1e6, "plain"), (96, 48, 1e6, "linear"), (128, 128, 1e10, "plain"), (256, 256, 1e4, "plain"),
    (64, 32, 1e4, "parts")]


@pytest.mark.parametrize("d,rot,base,kind", CASES)
@pytest.mark.parametrize("shape", ["first", "second", "small", "both"])
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("norm", [False, True])
def test_every_factor_is_off_by_a_few_steps_of_itself(ctx, d, rot, base, kind, shape, dtype, inter, norm):
    rng = np.random.default_rng(d + rot)
    words, magnitude = OR.turns(rot, base, kind, 4.0, 4096.0)
    turns = torch.tensor(words, dtype=torch.int64, device=device())  # (below 2^62)
    c, s = factors(words, POS, float(np.float32(magnitude)))
    eps, n, heads, kv_heads = 2.0 ** -17, len(POS), 3, 2
    w = (1 + torch.from_numpy(rng.normal(size=d).astype(np.float32)) / 4).to(dtype).to(device()) if norm else None
    r = t.rope(turns, dtype, d, rot, inter, magnitude, norm, eps, w, w)
    positions = torch.tensor(POS, dtype=torch.int32, device=device())
    q, k, gq, gk = (rows(rng, h, d, rot, inter, shape, dtype) for h in (heads, kv_heads) * 2)
    qo, ko, dq, dk = (torch.full_like(x, float("nan")) for x in (q, k, q, k))
    dw = [torch.full((d,), float("nan"), dtype=dtype, device=device()) if norm else None for _ in range(2)]
    ws = torch.empty(t.tp3d_qk_rope_bwd_workspace_bytes(ctx, r), dtype=torch.uint8, device=device()) if norm else None
    t.check(t.tp3d_qk_rope(ctx, r, q, k, positions, qo, ko))
    t.check(t.tp3d_qk_rope_bwd(ctx, r, q, k, positions, gq, gk, dq, dk, *dw, ws))
    assert t.tp3d_sync_status(ctx) == 0
    half = torch.finfo(dtype).eps / 2
    aw = np.ones(d) if w is None else host(w)
    for x, y, g, dx, dwx in ((q, qo, gq, dq, dw[0]), (k, ko, gk, dk, dw[1])):
        x, g = host(x), host(g)
        inv = OR.inverse_rms(x, eps) if norm else 1.0
        want, size = turned(x * inv * aw, c, s, inter)
        held(y, want, half * np.abs(want) + (22 if norm else 8) * E * size)
        g, size = turned(g, c, s, inter, back=True)
        if not norm:
            held(dx, g, half * np.abs(g) + 8 * E * size)
            continue
        z = x * inv
        want = inv * (aw * g - z * (aw * g * z).mean(-1, keepdims=True))
        tol = inv * (24 * E * np.abs(aw) * size + 80 * E * np.abs(z) * (np.abs(aw) * size * np.abs(z)).mean(-1, keepdims=True))
        held(dx, want, half * np.abs(want) + tol)
        want = (g * z).sum((0, 1))
        held(dwx, want, half * np.abs(want) + (24 + x.shape[0] * x.shape[1] + 64) * E * (size * np.abs(z)).sum((0, 1)))

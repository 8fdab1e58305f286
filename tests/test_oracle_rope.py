"""The oracle of the head norm with the rotation, and the frequencies that the
library computes on the host."""
import ctypes
import math

import numpy as np
import pytest

import tensor_transformer_layer_cube_gb300 as t
from oracle import rope as OR

KINDS = {"plain": t.TP3D_ROPE_PLAIN, "linear": t.TP3D_ROPE_LINEAR, "base": t.TP3D_ROPE_BASE, "parts": t.TP3D_ROPE_PARTS}


@pytest.fixture(scope="module", autouse=True)
def built():
    t.build()


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("rotary_dim", [2, 16, 48, 128, 250])
@pytest.mark.parametrize("base", [1.0, 10000.0, 1e6])
def test_turns(kind, rotary_dim, base):
    if kind == "base" and rotary_dim == 2:
        return
    words, magnitude = OR.turns(rotary_dim, base, kind, 4.0, 4096.0)
    got, m = t.rope_turns(rotary_dim, base, KINDS[kind], 4.0, 4096.0)
    got = [int(x) % 2 ** 64 for x in got]
    # two powers in double, each some units in the last place off
    assert all(abs(g - w) <= 16 * 2 ** -53 * w + 1 for g, w in zip(got, words)) and len(got) == len(words)
    assert m == np.float32(magnitude)


def test_what_scaling_keeps():
    plain = np.array(OR.turns(128)[0], dtype=np.float64)
    linear = np.array(OR.turns(128, kind="linear", factor=8.0)[0], dtype=np.float64)
    base = np.array(OR.turns(128, kind="base", factor=8.0)[0], dtype=np.float64)
    parts = np.array(OR.turns(128, kind="parts", factor=8.0, context=4096.0)[0], dtype=np.float64)
    np.testing.assert_allclose(linear, plain / 8)
    np.testing.assert_allclose([base[0], base[-1]], [plain[0], plain[-1] / 8])
    over = 4096 * plain / 2 ** 64
    np.testing.assert_allclose(parts[over > 32], plain[over > 32])
    np.testing.assert_allclose(parts[over < 1], plain[over < 1] / 8)
    assert ((parts <= plain * (1 + 1e-12)) & (parts >= plain / 8 * (1 - 1e-12))).all()


def test_refused_turns():
    EINVAL, ESHAPE = 1, 2
    lib = t.lib()
    words, m = (ctypes.c_uint64 * 64)(), ctypes.c_float()

    def call(r=16, base=10000.0, kind=0, factor=2.0, context=64.0, w=words, out=ctypes.byref(m)):
        return lib.tp3d_rope_turns(r, base, kind, factor, context, w, out)
    assert call() == 0
    assert call(w=None) == EINVAL and call(out=None) == EINVAL and call(kind=4) == EINVAL and call(kind=-1) == EINVAL
    assert call(r=0) == ESHAPE and call(r=7) == ESHAPE and call(r=-2) == ESHAPE
    for bad in (0.5, float("nan"), float("inf"), -1.0):
        assert call(base=bad) == EINVAL and call(kind=3, context=bad) == EINVAL
        assert all(call(kind=k, factor=bad) == EINVAL for k in (1, 2, 3)) and call(factor=bad) == 0
    assert call(r=2, kind=2) == EINVAL
    with pytest.raises(t.Tp3dError):
        t.rope_turns(16, 0.1)


def test_angles_of_far_positions():
    words, _ = OR.turns(64)
    p = [0, 1, -1, 2 ** 31 - 1, -2 ** 31]
    th = OR.angles(words, p)
    assert (th[0] == 0).all()
    np.testing.assert_allclose(np.cos(th[1]), np.cos(10000.0 ** (-np.arange(32) / 32)), rtol=0, atol=1e-15)
    np.testing.assert_allclose(np.sin(th[2]), -np.sin(th[1]), rtol=0, atol=1e-14)


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("norm", [False, True])
@pytest.mark.parametrize("rotary_dim", [0, 4, 8])
def test_backward_is_the_derivative(interleaved, norm, rotary_dim):
    rng = np.random.default_rng(rotary_dim)
    words, _ = OR.turns(rotary_dim) if rotary_dim else ([], 1.0)
    kw = dict(interleaved=interleaved, magnitude=1.3, norm=norm, eps=1e-3)
    x, dy, w, pos = rng.normal(size=(3, 2, 8)), rng.normal(size=(3, 2, 8)), 1 + rng.normal(size=8) / 4, [0, 5, -700]
    dx, dw = OR.backward(x, dy, words, pos, weight=w, **kw)

    def loss(x, w):
        return float((OR.forward(x, words, pos, weight=w, **kw) * dy).sum())
    h = 1e-5
    for i in np.ndindex(x.shape):
        up, down = x.copy(), x.copy()
        up[i] += h
        down[i] -= h
        assert abs((loss(up, w) - loss(down, w)) / (2 * h) - dx[i]) < 1e-7
    if norm:
        for i in range(8):
            up, down = w.copy(), w.copy()
            up[i] += h
            down[i] -= h
            assert abs((loss(x, up) - loss(x, down)) / (2 * h) - dw[i]) < 1e-7


def test_rotation_keeps_scores_of_equal_distances():
    rng = np.random.default_rng(1)
    words, _ = OR.turns(16)
    q, k = rng.normal(size=(1, 1, 16)), rng.normal(size=(1, 1, 16))
    for inter in (False, True):
        s = [float((OR.rotate(q, words, [p + 9], inter, 1.0) * OR.rotate(k, words, [p], inter, 1.0)).sum())
             for p in (0, 17, 100000, -40)]
        np.testing.assert_allclose(s, s[0], rtol=0, atol=1e-12)
    assert math.isclose(float((OR.rotate(q, words, [3], False, 2.0) ** 2).sum()), 4 * float((q ** 2).sum()))

"""The norm of query and key heads with the rotation by position, forward and
backward, in float64 from the definitions.  Angles come from the same 64-bit
fractions of a turn, in whole numbers."""
from __future__ import annotations

import math

import numpy as np


def turns(rotary_dim, base=10000.0, kind="plain", factor=1.0, context=1.0):
    """Fractions of a turn per position, times 2^64 (Python integers), and the magnitude."""
    if kind == "base":
        base = base * factor ** (rotary_dim / (rotary_dim - 2))
    out = []
    for j in range(rotary_dim // 2):
        f = base ** (-2.0 * j / rotary_dim)
        if kind == "linear":
            f /= factor
        elif kind == "parts":
            over = context * f / (2 * math.pi)  # turns over the context
            keep = min(max((over - 1) / (32 - 1), 0.0), 1.0)
            f = f * keep + f / factor * (1 - keep)
        out.append(int(round(math.ldexp(f / (2 * math.pi), 64))))
    return out, (0.1 * math.log(factor) + 1 if kind == "parts" else 1.0)


def angles(words, positions):
    """(token, pair) radians."""
    return np.array([[(int(p) * w % 2 ** 64) / 2 ** 64 * 2 * math.pi for w in words] for p in positions],
                    dtype=np.float64).reshape(len(positions), len(words))


def pairs(rotary_dim, interleaved):
    """The two columns of each pair."""
    j = np.arange(rotary_dim // 2)
    return (2 * j, 2 * j + 1) if interleaved else (j, j + rotary_dim // 2)


def rotate(x, words, positions, interleaved, magnitude, back=False):
    """x (token, head, column); ``back``: the transposed rotation."""
    a, b = pairs(2 * len(words), interleaved)
    th = angles(words, positions)[:, None]
    c, s = magnitude * np.cos(th), magnitude * np.sin(th) * (-1 if back else 1)
    y = np.array(x, dtype=np.float64)
    y[..., a], y[..., b] = x[..., a] * c - x[..., b] * s, x[..., a] * s + x[..., b] * c
    return y


def spread(x, words, interleaved, magnitude):
    """|x| with each turned column replaced by magnitude times the sum over its pair: what an error of the rotation's
    factors is relative to."""
    a, b = pairs(2 * len(words), interleaved)
    y = np.abs(np.asarray(x, dtype=np.float64))
    y[..., a] = y[..., b] = abs(magnitude) * (y[..., a] + y[..., b])
    return y


def inverse_rms(x, eps):
    return 1 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)


def forward(x, words, positions, interleaved=False, magnitude=1.0, norm=False, eps=0.0, weight=None):
    n = np.asarray(x, dtype=np.float64)
    if norm:
        n = n * inverse_rms(n, eps) * (1.0 if weight is None else weight)
    return rotate(n, words, positions, interleaved, magnitude)


def backward(x, dy, words, positions, interleaved=False, magnitude=1.0, norm=False, eps=0.0, weight=None):
    """(dx, dw); dw None without the norm."""
    g = rotate(dy, words, positions, interleaved, magnitude, back=True)
    if not norm:
        return g, None
    w = 1.0 if weight is None else weight
    s = inverse_rms(x, eps)
    n = x * s
    dx = s * (w * g - n * (w * g * n).mean(-1, keepdims=True))
    return dx, (g * n).sum((0, 1))

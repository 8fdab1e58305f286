"""Inputs and bounds that tell the probabilities' precision in the paged
attention apart from the output's own rounding.

The output is bf16, so an error of its probabilities shows only where the
output is small beside sum p|v|.  ``cancelling_values`` makes values with which
chosen (row, head, column) elements come out at about 2^-27 sum p|v|.  There
the bound is, with n the row's keys and s the scores' term of
test_gpu_paged.py:
- 2^-8 |want|, the output's rounding (8 significant bits: the unit roundoff);
- 2^-16 sum p|v| for probabilities of two bf16 terms.  With p in [2^e, 2^(e+1))
  a truncated first term leaves less than 2^(e-7), whose rounding to 8 bits is
  off by 2^(e-16) at most; a rounded one leaves half as much;
- (s + (2 n + 32) 2^-23) sum p|v| for the scores and for 2 n products (n
  probabilities of two terms) and a few parts added up in fp32, each addition
  off by 2^-23 of the sum at most, however it rounds.
Probabilities of one bf16 term are off by 2^-10.3 each (root mean square), so
such an element by about 2^-10.3 sqrt(2 / n) sum p|v|: for n = 40 some five
times the bound."""
import numpy as np
import torch

E = 2.0 ** -24


def to_bf16(x):
    return torch.from_numpy(np.asarray(x, dtype=np.float64)).to(torch.bfloat16).double().numpy()


def cancelling_values(rng, q, k, scale):
    """q (new, heads, d), k (keys, kv_heads, d).  Returns v (keys, kv_heads, d), exact in bf16, and
    the (token, head, column) elements that cancel, one for each key/value head and column."""
    new, heads, d = q.shape
    kv, kv_heads, _ = k.shape
    v, at = to_bf16(rng.normal(size=(kv, kv_heads, d))), []
    for h in range(kv_heads):
        for col in range(d):
            t, i = int(rng.integers(new)), h * (heads // kv_heads) + int(rng.integers(heads // kv_heads))
            n = kv - new + t + 1
            s = scale * (k[:n, h] @ q[t, i])
            p = np.exp(s - s.max())
            p /= p.sum()
            x = v[:n, h, col]
            keys = rng.permutation(n)[:3]
            x[keys] = 0
            for key in keys:  # each takes what is left, up to 2^-9 of it
                x[key] = to_bf16(-(p @ x) / p[key])
            at.append((t, i, col))
    return v, at


def bound(want, absum, amax, keys):
    """The largest error of O; ``want``, ``absum`` (token, head, column), ``amax``, ``keys`` (token, head)."""
    d = want.shape[2]
    s = 2 * (d + 8) * E * amax + 2.0 ** -20
    rest = (2.0 ** -16 + s + (2 * keys + 32) * 2.0 ** -23)[..., None] * absum
    return (2.0 ** -8 * np.abs(want) + rest) * (1 + 2.0 ** -7) + 1e-30

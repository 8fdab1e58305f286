"""The bound on the paged attention's precision holds for probabilities of two
bf16 terms and fails for those of one (on the CPU, from the definitions)."""
import numpy as np
import pytest

from oracle import paged as OP
from tests.paged_util import bound, cancelling_values, to_bf16


def truncated(x):
    return (np.asarray(x, dtype=np.float32).view(np.uint32) & 0xffff0000).view(np.float32).astype(np.float64)


ROUNDINGS = {
    "two terms, rounded": lambda p: to_bf16(p) + to_bf16(p - to_bf16(p)),
    "two terms, truncated": lambda p: truncated(p) + to_bf16(p - truncated(p)),
    "one term, rounded": to_bf16,
    "one term, truncated": truncated,
}


@pytest.mark.parametrize("rounding", sorted(ROUNDINGS))
def test_two_terms_hold_their_bits(rounding):
    # 2^-16 of p, over three binades and the whole mantissa
    p = np.float32(np.geomspace(0.125, 1.0, 200001)).astype(np.float64)
    off = np.abs(ROUNDINGS[rounding](p) - p) / p
    assert (off.max() <= 2.0 ** -16) == rounding.startswith("two")


@pytest.mark.parametrize("kv,new,heads,kv_heads", [(40, 1, 4, 4), (60, 21, 4, 2), (120, 70, 4, 1)])
@pytest.mark.parametrize("rounding", sorted(ROUNDINGS))
def test_bound_tells_one_term_from_two(kv, new, heads, kv_heads, rounding):
    rng = np.random.default_rng(kv)
    d, scale = 64, 0.125
    q, k = to_bf16(rng.normal(size=(new, heads, d)) * 0.05), to_bf16(rng.normal(size=(kv, kv_heads, d)))
    v, at = cancelling_values(rng, q, k, scale)
    pools = [x[None] for x in (k, v)]  # one page
    want, _, absum, amax = OP.attention(q, *pools, np.array([[0]]), [0, new], [kv], scale)
    keys = np.repeat(kv - new + 1.0 + np.arange(new)[:, None], heads, 1)
    tol, g = bound(want, absum, amax, keys), heads // kv_heads
    ratio = []
    for t, i, c in at:
        n = kv - new + t + 1
        s = scale * (k[:n, i // g] @ q[t, i])
        p = np.exp(s - s.max())
        got = to_bf16(ROUNDINGS[rounding](p) @ v[:n, i // g, c] / p.sum())
        assert abs(want[t, i, c]) <= 2.0 ** -20 * absum[t, i, c]
        ratio.append(abs(got - want[t, i, c]) / tol[t, i, c])
    if rounding.startswith("two"):
        assert max(ratio) <= 1
    else:
        assert np.median(ratio) > 1

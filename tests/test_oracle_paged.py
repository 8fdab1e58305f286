"""The paged-cache oracle against what its definitions fix: pages form a
partition, slots are distinct, and attention over the cache equals dense causal
attention however the tokens are cut into steps."""
import numpy as np
import pytest
import torch

from oracle import paged as OP


@pytest.mark.parametrize("page", [4, 16])
@pytest.mark.parametrize("seed", [0, 1])
def test_plan_steps_partition_the_pool(page, seed):
    rng = np.random.default_rng(seed)
    requests, width, pages = 7, 8, 40
    free = rng.permutation(pages)
    left = pages
    cached = np.zeros(requests, dtype=np.int64)
    table = np.full((requests, width), -1)
    seen = {}
    for _ in range(5):
        fresh = rng.integers(0, page + 3, requests)
        fresh = np.minimum(fresh, width * page - cached)
        total = int(fresh.sum())
        before = left
        q_start, kv, table, slots, pos, left, fits = OP.plan(page, cached, fresh, free, left, table, total + 3)
        assert fits and q_start[-1] == total and (slots[total:] == -1).all() and (pos[total:] == 0).all()
        need = sum(-(-int(a) // page) - -(-int(c) // page) for a, c in zip(kv, cached))
        assert before - left == need
        for b in range(requests):
            for j, t in enumerate(range(q_start[b], q_start[b + 1])):
                assert pos[t] == cached[b] + j
                assert seen.setdefault(int(slots[t]), (b, int(pos[t]))) == (b, int(pos[t]))
        cached = kv
    used = table[table >= 0]
    assert len(set(used.tolist())) == len(used) and len(used) + left == pages
    assert len(seen) == int(cached.sum())


def test_plan_reports_what_does_not_fit():
    t = np.full((2, 2), -1)
    assert not OP.plan(4, [0, 0], [4, 5], np.arange(2), 2, t, 9)[6]
    assert OP.plan(4, [0, 0], [4, 5], np.arange(3), 3, t, 9)[6]
    assert not OP.plan(4, [0, 0], [9, 0], np.arange(9), 9, t, 9)[6]
    assert not OP.plan(4, [-1, 0], [1, 1], np.arange(9), 9, t, 9)[6]
    assert not OP.plan(4, [0, 0], [4, 4], np.arange(9), 9, t, 7)[6]


@pytest.mark.parametrize("heads,kv_heads", [(4, 4), (6, 2), (3, 1)])
def test_attention_equals_dense_in_any_steps(heads, kv_heads):
    rng = np.random.default_rng(3)
    page, s, d = 4, 13, 8
    q, k, v = rng.normal(size=(s, heads, d)), rng.normal(size=(s, kv_heads, d)), rng.normal(size=(s, kv_heads, d))
    g = heads // kv_heads
    tq, tk, tv = (torch.from_numpy(x).transpose(0, 1) for x in (q, k.repeat(g, 1), v.repeat(g, 1)))
    want = torch.nn.functional.scaled_dot_product_attention(tq, tk, tv, is_causal=True).transpose(0, 1).numpy()
    pools = [np.full((9, page, kv_heads, d), np.nan) for _ in range(2)]
    table, free, left = np.full((1, 5), -1), rng.permutation(9), 9
    got, lens = [], [5, 1, 6, 1]
    cached = [0]
    for n in lens:
        q_start, kv, table, slots, pos, left, fits = OP.plan(page, cached, [n], free, left, table, n)
        assert fits
        at = slice(cached[0], cached[0] + n)
        pools = [OP.store(pools[0], k[at], slots), OP.store(pools[1], v[at], slots)]
        o, lse, _, _ = OP.attention(q[at], pools[0], pools[1], table, q_start, kv, d ** -0.5)
        got.append(o)
        cached = kv
    np.testing.assert_allclose(np.concatenate(got), want, rtol=1e-12, atol=1e-13)


def test_attention_rows_without_keys():
    q = np.ones((3, 1, 8))
    pool = np.ones((2, 4, 1, 8))
    o, lse, _, _ = OP.attention(q, pool, pool, np.array([[0]]), [0, 3], [1], 1.0)
    assert (o[:2] == 0).all() and np.isneginf(lse[:2]).all() and (o[2] == 1).all() and lse[2, 0] == 8.0

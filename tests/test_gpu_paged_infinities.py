"""Attention over the paged cache where keys that a row sees have scores of
-infinity: softmax gives them a probability of 0, and a row with no other
score 0 / 0."""
import pytest
import torch

import tensor_transformer_layer_cube_gb300 as t
from tests.test_gpu_paged import Case, compare
from tests.test_gpu_paged_order import want64

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ctx():
    c = t.tp3d_create(0)
    yield c
    t.tp3d_destroy(c)


def lowest(c, b, positions, head):
    """Keys of -infinity in column 0, where the tests make every query positive."""
    for x in positions:
        c.kp[int(c.table[b, x // c.page]), x % c.page, head, 0] = -torch.inf


# one and several rows of the kernel for few, rows of the kernel for many; whole items and items in several parts
SHAPES = [(300, 1, 4), (300, 5, 4), (300, 140, 4), (9000, 1, 2), (9000, 6, 4), (9000, 200, 2), (40000, 100, 2)]


@pytest.mark.parametrize("kv,new,heads", SHAPES)
@pytest.mark.parametrize("d", [64, 128])
def test_rows_whose_scores_are_all_lowest(ctx, kv, new, heads, d):
    c = Case([kv, 77, kv], [new, new if new < 77 else 70, new], heads, 2, d, 64, seed=new)
    c.q[..., 0] = c.q[..., 0].abs() + 1
    clean, cl = c.run(ctx)
    lowest(c, 0, range(kv), 1)
    o, l = c.run(ctx)
    assert t.tp3d_sync_status(ctx) == 0
    hit = torch.zeros_like(l, dtype=torch.bool)
    hit[:new, heads // 2:] = True
    assert bool(o[hit].isnan().all()) and bool(torch.isneginf(l[hit]).all())
    assert torch.equal(o[~hit], clean[~hit]) and torch.equal(l[~hit], cl[~hit])


@pytest.mark.parametrize("kv,new,heads", SHAPES)
@pytest.mark.parametrize("d", [64, 128])
def test_some_of_the_scores_lowest(ctx, kv, new, heads, d):
    # the first keys (whole parts of a row where it is split), and single ones
    c = Case([kv], [new], heads, heads // 2, d, 64, seed=new, v_mean=0.5)
    gone = [*range(kv // 2), kv // 2 + 3, kv - new - 1]
    c.q[..., 0] = c.q[..., 0].abs() + 1
    before = c.kp.clone()
    lowest(c, 0, gone, 0)
    o, l = c.run(ctx)
    assert t.tp3d_sync_status(ctx) == 0
    # the definition on the keys that are left, for the heads of the key/value head that has lost some
    c.kp, changed = before, c.kp
    want = [x[:, :2] for x in want64(c, gone)]
    c.kp = changed
    c.q_start = c.q_start[:2]
    compare(c, o[:, :2], l[:, :2], want)
    # an infinite value behind a probability of 0 is not silent: all these rows see its key
    c.vp[int(c.table[0, 5 // 64]), 5, 0, 7] = float("inf")
    got, gl = c.run(ctx)
    assert t.tp3d_sync_status(ctx) == 0
    hit = torch.zeros_like(o, dtype=torch.bool)
    hit[:, :2, 7] = True
    assert torch.equal(gl, l) and torch.equal(got[~hit], o[~hit]) and not bool(got[hit].isfinite().any())

"""The paged attention's probabilities keep 16 bits: elements that cancel are
held to the bound of paged_util.py, which those of one bf16 term exceed
(test_paged_precision.py)."""
import numpy as np
import pytest
import torch

import tensor_transformer_layer_cube_gb300 as t
from tests.gpu_util import device
from tests.paged_util import bound, cancelling_values
from tests.test_gpu_paged import Case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ctx():
    c = t.tp3d_create(0)
    yield c
    t.tp3d_destroy(c)


# kernel for few rows: one row, rows of a group, several tokens, two blocks of rows; with four warps a CTA (many
# requests) and eight.  Kernel for many: one and two query tiles, a ragged last key tile, several pairs of tiles
@pytest.mark.parametrize("requests", [2, 40])
@pytest.mark.parametrize("kv,new,heads,kv_heads", [
    (40, 1, 4, 4), (33, 1, 8, 2), (60, 3, 8, 2), (60, 21, 4, 2), (50, 17, 2, 2), (128, 64, 4, 1), (130, 130, 2, 2),
    (200, 150, 6, 3), (300, 280, 2, 2)])
@pytest.mark.parametrize("d", [64, 128])
def test_probabilities_of_two_terms(ctx, requests, kv, new, heads, kv_heads, d):
    c = Case([kv] * requests, [new] * requests, heads, kv_heads, d, 16, std=0.05, seed=kv)
    rng, ids = np.random.default_rng(new), [torch.from_numpy(c.table[b, :-(-kv // 16)]).to(device()) for b in range(requests)]
    at = []
    for b in range(min(requests, 4)):
        q = c.q[b * new:(b + 1) * new].double().cpu().numpy()
        k = c.kp[ids[b]].flatten(0, 1)[:kv].double().cpu().numpy()
        v, cancels = cancelling_values(rng, q, k, c.scale)
        rows = c.vp[ids[b]].flatten(0, 1)
        rows[:kv] = torch.from_numpy(v).to(torch.bfloat16).to(device())
        c.vp[ids[b]] = rows.view(-1, 16, kv_heads, d)
        at += [(b * new + j, i, col) for j, i, col in cancels]
    o, _ = c.run(ctx)
    assert t.tp3d_sync_status(ctx) == 0
    want, _, absum, amax = c.want()
    keys = np.tile(np.repeat(kv - new + 1.0 + np.arange(new)[:, None], heads, 1), (requests, 1))
    err, tol = np.abs(o.double().cpu().numpy() - want), bound(want, absum, amax, keys)
    assert (err <= tol).all(), (err / tol).max()
    x = tuple(np.array(at).T)
    assert (np.abs(want[x]) <= 2.0 ** -20 * absum[x]).all()  # they do cancel: their bound is that of the probabilities

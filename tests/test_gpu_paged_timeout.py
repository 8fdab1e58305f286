"""The bounded waits of the paged attention's kernel for many rows, made to run
out on purpose (as test_gpu_timeout.py does for the GEMM): its producers stop
loading after a given number of key and value tiles, so every role's next wait
can only run out.  The CTAs let what they issued land and return, the host reads
TP3D_ETIMEOUT, and the same call then gives what it gave before, bit for bit:
the unfinished counts of split items, too, are cleared with the error."""
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
    t.tp3d_inject_load_stall(c, -1)
    t.tp3d_set_wait_limit_ns(c, 0)
    t.tp3d_destroy(c)


# 28 tiles of keys and values a CTA, most items in parts.  Stalls before anything is loaded, with a key tile and not
# its values, in the ring's first and later rounds, and after some CTAs have ended
@pytest.mark.parametrize("stall", [0, 1, 2, 5, 12, 27])
@pytest.mark.parametrize("d", [64, 128])
def test_wait_runs_out_then_the_call_recovers(ctx, stall, d):
    c = Case([9000, 300, 8000], [200, 1, 130], 16, 16, d, 64, seed=stall)
    want, wl = c.run(ctx)
    assert t.tp3d_sync_status(ctx) == 0
    if stall == 0:
        compare(c, want, wl, want64(c))
    assert t.tp3d_set_wait_limit_ns(ctx, 20_000_000) == 0
    assert t.tp3d_inject_load_stall(ctx, stall) == 0
    o, _ = c.run(ctx)
    assert t.STATUS[t.tp3d_sync_status(ctx)] == "TP3D_ETIMEOUT"
    # the single token is the other kernel's
    assert torch.equal(o[200].view(torch.int16), want[200].view(torch.int16))
    assert t.tp3d_inject_load_stall(ctx, -1) == 0
    assert t.tp3d_set_wait_limit_ns(ctx, 0) == 0
    for _ in range(2):
        o, l = c.run(ctx)
        assert t.tp3d_sync_status(ctx) == 0
        assert torch.equal(o.view(torch.int16), want.view(torch.int16)) and torch.equal(l, wl)


def test_single_tokens_do_not_see_the_hook(ctx):
    c = Case([700, 40], [1, 1], 8, 2, 64)
    want, _ = c.run(ctx)
    assert t.tp3d_inject_load_stall(ctx, 0) == 0
    o, _ = c.run(ctx)
    assert t.tp3d_sync_status(ctx) == 0 and torch.equal(o, want)
    assert t.tp3d_inject_load_stall(ctx, -1) == 0

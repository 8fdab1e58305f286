"""The example server against the layer: the same tokens in prompt chunks and one
at a time through the paged cache, and in one tp3d_layer_fwd.

Both store activations in bf16 between steps and are held to 1e-2 of the exact
layer (max-normalised and Frobenius); so they may differ by 2e-2 in either."""
import numpy as np
import pytest

from examples import serve_layer
from oracle.metrics import BF16_TOL, fro_err, max_rel_err

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("case", [dict(), dict(q=1, heads=4, hidden=256, batch=3, seq=128,
                                               chunks=((128, 1, 70), (0, 30, 1)))])
def test_served_layer_equals_the_whole_forward(case):
    got, want = (t.float().cpu().numpy().astype(np.float64) for t in serve_layer.compare(**case))
    assert np.isfinite(got).all()
    assert max_rel_err(got, want) <= 2 * BF16_TOL and fro_err(got, want) <= 2 * BF16_TOL

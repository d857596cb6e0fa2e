"""Where a NaN of one token's input goes in the gradients of the vocabulary
loss: the products of the formula, with dz = 0 for a token that is ignored."""
import numpy as np
import pytest
import torch

from tests import test_gpu_cross_entropy as ce
from tests.step_util import f64

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def B():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from top_routing_grouped_moe_gb300 import _binding
    return _binding


@pytest.mark.parametrize("value", [float("nan"), float("inf")])
def test_ignored_token(B, value):
    """dx and the losses of all other tokens are what they are without it; in dW
    = dz^T x its row meets dz = 0 and 0 x NaN is NaN, in the channels that hold
    one and in no other."""
    T, V, d = 200, 300, 128
    x, W, t, up = ce._inputs(T, V, d, seed=8)
    t[:] = torch.arange(T) % V
    t[9] = -1
    x[9] = 0.0
    clean = ce._run(B, x, W, t, up, 1e-3)
    x[9, 5], x[9, 77] = value, value
    out = ce._run(B, x, W, t, up, 1e-3)
    rest = np.arange(T) != 9
    assert not f64(out["dx"])[9].any() and float(out["loss"][9]) == 0.0
    for k in ("loss", "lse", "dx"):
        assert np.array_equal(f64(out[k])[rest], f64(clean[k])[rest]), k
    dW, ref = f64(out["dW"]), f64(clean["dW"])
    hit = np.isin(np.arange(d), (5, 77))
    assert np.isnan(dW[:, hit]).all() and np.array_equal(dW[:, ~hit], ref[:, ~hit])
    assert B.moe_device_status() == 0

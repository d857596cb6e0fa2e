"""A clip whose coefficient is 1 passes every bit, whatever the offsets: the
payload of a NaN too, in the elements around the 16-byte vectors and in outputs
at another offset from a 16-byte boundary."""
import pytest
import torch

pytestmark = pytest.mark.gpu

BITS = {torch.bfloat16: (torch.int16, 0x7FA5), torch.float16: (torch.int16, 0x7D35),
        torch.float32: (torch.int32, 0x7FA51234)}


@pytest.fixture(scope="module")
def B():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from top_routing_grouped_moe_gb300 import _binding
    return _binding


@pytest.mark.parametrize("dt", list(BITS))
@pytest.mark.parametrize("at_in,at_out", [(0, 0), (1, 1), (3, 3), (1, 2), (0, 3)])
def test_unscaled_gradients_keep_their_bits(B, dt, at_in, at_out):
    n = 1003
    bits, nan = BITS[dt]
    flat = torch.randn(n + 8, device="cuda").to(dt)
    g = flat[at_in:at_in + n]
    g.view(bits)[::2] = nan
    out = torch.zeros(n + 8, dtype=dt, device="cuda")
    o = out[at_out:at_out + n]
    plan = B.GradList([g], [o])
    size = B.moe_grad_clip_workspace(plan)
    ws = torch.empty(size, dtype=torch.uint8, device="cuda")
    norm, coef = torch.empty(1, device="cuda"), torch.empty(1, device="cuda")
    B.moe_grad_clip(plan, 1.0, norm, coef, ws, size)
    assert bool(norm.isnan()) and float(coef) == 1.0
    assert torch.equal(o.view(bits), g.view(bits))
    assert not out[:at_out].any() and not out[at_out + n:].any()
    assert B.moe_device_status() == B.MOE_ERR_RANGE

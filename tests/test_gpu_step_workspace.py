"""One workspace, sized for the longest batch, serves every shorter one."""
import pytest
import torch

from tests.step_util import Rand, dev, same_bits

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def B():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from top_routing_grouped_moe_gb300 import _binding
    return _binding


def test_embedding_gradient(B):
    d, V, longest = 2048, 500, 8192
    n = B.moe_embedding_workspace(longest, V, d)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    R = Rand(1)
    ids, dout = dev(R.ints(0, V, longest)), dev(R.normal(longest, d))
    for T in (longest, 2401, 2400, 1, 37):
        own = B.moe_embedding_workspace(T, V, d)
        g = [torch.empty(V, d, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
        B.moe_embedding_bwd(dout[:T], ids[:T], T, V, d, 1.0, False, g[0], ws, n)
        B.moe_embedding_bwd(dout[:T], ids[:T], T, V, d, 1.0, False, g[1],
                            torch.empty(own, dtype=torch.uint8, device="cuda"), own)
        assert same_bits(*g), T


@pytest.mark.parametrize("d,V,longest", [(64, 50257, 150), (1024, 1000, 1200), (512, 5544, 700)])
def test_cross_entropy(B, d, V, longest):
    R = Rand(2)
    x, W, t = dev(R.normal(longest, d)), dev(R.normal(V, d, scale=0.05)), dev(R.ints(0, V, longest))
    up = torch.full((longest,), 1.0 / longest, device="cuda")
    for grad in (False, True):
        n = B.moe_cross_entropy_workspace(longest, d, V, 0, grad)
        ws = torch.empty(n, dtype=torch.uint8, device="cuda")
        for T in sorted({1, 5, 100, 128, 129, 300, 511, 512, 600, 767, 900, 1024, longest} - set(range(longest + 1, 2000))):
            loss, lse = torch.empty(T, device="cuda"), torch.empty(T, device="cuda")
            B.moe_cross_entropy(x, W, t, T, d, V, 0.0, loss, lse, ws, n)
            if grad:
                dx, dW = torch.empty(T, d, dtype=torch.bfloat16, device="cuda"), torch.empty_like(W)
                B.moe_cross_entropy_bwd(x, W, t, lse, up, T, d, V, 0.0, 0, dx, dW, ws, n)
    torch.cuda.synchronize()
    assert B.moe_device_status() == 0

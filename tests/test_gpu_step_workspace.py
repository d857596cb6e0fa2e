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

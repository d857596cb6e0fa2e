"""A model's step uses the same buffers every time: a graph captured on the
first one replays what a later eager step computes, in the same places."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def lm():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from top_routing_grouped_moe_gb300 import lm
    return lm


@pytest.mark.parametrize("blocks", [1, 3])
def test_step_keeps_its_buffers(lm, blocks):
    T, V, d = 70, 90, 128
    m = lm.MoELM(T, V, d, blocks, E=8, k=2, H=128, Hs=128)
    p = m.init_weights(seed=1)
    g = torch.Generator(device="cuda").manual_seed(2)
    ids = torch.randint(0, V, (T,), generator=g, device="cuda", dtype=torch.int32)
    targets = (ids * 7 + 3) % V
    up = torch.full((T,), 1.0 / T, device="cuda")
    at = {k: v.data_ptr() for k, v in vars(m).items() if isinstance(v, torch.Tensor)}
    bits = []
    for _ in range(3):
        m.forward(ids, targets, p)
        m.backward(ids, targets, up, p)
        torch.cuda.synchronize()
        bits.append({k: v.clone() for k, v in m.grads.items()})
        assert {k: v.data_ptr() for k, v in vars(m).items() if isinstance(v, torch.Tensor)} == at
    for k in bits[0]:
        assert torch.equal(bits[0][k], bits[1][k]) and torch.equal(bits[0][k], bits[2][k]), k

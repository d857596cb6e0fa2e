"""Token ids and targets that are not what the kernels read are refused before
anything reaches a device (no GPU)."""
import pytest
import torch


@pytest.fixture(scope="module")
def L():
    import __graft_entry__
    __graft_entry__.build()
    from top_routing_grouped_moe_gb300 import _binding
    return _binding


P, BIG, T = 1 << 12, 1 << 40, 6  # a stand-in device address; never dereferenced

CALLS = {
    "embedding": lambda L, i: L.moe_embedding(P, i, T, 10, 64, 1.0, P, 0),
    "embedding_bwd": lambda L, i: L.moe_embedding_bwd(P, i, T, 10, 64, 1.0, 0, P, P, BIG, 0),
    "cross_entropy": lambda L, i: L.moe_cross_entropy(P, P, i, T, 64, 10, 0.0, P, P, P, BIG, 0),
    "cross_entropy_bwd": lambda L, i: L.moe_cross_entropy_bwd(P, P, i, P, P, T, 64, 10, 0.0, 0, P, P, P, BIG, 0),
}


@pytest.mark.parametrize("call", list(CALLS))
@pytest.mark.parametrize("dtype", [torch.int64, torch.int16, torch.uint8, torch.float32])
def test_other_types(L, call, dtype):
    with pytest.raises(TypeError):
        CALLS[call](L, torch.zeros(T, dtype=dtype))


@pytest.mark.parametrize("call", list(CALLS))
def test_slices_of_a_batch_and_short_ones(L, call):
    batch = torch.zeros(2, T // 2 + 1, dtype=torch.int32)
    for ids in (batch[:, 1:], batch.t(), torch.zeros(2 * T, dtype=torch.int32)[::2], torch.zeros(T - 1, dtype=torch.int32)):
        with pytest.raises(ValueError):
            CALLS[call](L, ids)


def test_gradients_on_the_host(L):
    """A list of their addresses would be read by the GPU."""
    g = torch.ones(8)
    for outs in (None, [g], [torch.empty(8)]):
        with pytest.raises(ValueError):
            L.GradList([g], outs)

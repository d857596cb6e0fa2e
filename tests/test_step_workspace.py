"""Workspace sizes of the training-step operators never fall as the batch grows:
a buffer sized for the longest batch serves every shorter one (no GPU)."""
import pytest


@pytest.fixture(scope="module")
def L():
    import __graft_entry__
    __graft_entry__.build()
    from top_routing_grouped_moe_gb300 import _binding
    return _binding


def _rising(sizes):
    return all(a <= b for a, b in zip(sizes, sizes[1:]))


@pytest.mark.parametrize("d", [64, 1024, 1088, 2048, 4096, 8192, 65536])
def test_embedding(L, d):
    assert _rising([L.moe_embedding_workspace(T, 1000, d) for T in [*range(1, 6000), *range(6000, 40000, 31)]])


@pytest.mark.parametrize("d,V", [(64, 50257), (320, 5544), (1024, 1000), (1024, 50257), (4096, 5544), (4096, 50257),
                                 (4096, 1)])
@pytest.mark.parametrize("grad,piece", [(False, 0), (True, 0), (True, 600), (True, 1 << 20)])
def test_cross_entropy(L, d, V, grad, piece):
    tokens = [*range(1, 1300), *range(1300, 9000, 37), *range(9000, 70000, 1021)]
    assert _rising([L.moe_cross_entropy_workspace(T, d, V, piece, grad) for T in tokens])

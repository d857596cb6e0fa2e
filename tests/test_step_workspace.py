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

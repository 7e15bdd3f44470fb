"""Sizes that the page calls refuse have no workspace size."""
import pytest

from hybrid_local_global_b200 import native

MOST = [(4096, 1 << 18, 1 << 20), (1, 1 << 30, 1), (4096, 1, 1)]


@pytest.mark.parametrize("sizes", MOST, ids=str)
def test_workspace_size(sizes):
    assert native.gemma_kv_pages_workspace_size(*sizes) > 0
    for i, limit in enumerate((4096, (1 << 30) // sizes[0], 1 << 20)):
        over = list(sizes)
        over[i] = limit + 1
        assert native.gemma_kv_pages_workspace_size(*over) == 0, over

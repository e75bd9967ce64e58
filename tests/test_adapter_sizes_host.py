"""Workspace of the adapter calls, on the host (no GPU)."""
import pytest

from helpers import build_lib


@pytest.fixture(scope="module")
def ql():
    return build_lib()


def test_only_ranks_of_4_modulo_8_hold_a_padded_b(ql):
    """The tensor-core kernels read B with rows of a multiple of 8 ranks; odd ranks never reach them."""
    size = lambda r: ql.adapters_workspace_size(16, 14336, 4096, 1024, r)  # noqa: E731
    pad = 1024 * 14336 * 2
    assert size(4) >= pad * 8 and size(12) >= pad * 16
    for r in (1, 2, 3, 5, 6, 7, 8, 9, 15, 16, 127):
        assert size(r) < pad * 8, r

"""Limits of the 8-bit checkpoint calls, on the host (no GPU)."""
import ctypes as C

import pytest
import torch

from helpers import build_lib

P = C.c_void_p(1 << 20)  # non-null and aligned; never dereferenced on these paths


@pytest.fixture(scope="module")
def ql():
    return build_lib()


def test_tokens_of_a_weight_gradient(ql):
    call = lambda m: ql.lib().pergroup_wgrad(P, 1, m, 64, P, P, 64, 64, P, None, None)  # noqa: E731
    assert call((1 << 24) + 1) == call(1 << 30) == ql.QLIN_ERR_UNSUPPORTED
    if not torch.cuda.is_available():
        assert call(1 << 24) == ql.QLIN_ERR_DEVICE

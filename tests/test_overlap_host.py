"""Outputs of the adapter calls over what they read, on the host (no GPU): refused before anything else is asked."""
import ctypes as C

import pytest
import torch

from helpers import build_lib

BASE, BIG = 1 << 20, 1 << 40


def at(i):
    """The i-th of buffers that lie far apart; never dereferenced."""
    return C.c_void_p(BASE + (i << 34))


@pytest.fixture(scope="module")
def ql():
    return build_lib()


def forward(ql, **k):
    d = dict(x=at(0), a=at(1), b=at(2), s=at(3), plan=at(4), base=at(5), out=at(6), u=at(7), ws=at(8))
    d.update(k)
    return ql.lib().qlin_adapters_forward(d["x"], 1, 40, 64, d["a"], d["b"], d["s"], 2, 8, 64, d["plan"], BIG, d["base"],
                                          d["out"], d["u"], d["ws"], BIG, None)


def backward(ql, **k):
    d = dict(dy=at(0), a=at(1), b=at(2), s=at(3), plan=at(4), u=at(5), x=None, q=at(6), qs=at(7), dxb=at(8), dx=at(9),
             da=at(10), db=at(11), ws=at(12))
    d.update(k)
    return ql.lib().qlin_adapters_backward(d["dy"], 1, 40, 64, d["a"], d["b"], d["s"], 2, 8, 64, d["plan"], BIG, d["u"],
                                           d["x"], d["q"], d["qs"], 64, d["dxb"], d["dx"], d["da"], d["db"], d["ws"],
                                           BIG, None)


def near(i, off):
    return C.c_void_p(BASE + (i << 34) + off)


@pytest.mark.parametrize("k", [dict(u=at(0)), dict(u=at(1)), dict(u=at(2)), dict(u=at(3)), dict(u=at(4)), dict(u=at(5)),
                               dict(u=at(6)), dict(u=near(0, 40 * 64 * 2 - 4)), dict(u=near(0, 4 - 40 * 8 * 4)),
                               dict(out=at(0)), dict(out=at(1)), dict(out=at(2)), dict(out=at(3)), dict(out=at(4)),
                               dict(out=near(5, 2))], ids=str)
def test_forward(ql, k):
    assert forward(ql, **k) == ql.QLIN_ERR_INVALID_ARG


@pytest.mark.parametrize("k", [dict(dx=at(i)) for i in (0, 1, 2, 3, 4, 5, 6, 7)] + [dict(dx=near(8, 2))]
                         + [dict(dx=near(7, -40 * 64 * 2 + 2))], ids=str)
def test_backward(ql, k):
    assert backward(ql, **k) == ql.QLIN_ERR_INVALID_ARG


@pytest.mark.skipif(torch.cuda.is_available(), reason="these calls would be launched, at addresses of nothing")
def test_buffers_that_touch_are_apart(ql):
    fine = forward(ql)
    assert fine != ql.QLIN_ERR_INVALID_ARG
    assert forward(ql, u=near(0, 40 * 64 * 2)) == forward(ql, u=near(0, -40 * 8 * 4)) == fine
    assert forward(ql, out=at(5)) == forward(ql, base=None) == fine  # in place
    assert backward(ql) == backward(ql, dx=at(8)) == backward(ql, dx=None, dxb=None) == fine

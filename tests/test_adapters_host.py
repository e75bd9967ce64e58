"""Refusals and sizes of the adapter, checkpoint and weight-gradient calls, on the host (no GPU)."""
import ctypes as C

import pytest
import torch

from helpers import build_lib

P = C.c_void_p(1 << 20)  # non-null and aligned; never dereferenced on these paths
BIG = 1 << 40            # "enough" for every plan and workspace


def at(off):
    return C.c_void_p((1 << 20) + off)


@pytest.fixture(scope="module")
def ql():
    return build_lib()


def forward(ql, **k):
    d = dict(x=P, dt=1, M=4, K=64, a=P, b=P, s=P, L=2, R=8, N=64, plan=P, pn=BIG, base=None, out=at(1 << 30), u=None,
             ws=P, wn=BIG)
    d.update(k)
    return ql.lib().qlin_adapters_forward(d["x"], d["dt"], d["M"], d["K"], d["a"], d["b"], d["s"], d["L"], d["R"],
                                          d["N"], d["plan"], d["pn"], d["base"], d["out"], d["u"], d["ws"], d["wn"],
                                          None)


def backward(ql, **k):
    d = dict(dy=P, dt=1, M=4, N=64, a=P, b=P, s=P, L=2, R=8, K=128, plan=P, pn=BIG, u=P, x=P, q=None, qs=None, g=0,
             dxb=None, dx=at(1 << 30), da=P, db=P, ws=P, wn=BIG)
    d.update(k)
    return ql.lib().qlin_adapters_backward(d["dy"], d["dt"], d["M"], d["N"], d["a"], d["b"], d["s"], d["L"], d["R"],
                                           d["K"], d["plan"], d["pn"], d["u"], d["x"], d["q"], d["qs"], d["g"],
                                           d["dxb"], d["dx"], d["da"], d["db"], d["ws"], d["wn"], None)


@pytest.mark.parametrize("k", [dict(x=None), dict(a=None), dict(b=None), dict(s=None), dict(plan=None), dict(out=None),
                               dict(M=0), dict(M=-1), dict(K=0), dict(N=0), dict(L=0), dict(R=0), dict(pn=16),
                               dict(out=P), dict(out=at(128)), dict(base=at((1 << 30) + 128)), dict(u=at(1 << 30))],
                         ids=str)
def test_forward_invalid(ql, k):
    assert forward(ql, **k) == ql.QLIN_ERR_INVALID_ARG


@pytest.mark.parametrize("k", [dict(dt=3), dict(R=129), dict(L=1025), dict(M=(1 << 20) + 1), dict(K=1 << 21),
                               dict(N=1 << 21)], ids=str)
def test_forward_unsupported(ql, k):
    assert forward(ql, **k) == ql.QLIN_ERR_UNSUPPORTED


@pytest.mark.parametrize("k", [dict(x=at(1)), dict(a=at(1)), dict(b=at(3)), dict(out=at((1 << 30) + 1)),
                               dict(s=at(2)), dict(u=at(2)), dict(plan=at(4)), dict(dt=0, x=at(2))], ids=str)
def test_forward_misaligned(ql, k):
    assert forward(ql, **k) == ql.QLIN_ERR_MISALIGNED


@pytest.mark.parametrize("k", [dict(ws=None), dict(wn=0), dict(ws=at(16))], ids=str)
def test_workspace_refused(ql, k):
    assert forward(ql, **k) == ql.QLIN_ERR_WORKSPACE
    assert backward(ql, **k) == ql.QLIN_ERR_WORKSPACE


@pytest.mark.parametrize("k", [dict(dy=None), dict(u=None), dict(da=None), dict(db=None), dict(plan=None),
                               dict(x=None), dict(q=P, qs=P, g=64), dict(x=None, q=P, qs=None, g=64),
                               dict(dx=None, dxb=P), dict(x=None, q=P, qs=P, g=64, K=96), dict(M=0), dict(R=0),
                               dict(dx=P), dict(dxb=at((1 << 30) + 64))], ids=str)
def test_backward_invalid(ql, k):
    assert backward(ql, **k) == ql.QLIN_ERR_INVALID_ARG


@pytest.mark.parametrize("k", [dict(x=None, q=P, qs=P, g=32), dict(x=None, q=P, qs=P, g=0), dict(dt=-1), dict(R=200),
                               dict(L=2000)], ids=str)
def test_backward_unsupported(ql, k):
    assert backward(ql, **k) == ql.QLIN_ERR_UNSUPPORTED


@pytest.mark.parametrize("k", [dict(dy=at(1)), dict(u=at(1)), dict(dx=at((1 << 30) + 1)), dict(da=at(1)),
                               dict(x=None, q=P, qs=at(2), g=64)], ids=str)
def test_backward_misaligned(ql, k):
    assert backward(ql, **k) == ql.QLIN_ERR_MISALIGNED


def test_plan_refusals(ql):
    L = ql.lib()
    assert L.qlin_adapters_plan(None, 4, 2, P, BIG, None) == ql.QLIN_ERR_INVALID_ARG
    assert L.qlin_adapters_plan(P, 4, 2, None, BIG, None) == ql.QLIN_ERR_INVALID_ARG
    assert L.qlin_adapters_plan(P, 0, 2, P, BIG, None) == ql.QLIN_ERR_INVALID_ARG
    assert L.qlin_adapters_plan(P, 4, 0, P, BIG, None) == ql.QLIN_ERR_INVALID_ARG
    assert L.qlin_adapters_plan(P, 4, 2, P, 16, None) == ql.QLIN_ERR_INVALID_ARG
    assert L.qlin_adapters_plan(P, 4, 1025, P, BIG, None) == ql.QLIN_ERR_UNSUPPORTED
    assert L.qlin_adapters_plan(P, (1 << 20) + 1, 2, P, BIG, None) == ql.QLIN_ERR_UNSUPPORTED
    assert L.qlin_adapters_plan(P, 4, 2, at(8), BIG, None) == ql.QLIN_ERR_MISALIGNED
    assert L.qlin_adapters_plan(at(2), 4, 2, P, BIG, None) == ql.QLIN_ERR_MISALIGNED


def test_sizes(ql):
    L = ql.lib()
    assert L.qlin_adapters_plan_size(0, 1) == L.qlin_adapters_plan_size(1, 0) == 0
    assert L.qlin_adapters_plan_size((1 << 20) + 1, 1) == L.qlin_adapters_plan_size(1, 1025) == 0
    for m, n in [(1, 1), (5, 3), (4096, 4), (1 << 20, 1024)]:
        # tokens by adapter, and a tile of 8 and of 128 for each part of a segment
        assert L.qlin_adapters_plan_size(m, n) >= 4 * (m + 4 * (m // 8) + 4 * (m // 128))
    assert ql.adapters_workspace_size(0, 64, 64, 1, 8) == 0
    assert ql.adapters_workspace_size(4, 64, 64, 1, 129) == 0
    assert ql.adapters_workspace_size(4, 64, 64, 1, 8) % 256 == 0


def restore(ql, q=P, s=P, N=4, K=64, g=64, out=P, dt=1):
    return ql.lib().qlin_dequantize_int8_groups(q, s, N, K, g, out, dt, None)


def wgrad(ql, dy=P, dt=1, M=4, N=64, q=P, s=P, K=64, g=64, dw=P, db=None):
    return ql.lib().pergroup_wgrad(dy, dt, M, N, q, s, K, g, dw, db, None)


def test_checkpoint_refusals(ql):
    for k in [dict(q=None), dict(s=None), dict(out=None), dict(N=0), dict(K=0), dict(K=96)]:
        assert restore(ql, **k) == ql.QLIN_ERR_INVALID_ARG, k
    for k in [dict(g=32), dict(g=0), dict(dt=3)]:
        assert restore(ql, **k) == ql.QLIN_ERR_UNSUPPORTED, k
    for k in [dict(q=at(8)), dict(out=at(8)), dict(s=at(2))]:
        assert restore(ql, **k) == ql.QLIN_ERR_MISALIGNED, k
    for k in [dict(dy=None), dict(q=None), dict(s=None), dict(dw=None), dict(M=0), dict(N=0), dict(K=0), dict(K=96)]:
        assert wgrad(ql, **k) == ql.QLIN_ERR_INVALID_ARG, k
    for k in [dict(dt=0), dict(dt=3), dict(g=32), dict(K=1 << 21), dict(N=1 << 21)]:
        assert wgrad(ql, **k) == ql.QLIN_ERR_UNSUPPORTED, k
    for k in [dict(N=60), dict(dy=at(8)), dict(q=at(4)), dict(dw=at(2)), dict(s=at(1)), dict(db=at(1))]:
        assert wgrad(ql, **k) == ql.QLIN_ERR_MISALIGNED, k


def test_valid_calls_reach_the_device_check(ql):
    if torch.cuda.is_available():
        pytest.skip("a GPU is present")
    assert forward(ql) == forward(ql, base=at(1 << 30)) == ql.QLIN_ERR_DEVICE
    assert backward(ql) == backward(ql, dx=None) == backward(ql, x=None, q=P, qs=P, g=64) == ql.QLIN_ERR_DEVICE
    assert restore(ql) == wgrad(ql) == ql.QLIN_ERR_DEVICE
    assert ql.lib().qlin_adapters_plan(P, 4, 2, P, BIG, None) == ql.QLIN_ERR_DEVICE


def test_python_refuses_host_tensors(ql):
    with pytest.raises(ValueError):
        ql.adapters_plan(torch.zeros(4, dtype=torch.int32), 2)
    with pytest.raises(ValueError):
        ql.dequantize_int8_groups(torch.zeros(4, 64, dtype=torch.int8), torch.ones(1, 4), 64)
    with pytest.raises(ValueError):
        ql.pergroup_wgrad(torch.zeros(4, 64, dtype=torch.bfloat16), torch.zeros(4, 64, dtype=torch.int8),
                          torch.ones(1, 4), 64)

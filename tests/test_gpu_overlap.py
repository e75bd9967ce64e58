"""What a call would write lies over what it reads: refused on the host, nothing launched, nothing written."""
import ctypes as C

import pytest
import torch

import adapter_ref as ref
from helpers import build_lib

pytestmark = pytest.mark.gpu

M, K, N, L, R = 40, 64, 64, 2, 8


@pytest.fixture(scope="module")
def ql():
    return build_lib()


def refused(ql, name, order, args, where, onto):
    """The call with argument `where` at the address of `onto`: INVALID_ARG, and every buffer as it was."""
    before = {k: t.clone() for k, t in args.items() if isinstance(t, torch.Tensor)}
    ptr = {k: C.c_void_p(t.data_ptr()) if isinstance(t, torch.Tensor) else t for k, t in args.items()}
    ptr[where] = ptr[onto]
    status = getattr(ql.lib(), name)(*[ptr[k] for k in order.split()], None)
    torch.cuda.synchronize()
    assert status == ql.QLIN_ERR_INVALID_ARG, (where, onto)
    assert all(torch.equal(args[k], t) for k, t in before.items()), (where, onto)


def room(t, n):
    """t at the front of n bytes on a 256-byte boundary: long enough for whatever is put there."""
    flat = torch.zeros(n, dtype=torch.uint8, device="cuda")
    flat[:t.numel() * t.element_size()] = t.contiguous().view(-1).view(torch.uint8)
    return flat


def test_adapters(ql):
    d = ref.make((torch.bfloat16, M, K, N, L, R, "random"))
    plan = ql.adapters_plan(d["ids"], L)
    ws = ql.adapters_workspace_size(M, N, K, L, R, True)
    n = max(ws, 1 << 16)
    t = {k: room(d[k], n) for k in ("x", "a", "b", "scales", "base", "dy", "dx_base", "ids")}
    t.update(plan=room(plan.buffer, n), u=room(torch.zeros(M, R, device="cuda"), n), M=M, K=K, N=N, L=L, R=R, dt=1, big=n)
    q, s = ql.quantize_int8_groups(d["x"], 64)
    t.update(q=room(q, n), qs=room(s, n), g=64, none=None)
    for k in ("out", "dx", "da", "db", "ws"):
        t[k] = torch.zeros(n, dtype=torch.uint8, device="cuda")
    fwd = "x dt M K a b scales L R N plan big base out u ws big"
    for onto in ("x", "a", "b", "scales", "base", "plan", "u", "out"):
        refused(ql, "qlin_adapters_forward", fwd, t, "ws", onto)
    bwd = "dy dt M N a b scales L R K plan big u none q qs g dx_base dx da db ws big"
    read = ("dy", "a", "b", "scales", "plan", "u", "q", "qs", "dx_base")
    for where in ("da", "db", "ws"):
        for onto in read + tuple(k for k in ("dx", "da", "db", "ws") if k != where):
            refused(ql, "qlin_adapters_backward", bwd, t, where, onto)
    refused(ql, "qlin_adapters_backward", bwd.replace("none q qs", "x none none"), t, "da", "x")
    refused(ql, "qlin_adapters_plan", "ids M L plan big", t, "plan", "ids")


def test_checkpoints(ql):
    x = torch.randn(M, K, device="cuda", dtype=torch.bfloat16)
    q, s = ql.quantize_int8_groups(x, 64)
    n = 1 << 16
    t = dict(q=room(q, n), s=room(s, n), x=room(x, n), M=M, K=K, g=64, dt=1, N=K, dw=torch.zeros(n, dtype=torch.uint8, device="cuda"))
    t["db"] = torch.zeros(n, dtype=torch.uint8, device="cuda")
    t["out"] = t["dw"].clone()
    for onto in ("q", "s"):
        refused(ql, "qlin_dequantize_int8_groups", "q s M K g out dt", t, "out", onto)
    for where in ("dw", "db"):
        for onto in ("x", "q", "s", "db" if where == "dw" else "dw"):
            refused(ql, "pergroup_wgrad", "x dt M N q s K g dw db", t, where, onto)


def test_python_calls(ql):
    """The same through the binding: u in x's memory, dw in dy's."""
    buf = torch.zeros(M * K, device="cuda")
    d = ref.make((torch.float32, M, K, N, L, R, "random"))
    plan = ql.adapters_plan(d["ids"], L)
    x = buf.view(M, K)
    with pytest.raises(ql.QlinError) as e:
        ql.adapters_forward(x, d["a"], d["b"], d["scales"], plan, u=buf[:M * R].view(M, R))
    assert e.value.status == ql.QLIN_ERR_INVALID_ARG
    half = torch.zeros(64 * 64 * 2, dtype=torch.bfloat16, device="cuda")
    q, s = ql.quantize_int8_groups(torch.randn(64, 64, device="cuda"), 64)
    with pytest.raises(ql.QlinError) as e:
        ql.pergroup_wgrad(half[:4096].view(64, 64), q, s, 64, dw=half[2048:2048 + 4096].view(64, 64))
    assert e.value.status == ql.QLIN_ERR_INVALID_ARG

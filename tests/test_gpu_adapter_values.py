"""Adapters whose inner values u and v lie far from 1, outside fp16's own range or far apart from one another.  A
result is infinite where its 64-bit value lies beyond the type's range and nowhere else, and within the bounds of
adapter_ref where it is finite."""
import pytest
import torch

import adapter_ref as ref
from helpers import build_lib

pytestmark = pytest.mark.gpu

BF, HF = torch.bfloat16, torch.float16


@pytest.fixture(scope="module")
def ql():
    return build_lib()


def close(got, want, slack, what):
    """ref.close, but for values that round to an infinity in 64 bits too (either, where the slack reaches the end)."""
    top = torch.finfo(got.dtype).max * (1 + ref.half(got.dtype) / 2)  # what lies above rounds to infinity
    beyond, near = want.abs() - slack > top, want.abs() + slack > top
    inf = torch.where(want > 0, float("inf"), float("-inf"))
    same = torch.where(near, got.double() == inf, False)
    assert bool(same[beyond].all()), f"{what}: not infinite where it has to be"
    fixed = torch.where(same, 0.0, got.double())
    assert bool(fixed.isfinite().all()), f"{what}: not finite in {int((~fixed.isfinite()).sum())} places"
    ref.close(fixed.to(got.dtype), torch.where(same, 0.0, want), torch.where(same, 0.0, slack), what)


# factors of u, the scales, b, a and x: u or v far outside the type's range or far below its smallest step
SIZES = [(HF, 1e7, 1e-8, 1, 1, 1), (HF, 1e-6, 1e4, 1e-4, 1, 1), (HF, 1e-6, 1e6, 1, 1e-5, 1e-4),
         (HF, 1e5, 1e-6, 1, 1e2, 1e2), (HF, 1e9, 1e-9, 1, 1, 1), (HF, 1e-12, 1, 1, 1, 1),
         (BF, 1e30, 1e-30, 1, 1, 1), (BF, 1e-30, 1e30, 1, 1e-30, 1e-5), (BF, 1e15, 1, 1e-20, 1e10, 1)]


@pytest.mark.parametrize("M,R,kind", [(300, 16, "runs"), (257, 72, "random"), (700, 12, "blocks")])
@pytest.mark.parametrize("sizes", SIZES, ids=str)
def test_gradients_of_any_size(ql, sizes, M, R, kind):
    dt, fu, fs, fb, fa, fx = sizes
    K, N, L = 256, 264, 2
    d = ref.make((dt, M, K, N, L, R, kind), seed=5)
    gen = torch.Generator(device="cuda").manual_seed(6)
    u = torch.randn(M, R, generator=gen, device="cuda") * fu
    d["scales"] *= fs
    for k, f in (("b", fb), ("a", fa), ("x", fx)):
        d[k] = (d[k].double() * f).to(dt)
    plan = ql.adapters_plan(d["ids"], L)
    dx, da, db = ql.adapters_backward(d["dy"], d["a"], d["b"], d["scales"], plan, u, x=d["x"], dx_base=d["dx_base"])
    assert ql.device_status() == ql.QLIN_OK
    wx, mx = d["dx_base"].double(), d["dx_base"].double().abs() * 2.0 ** -23
    for i in range(L):
        m = ref.rows_of(d["ids"], i)
        a, b, sc, y, x = (t.double() for t in (d["a"][i], d["b"][i], d["scales"][i], d["dy"][m], d["x"][m]))
        v, vm = sc * (y @ b), sc.abs() * (y.abs() @ b.abs())
        wx[m] += v @ a
        mx[m] += (ref.SPLIT + ref.acc(N + R + 2)) * (vm @ a.abs())
        close(da[i], v.T @ x, (ref.SPLIT + ref.acc(N + M + 2)) * (vm.T @ x.abs()), f"da[{i}]")
        close(db[i], sc * (y.T @ u[m].double()),
              (ref.SPLIT + ref.acc(M + 2)) * sc.abs() * (y.abs().T @ u[m].double().abs()), f"db[{i}]")
    close(dx, wx, mx, "dx")


@pytest.mark.parametrize("M", [5, 200])
@pytest.mark.parametrize("dt", [HF, BF], ids=str)
def test_values_far_apart_in_one_token(ql, dt, M):
    """u of rank 0 is 2^25 times that of the others, and the odd outputs do not use rank 0: what they get is held
    within 2^-16 of its value, or (fp16) 2^-39 of the token's largest."""
    K, N, R = 256, 256, 16
    d = ref.make((dt, M, K, N, 1, R, "one"), seed=2)
    if dt == HF:
        d["a"] = (d["a"].double() * 2.0 ** -9).to(dt)
    d["a"][:, 0] = (d["a"][:, 0].double() * 2.0 ** (12 if dt == HF else 25)).to(dt)
    if dt == HF:  # the rest of the factor from x: rank 0 sees the first half of x, the others the second
        d["a"][:, 0, K // 2:] = 0
        d["a"][:, 1:, :K // 2] = 0
        d["x"] = d["x"].clamp(-4, 4)
        d["x"][:, :K // 2] *= 64
        d["x"][:, K // 2:] = (d["x"][:, K // 2:].double() * 2.0 ** -7).to(dt)
    d["b"][:, 1::2, 0] = 0
    plan = ql.adapters_plan(d["ids"], 1)
    u = torch.zeros(M, R, device="cuda")
    out = ql.adapters_forward(d["x"], d["a"], d["b"], d["scales"], plan, u=u)
    x, a, b, s = d["x"].double(), d["a"][0].double(), d["b"][0].double(), d["scales"][0].double()
    uref = x @ a.T
    umag = x.abs() @ a.abs().T
    assert float((uref[:, 0].abs().max() / uref[:, 1:].abs().max())) > 2.0 ** 22
    want, mag = s * (uref @ b.T), s.abs() * (umag @ b.abs().T)
    far = 0.0 if dt == BF else 2.0 ** -39 * s.abs() * uref.abs().amax(1)[:, None] * b.abs().sum(1)
    ref.close(out[:, 1::2], want[:, 1::2], ((ref.SPLIT + ref.acc(K + R + 2)) * mag + far)[:, 1::2], "out")


@pytest.mark.parametrize("dt", [HF, BF], ids=str)
def test_values_far_apart_in_one_adapter(ql, dt):
    """Tokens whose u (and v) are 2^25 times another token's, and outputs (inputs) that only the other has: its part
    of db (da) is held within 2^-16, or (fp16) 2^-39 of the adapter's largest."""
    M, K, N, R = 200, 128, 128, 16
    d = ref.make((dt, M, K, N, 1, R, "one"), seed=4)
    gen = torch.Generator(device="cuda").manual_seed(6)
    u = torch.randn(M, R, generator=gen, device="cuda")
    u[::2] *= 2.0 ** 25
    d["scales"][:] = 2.0 ** -12
    d["dy"][::2, 64:] = 0   # the columns from 64 on: only the odd tokens, of small u
    d["dy"][1::2, :64] = 0
    d["b"][:, 64:] = (d["b"][:, 64:].double() * 2.0 ** -12).to(dt)  # v of the odd tokens is 2^-12 of the others'
    d["x"][::2, 64:] = 0
    plan = ql.adapters_plan(d["ids"], 1)
    dx, da, db = ql.adapters_backward(d["dy"], d["a"], d["b"], d["scales"], plan, u, x=d["x"], want_dx=False)
    dy, b, s, x, ud = d["dy"].double(), d["b"][0].double(), d["scales"][0].double(), d["x"].double(), u.double()
    v, vm = s * (dy @ b), s * (dy.abs() @ b.abs())
    far = 0.0 if dt == BF else 2.0 ** -39
    close(db[0], s * (dy.T @ ud), (ref.SPLIT + ref.acc(M + 2)) * s * (dy.abs().T @ ud.abs())
          + far * s * ud.abs().max() * dy.abs().sum(0)[:, None], "db")
    close(da[0], v.T @ x, (ref.SPLIT + ref.acc(N + M + 2)) * (vm.T @ x.abs())
          + far * v.abs().max() * x.abs().sum(0)[None], "da")

"""Adapters and the weight gradient on whole numbers.  Every product and every sum stays below 2^24, the scales are
powers of two and the inner values fit the two halves (16 bits at least), so nothing is rounded before the result: it
has to be the 64-bit value's own rounding, at any length, split or order.  The inner values have more bits than one
half holds, and outputs are differences of them, so a lost half shows."""
import pytest
import torch

import adapter_ref as ref
from helpers import build_lib

pytestmark = pytest.mark.gpu

BF, HF, F32 = torch.bfloat16, torch.float16, torch.float32


@pytest.fixture(scope="module")
def ql():
    return build_lib()


CASES = [
    (BF, 1, 4096, 4096, 8, 16, "one"), (HF, 61, 4096, 11008, 32, 16, "random"), (BF, 16, 14336, 1024, 2, 128, "random"),
    (BF, 777, 11008, 4096, 12, 32, "random"), (HF, 300, 14336, 4096, 3, 24, "runs"), (BF, 1500, 4096, 14336, 4, 64, "blocks"),
    (HF, 2000, 4096, 8192, 2, 64, "blocks"), (BF, 4096, 4096, 4096, 1, 128, "one"), (BF, 257, 8200, 4104, 5, 12, "random"),
    (HF, 1000, 2048, 14336, 7, 80, "random"), (F32, 200, 4096, 2056, 3, 16, "runs"), (BF, 100, 4099, 1031, 2, 7, "random"),
]


def name(c):
    return f"{str(c[0])[6:]}_M{c[1]}_K{c[2]}_N{c[3]}_L{c[4]}_R{c[5]}_{c[6]}"


@pytest.mark.parametrize("case", CASES, ids=name)
def test_forward_and_backward(ql, case):
    dt, M, K, N, L, R, kind = case
    gen = torch.Generator(device="cuda").manual_seed(K + M)
    whole = lambda lo, hi, *s: torch.randint(lo, hi + 1, s, generator=gen, device="cuda", dtype=torch.int8)  # noqa: E731
    ids = ref.make_ids(kind, M, L, gen)
    q = whole(-2, 2, M, K)
    x, a, b, dy = q.to(dt), whole(-1, 1, L, R, K).to(dt), whole(-1, 1, L, N, R).to(dt), whole(-2, 2, M, N).to(dt)
    base, dx_base = (whole(-127, 127, M, n).to(dt) / 16 for n in (N, K))
    scales = torch.tensor([1, -0.5, 2, 0.25], device="cuda")[torch.arange(L, device="cuda") % 4].contiguous()
    plan = ql.adapters_plan(ids, L)
    u = torch.full((M, R), float("nan"), device="cuda")
    out = ql.adapters_forward(x, a, b, scales, plan, base=base, u=u)
    dx, da, db = ql.adapters_backward(dy, a, b, scales, plan, u, x=x, dx_base=dx_base)
    assert ql.device_status() == ql.QLIN_OK
    uref = torch.zeros(M, R, dtype=torch.float64, device="cuda")
    want, dref = base.double(), dx_base.double()
    for i in range(L):
        m = ref.rows_of(ids, i)
        ad, bd, xd, yd, s = a[i].double(), b[i].double(), x[m].double(), dy[m].double(), float(scales[i])
        uref[m] = xd @ ad.T
        want[m] += s * (uref[m] @ bd.T)
        v = s * (yd @ bd)
        assert not len(m) or (float(uref[m].abs().max()) < 2 ** 16 and float((v / s).abs().max()) < 2 ** 16)
        dref[m] += v @ ad
        assert torch.equal(da[i], (v.T @ xd).to(dt)), f"da[{i}]"
        assert torch.equal(db[i], (s * (yd.T @ uref[m])).to(dt)), f"db[{i}]"
    assert torch.equal(u.double(), uref) and torch.equal(out, want.to(dt)) and torch.equal(dx, dref.to(dt))
    for g in (64, 256):  # the input from codes of scale 1
        if K % g == 0:
            ones = torch.ones(K // g, M, device="cuda")
            got = ql.adapters_backward(dy, a, b, scales, plan, u, checkpoint=(q, ones, g), dx_base=dx_base)
            assert all(torch.equal(s, t) for s, t in zip(got, (dx, da, db)))


@pytest.mark.parametrize("dt,M,K,N,g", [(BF, 4096, 4096, 14336, 128), (HF, 1000, 11008, 4096, 256), (HF, 129, 4096, 4096, 64),
                                        (BF, 555, 4160, 9000, 64)], ids=str)
def test_weight_gradient(ql, dt, M, K, N, g):
    gen = torch.Generator(device="cuda").manual_seed(M)
    q = torch.randint(-127, 128, (M, K), generator=gen, device="cuda", dtype=torch.int8)
    dy = torch.randint(-4, 5, (M, N), generator=gen, device="cuda", dtype=torch.int8).to(dt)
    s = 2.0 ** torch.randint(-2, 1, (K // g, M), generator=gen, device="cuda").float()
    dw, db = ql.pergroup_wgrad(dy, q, s, g)
    assert ql.device_status() == ql.QLIN_OK and torch.equal(db, dy.double().sum(0).to(dt))
    xh, yd = ref.restored(q, s, g), dy.double()
    for c in range(0, K, 2048):
        assert torch.equal(dw[:, c:c + 2048], (yd.T @ xh[:, c:c + 2048]).to(dt)), c

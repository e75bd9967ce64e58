"""Large pools of adapters beside long layers: on the tensor cores, as smaller ones."""
import pytest
import torch

import adapter_ref as ref
from helpers import build_lib

pytestmark = pytest.mark.gpu

BF, HF = torch.bfloat16, torch.float16


@pytest.fixture(scope="module")
def ql():
    return build_lib()


def kernels(call):
    """Names of the kernels that a call launches."""
    call()
    torch.cuda.synchronize()
    with torch.profiler.profile(activities=[torch.profiler.ProfilerActivity.CUDA]) as prof:
        call()
        torch.cuda.synchronize()
    return " ".join(e.key for e in prof.key_averages())


# adapters x strips of 256 columns: 65536, 73728 and 131072 of dA's and dB's parts
@pytest.mark.parametrize("case", [(BF, 70, 8192, 8192, 1024, 4, "random"), (HF, 300, 4096, 14336, 1024, 8, "random"),
                                  (BF, 200, 4096, 61440, 512, 4, "runs")], ids=str)
def test_large_pools(ql, case):
    dt, M, K, N, L, R, _ = case
    d = ref.make(case)
    plan = ql.adapters_plan(d["ids"], L)
    u = torch.full((M, R), float("nan"), device="cuda")
    forward = lambda: ql.adapters_forward(d["x"], d["a"], d["b"], d["scales"], plan, base=d["base"], u=u)  # noqa: E731
    out = forward()
    ref.check_forward(d["x"], d["a"], d["b"], d["scales"], d["ids"], d["base"], out, u)
    back = lambda: ql.adapters_backward(d["dy"], d["a"], d["b"], d["scales"], plan, u, x=d["x"], dx_base=d["dx_base"])  # noqa: E731
    dx, da, db = back()
    assert ql.device_status() == ql.QLIN_OK
    used = [i for i in range(L) if bool((d["ids"] == i).any())]
    rest = torch.ones(L, dtype=torch.bool)
    rest[used] = False
    assert not da[rest].any() and not db[rest].any()  # written whole: zeros without tokens
    remap = torch.full((L + 2,), -1, dtype=torch.int32, device="cuda")
    remap[used] = torch.arange(len(used), dtype=torch.int32, device="cuda")
    ids = remap[torch.where((d["ids"] < 0) | (d["ids"] >= L), L, d["ids"]).long()]
    ref.check_backward(d["dy"], d["a"][used], d["b"][used], d["scales"][used], ids, u, d["x"].double(), d["dx_base"],
                       dx, da[used], db[used], False)
    names = kernels(forward)
    if "adapters_" not in names:
        pytest.skip("no trace of kernels can be had here")
    assert "adapters_decode_kernel" in names or "adapters_narrow_kernel" in names
    assert "adapters_sum_kernel" not in names  # of the general kernels
    names = kernels(back)
    assert "adapters_gram_kernel" in names and "adapters_sum_kernel" not in names

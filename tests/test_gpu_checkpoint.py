"""Activations kept in 8 bits: restoring them, and the weight gradient from them, against 64 bits."""
import pytest
import torch

import adapter_ref as ref
from helpers import build_lib

pytestmark = pytest.mark.gpu

BF, HF, F32 = torch.bfloat16, torch.float16, torch.float32


@pytest.fixture(scope="module")
def ql():
    return build_lib()


def rn(seed, *shape):
    return torch.randn(*shape, generator=torch.Generator(device="cuda").manual_seed(seed), device="cuda")


@pytest.mark.parametrize("dt", [BF, HF, F32], ids=str)
@pytest.mark.parametrize("M,K,g", [(1, 64, 64), (3, 256, 256), (65, 4096, 128), (1000, 448, 64), (7, 14336, 256)])
def test_save_and_restore(ql, dt, M, K, g):
    x = rn(M, M, K) * torch.exp(3 * rn(K, M, 1))
    x[0, :g] = 0
    x = x.to(dt)
    q, s = ql.quantize_int8_groups(x, g)
    back = ql.dequantize_int8_groups(q, s, g, dt)
    want = (q.float().reshape(M, -1, g) * s.t()[:, :, None]).reshape(M, K).to(dt)
    # one fp32 product, one rounding; an input beyond fp16's range is infinite there, so its group's scale is, and
    # its products are not numbers on either side
    assert torch.equal(back.nan_to_num(1e4), want.nan_to_num(1e4))
    top = x.double().reshape(M, -1, g).abs().amax(2)
    off = (back.double() - x.double()).reshape(M, -1, g).abs()
    fine = top.isfinite()
    assert bool(fine.float().mean() > 0.99) and bool(back.reshape(M, -1, g)[fine].isfinite().all())
    # half a code's step (the code itself rounds a quotient with 24 bits), then half a step of the type
    assert bool((off <= (0.5 / 127 + 2.0 ** -16 + ref.half(dt)) * top[:, :, None] + ref.TINY[dt])[fine].all())


def test_restore_far_into_a_long_tensor(ql):
    """More than 2^31 values: offsets need 64 bits."""
    M, K, g = (1 << 31) // 8192 + 3, 8192, 256
    q = torch.empty((M, K), dtype=torch.int8, device="cuda")
    q[:1000] = torch.randint(-127, 128, (1000, K), device="cuda", dtype=torch.int8)
    q[-1000:] = torch.randint(-127, 128, (1000, K), device="cuda", dtype=torch.int8)
    s = torch.rand(K // g, M, device="cuda")
    back = ql.dequantize_int8_groups(q, s, g, HF)
    for part in (slice(0, 1000), slice(M - 1000, M)):
        want = (q[part].float().reshape(1000, -1, g) * s[:, part].t()[:, :, None]).reshape(1000, K).to(HF)
        assert torch.equal(back[part], want)


WGRAD = [(BF, 1, 64, 64, 64), (HF, 3, 64, 8, 64), (BF, 64, 256, 128, 256), (HF, 129, 512, 264, 64),
         (BF, 63, 128, 136, 128), (BF, 65, 320, 1000, 64), (HF, 257, 768, 520, 256), (BF, 1000, 1024, 904, 256),
         (HF, 512, 4096, 512, 128), (BF, 2048, 512, 2056, 64), (BF, 96, 14336, 72, 128), (HF, 4100, 256, 264, 128),
         (BF, 128, 4096, 4096, 64)]


@pytest.mark.parametrize("case", WGRAD, ids=lambda c: f"{str(c[0])[6:]}_M{c[1]}_K{c[2]}_N{c[3]}_g{c[4]}")
def test_wgrad(ql, case):
    dt, M, K, N, g = case
    x = (rn(1, M, K) * (1 + 30 * (rn(2, K) > 2))).to(dt)
    dy = (rn(3, M, N) * torch.exp(rn(4, M, 1)) * 0.05).to(dt)
    q, s = ql.quantize_int8_groups(x, g)
    dw, db = ql.pergroup_wgrad(dy, q, s, g)
    assert ql.device_status() == ql.QLIN_OK
    xh, yd = ref.restored(q, s, g), dy.double()
    ref.close(dw, yd.T @ xh, (ref.half(dt) + ref.acc(M)) * (yd.abs().T @ xh.abs()), "dw")
    ref.close(db, yd.sum(0), ref.acc(M) * yd.abs().sum(0), "db")
    again, none = ql.pergroup_wgrad(dy, q, s, g, bias=False, dw=torch.full_like(dw, float("nan")))
    assert none is None and torch.equal(again, dw)


def test_wgrad_of_tokens_that_are_not_finite(ql):
    """A NaN in dy reaches its own row of dw, one in the scales its own columns."""
    M, K, N, g = 100, 256, 128, 64
    x, dy = rn(1, M, K).to(BF), rn(2, M, N).to(BF)
    q, s = ql.quantize_int8_groups(x, g)
    dy[7, 5], s[1, 3] = float("nan"), float("nan")
    dw, db = ql.pergroup_wgrad(dy, q, s, g)
    assert dw[5].isnan().all() and dw[:, 64:128].isnan().all() and db[5].isnan()
    fine = torch.ones(N, K, dtype=torch.bool, device="cuda")
    fine[5], fine[:, 64:128] = False, False
    assert dw[fine].isfinite().all() and int(db.isnan().sum()) == 1


def test_wgrad_in_a_graph_and_on_a_stream(ql):
    M, K, N, g = 300, 512, 520, 64
    x, dy = rn(1, M, K).to(BF), rn(2, M, N).to(BF)
    q, s = ql.quantize_int8_groups(x, g)
    dw, _ = ql.pergroup_wgrad(dy, q, s, g)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        other, _ = ql.pergroup_wgrad(dy, q, s, g)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    assert torch.equal(other, dw)
    with torch.cuda.graph(graph):
        held, bias = ql.pergroup_wgrad(dy, q, s, g)
    dy.mul_(-2)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(held, dw * -2)
    ref.close(bias, dy.double().sum(0), ref.acc(M) * dy.double().abs().sum(0), "db")


def test_python_refusals(ql):
    q = torch.zeros(4, 64, dtype=torch.int8, device="cuda")
    s = torch.ones(1, 4, device="cuda")
    dy = torch.zeros(4, 64, dtype=BF, device="cuda")
    for bad in (lambda: ql.dequantize_int8_groups(q, s.t(), 64), lambda: ql.dequantize_int8_groups(q, s, 32),
                lambda: ql.pergroup_wgrad(dy[:2], q, s, 64), lambda: ql.pergroup_wgrad(dy, q, s[:, :2], 64),
                lambda: ql.dequantize_int8_groups(q, s.cpu(), 64)):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(TypeError):
        ql.dequantize_int8_groups(q.float(), s, 64)
    with pytest.raises(ql.QlinError) as e:
        ql.pergroup_wgrad(dy.float(), q, s, 64)
    assert e.value.status == ql.QLIN_ERR_UNSUPPORTED

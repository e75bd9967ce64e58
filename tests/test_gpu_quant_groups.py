"""The per-group int8 quantiser over row lengths and sizes: every way a warp's lanes fall on rows and columns, one
and two steps of rows a block, and more blocks than a grid holds down."""
import numpy as np
import pytest
import torch

from helpers import build_lib

pytestmark = pytest.mark.gpu

BF, HF, F32 = torch.bfloat16, torch.float16, torch.float32


@pytest.fixture(scope="module")
def ql():
    return build_lib()


def values(N, K, dt, seed):
    """Rows of different size, a group of zeros, values half-way between two codes (x = (k + 1/2) s exactly)."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(N, K, generator=gen, device="cuda") * torch.exp(2 * torch.randn(N, 1, generator=gen, device="cuda"))
    x[N // 2, :64] = 0
    x[0] = torch.arange(K, device="cuda") % 127 + 0.5
    x[0, ::64] = 127
    x[-1] = x[0] * 2 ** -7
    return x.to(dt)


def plain(x, g):
    """fp32 division by 127 and by the scale, each rounded once; half to even; |code| <= 127 by the scale's choice."""
    groups = x.float().reshape(x.shape[0], -1, g)
    top = groups.abs().amax(2)
    scale = top / torch.full_like(top, 127)
    scale = torch.where(scale == 0, 1.0, scale)
    codes = (groups / scale[:, :, None]).round().clamp(-128, 127)
    codes = torch.where(codes.isnan(), -128.0, codes)  # an infinity over its group's scale, as the oracle has it
    return codes.to(torch.int8).reshape(x.shape), scale.t().contiguous()


# K of every power of two that divides it: 64, 128, 256, 512 columns a warp
@pytest.mark.parametrize("dt", [BF, HF, F32], ids=str)
@pytest.mark.parametrize("N,K,g", [(1, 64, 64), (3, 64, 64), (33, 64, 64), (100, 128, 128), (37, 192, 64),
                                   (15, 256, 256), (50, 384, 128), (31, 448, 64), (2, 576, 64), (19, 640, 128),
                                   (5, 768, 256), (77, 1024, 64), (9, 1280, 256), (130, 4160, 64), (1, 14336, 256)])
def test_codes_and_scales_are_the_oracles(ql, orc, dt, N, K, g):
    x = values(N, K, dt, N + K)
    q, s = ql.quantize_int8_groups(x, g)
    q_ref, s_ref = orc.quantize_int8_groups(x.float().cpu().numpy(), g)
    assert np.array_equal(q.cpu().numpy(), q_ref) and np.array_equal(s.cpu().numpy(), s_ref)


# two steps of rows a block (more than 128 blocks an SM), rows past the last whole step; above 65535 blocks down
@pytest.mark.parametrize("dt", [BF, HF, F32], ids=str)
@pytest.mark.parametrize("N,K,g", [(38001, 512, 128), (5001, 4096, 256), (303201, 64, 64), (80003, 128, 64),
                                   (2200017, 64, 64), (140001, 512, 64), (14336, 4096, 64)])
def test_large(ql, dt, N, K, g):
    x = values(N, K, dt, K)
    q, s = ql.quantize_int8_groups(x, g)
    q_ref, s_ref = plain(x, g)
    assert torch.equal(q, q_ref) and torch.equal(s, s_ref)


def test_short_rows_cost_no_more_than_long_ones():
    """64 million values as rows of 64 and of 4096: the same bytes, about the same time (a warp of idle lanes took 5x)."""
    ql = build_lib()

    def ms(N, K):
        x = torch.randn(N, K, device="cuda", dtype=BF)
        call = lambda: ql.quantize_int8_groups(x, 64)  # noqa: E731
        [call() for _ in range(5)]
        ts = []
        for _ in range(9):
            a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
            a.record()
            [call() for _ in range(10)]
            b.record()
            b.synchronize()
            ts.append(a.elapsed_time(b))
        return sorted(ts)[4]

    assert ms(1000000, 64) < 2 * ms(15625, 4096)

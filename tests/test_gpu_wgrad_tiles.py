"""The weight gradient's launches of many tiles: CTA pairs that take several whole tiles, halves of the last round's,
an odd number of stages a tile, column sums handed over in every tile."""
import pytest
import torch

import adapter_ref as ref
from helpers import build_lib

pytestmark = pytest.mark.gpu

BF, HF = torch.bfloat16, torch.float16


@pytest.fixture(scope="module")
def ql():
    return build_lib()


# tiles of 512 outputs by 256 inputs on 74 pairs, stages of 64 tokens
CASES = [
    (BF, 545, 4096, 4616, 64),     # 10 x 16 = 160 tiles: 148 whole, the last 12 cut; 9 stages
    (HF, 577, 2560, 4616, 128),    # 100: 74 whole, 26 cut; 10 stages, the last of one token
    (BF, 640, 1024, 15800, 256),   # 31 x 4 = 124: the last round of 50 whole
    (HF, 1100, 512, 20000, 64),    # 40 x 2 = 80: 74 whole, 6 cut; 18 stages, the last of 12 tokens
    (BF, 600, 256, 102400, 128),   # 200 x 1: every tile is in the first column, so each has column sums
    (HF, 2049, 4160, 2056, 64),    # 5 x 17 = 85, the last column of tiles 64 inputs wide; 33 stages
    (BF, 4096, 2048, 5000, 128),   # 10 x 8 = 80; 64 stages
    # one CTA a tile of 128 by 256, several each
    (BF, 500, 4096, 4096, 128), (HF, 129, 2112, 5008, 64), (BF, 1, 1024, 9000, 256), (HF, 64, 14336, 1032, 256),
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: f"{str(c[0])[6:]}_M{c[1]}_K{c[2]}_N{c[3]}_g{c[4]}")
def test_many_tiles(ql, case):
    dt, M, K, N, g = case
    gen = torch.Generator(device="cuda").manual_seed(M + K)
    rn = lambda *s: torch.randn(*s, generator=gen, device="cuda")  # noqa: E731
    x = (rn(M, K) * (1 + 30 * (rn(K) > 2))).to(dt)
    dy = (rn(M, N) * torch.exp(rn(M, 1)) * 0.05).to(dt)
    q, s = ql.quantize_int8_groups(x, g)
    dw, db = torch.full((N, K), float("nan"), device="cuda", dtype=dt), None
    dw, db = ql.pergroup_wgrad(dy, q, s, g, dw=dw)
    assert ql.device_status() == ql.QLIN_OK
    xh, yd = ref.restored(q, s, g), dy.double()
    ref.close(db, yd.sum(0), ref.acc(M) * yd.abs().sum(0), "db")
    for c in range(0, K, 512):  # the bound takes as much memory as the product
        p = slice(c, min(c + 512, K))
        ref.close(dw[:, p], yd.T @ xh[:, p], (ref.half(dt) + ref.acc(M)) * (yd.abs().T @ xh[:, p].abs()), f"dw from {c}")
    again, b2 = ql.pergroup_wgrad(dy, q, s, g)
    assert torch.equal(again, dw) and torch.equal(b2, db)


@pytest.mark.parametrize("N,K", [(8, 64), (264, 256)])
def test_the_longest_batch(ql, N, K):
    """2^24 tokens (one CTA a tile, and a pair), codes and gradients of -1, 0 and 1: the sums are whole numbers below
    2^24, exact in fp32, whatever their order."""
    M, g = 1 << 24, 64
    gen = torch.Generator(device="cuda").manual_seed(1)
    q = torch.randint(-1, 2, (M, K), generator=gen, device="cuda", dtype=torch.int8)
    dy = torch.randint(-1, 2, (M, N), generator=gen, device="cuda", dtype=torch.int8).to(BF)
    s = torch.ones(K // g, M, device="cuda")
    dw, db = ql.pergroup_wgrad(dy, q, s, g)
    assert ql.device_status() == ql.QLIN_OK
    want, sums = torch.zeros(N, K, dtype=torch.float64, device="cuda"), dy.sum(0, dtype=torch.float64)
    for m in range(0, M, 1 << 20):
        want += dy[m:m + (1 << 20)].double().T @ q[m:m + (1 << 20)].double()
    assert torch.equal(dw, want.to(BF)) and torch.equal(db, sums.to(BF))

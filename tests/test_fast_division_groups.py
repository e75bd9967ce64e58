"""The per-group int8 quantiser's code of x at scale s (k_quant.cu quantize_int8_groups_vec_kernel): r = 1/s rounded
once, t = fma(x, r, 1.5 2^23), whose low byte is the product rounded half to even, and the IEEE division where the
product lies 0.49997 or more from t's integer.  Emulated here and checked against rint of the float32 quotient."""
import os

import numpy as np
import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SRC = os.path.join(ROOT, "bit_quantized_linear_qmm_b200", "csrc", "k_quant.cu")
f32 = np.float32


def code(x, s):
    """(code, whether the product gave it).  A float32 product has 48 bits, so float64 holds it whole; an fma with
    1.5 2^23, where floats are whole numbers, is its rint; the fma that measures the distance rounds it once."""
    m = x.astype(np.float64) * np.float64(f32(1) / f32(s))
    k = np.rint(m)
    near = ~(np.abs((m - k).astype(f32)) < f32(0.49997))
    exact = np.rint((x / f32(s)).astype(f32))
    # the byte: |k| <= 127 wherever it is used
    assert np.all(np.abs(k[~near]) <= 127)
    return np.where(near, exact, k), near


def check(x, s):
    got, near = code(x, s)
    assert np.array_equal(got, np.rint((x / f32(s)).astype(f32)))
    return near


def scale_of(amax):
    return f32(amax) / f32(127)


def test_constants_match_the_kernel():
    src = open(SRC).read()
    assert "t = __fmaf_rn(x, r, 12582912.f);" in src
    assert "return !(fabsf(__fmaf_rn(x, r, __fsub_rn(12582912.f, t))) < 0.49997f); };" in src
    assert "rcp_ok(sc) ? __frcp_rn(sc) : __uint_as_float(0x7fc00000u)" in src
    assert "return s >= 1.17549435e-38f && s <= 8.0e37f;" in src


def test_next_to_every_half_integer():
    """x a few floats from (k + 1/2) s, s of every significand pattern and normal size."""
    rng = np.random.default_rng(1)
    seen = 0
    for _ in range(1500):
        amax = f32(2.0 ** rng.uniform(-110, 125))
        s = scale_of(amax)
        half = ((np.arange(-127, 127) + 0.5) * np.float64(s)).astype(f32)
        x = half.view(np.int32)[:, None] + np.arange(-8, 9, dtype=np.int32)
        x = x.astype(np.int32).view(f32).ravel()
        x = x[np.abs(x) <= amax]
        seen += int(check(x, s).sum())
    assert seen > 100000  # the division's branch is what these reach


def test_random_values():
    rng = np.random.default_rng(2)
    divided = total = 0
    for _ in range(300):
        x = (rng.standard_normal(8192) * 2.0 ** rng.uniform(-100, 100)).astype(f32)
        near = check(x, scale_of(np.abs(x).max()))
        divided, total = divided + near.sum(), total + near.size
    assert divided < 2e-4 * total  # 6e-5 of evenly spread fractions


@pytest.mark.parametrize("kind", ["bf16", "f16"])
def test_every_16_bit_value(kind):
    """All values of a 16-bit type up to amax, for every significand of amax at several exponents."""
    bits = np.arange(1 << 15, dtype=np.uint32)
    v = (bits << 16).astype(np.uint32).view(f32) if kind == "bf16" else bits.astype(np.uint16).view(np.float16).astype(f32)
    v = np.sort(v[np.isfinite(v)])
    tops = [t for e in ((-60, 0, 1, 90) if kind == "bf16" else (-10, 0, 1, 14))
            for t in np.unique((2.0 ** e * (1 + np.arange(0, 1, 1 / 128 if kind == "bf16" else 1 / 64))))]
    for top in tops:
        x = v[v <= f32(top)]
        x = x[x >= f32(top) * f32(2.0 ** -9)]  # smaller ones are code 0
        check(np.concatenate([x, -x]), scale_of(top))

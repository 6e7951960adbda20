"""Facts about the packed caches' numbers that the kernels rely on, exhaustively, on the CPU."""

import numpy as np

import oracle.kv4 as K4
import oracle.kv8 as K8


def _bf16(x):
    """The nearest value of 8 significant bits, ties to even, of float64 values (no subnormals among them)."""
    m, e = np.frexp(x)
    return np.ldexp(np.rint(m * 256.0), e - 8)


def test_8_bit_values_rounded_to_fp32_and_then_to_bf16_are_rounded_once():
    """Every significand that the largest element of a bf16 block may have, every code, small and large exponents."""
    codes = K8.e4m3_values()[1:127]
    for e in (-95, -20, 0, 1, 7, 100, 119):
        amax = ((128 + np.arange(128)) / 128 * 2.0 ** e).astype(np.float32)
        scale = amax / K8.E4M3_MAX
        exact = scale.astype(np.float64)[:, None] * codes
        product = scale[:, None] * codes.astype(np.float32)
        assert (product.astype(np.float64) != exact).any()
        assert np.array_equal(_bf16(product.astype(np.float64)), _bf16(exact))


def test_4_bit_values_are_exact_in_fp16_and_in_bf16():
    """code * scale fits fp16, and times any power of two of the format bf16."""
    v = np.unique(K4.E2M1[:, None] * K8.e4m3_values()[:127])
    assert np.array_equal(v.astype(np.float16).astype(np.float64), v)
    for e in (K4.EXP_MIN, 0, K4.EXP_MAX):
        assert np.array_equal(_bf16(np.ldexp(v, e)), np.ldexp(v, e)) and np.abs(np.ldexp(v, e)).max() < 2.0 ** 128

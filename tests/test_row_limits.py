"""The largest number of rows of the grouped calls (host only): up to the end of
a last tile of 256 rows they are counted in 32 bits in the kernels, so that more
than 2^31 - 256 are refused; with fewer, the next thing that is wrong is (here a
null pointer)."""
import ctypes

import pytest

from fp8_block_scaled_bias_amd import _lib as L

P = ctypes.c_void_p(4096)   # never dereferenced
CALLS = {
    "grouped_fp8_gemm": lambda f, M: f(None, P, P, 8, P, P, P, 2, M, 128, 128, P, None),
    "grouped_fp8_gemm_dgrad": lambda f, M: f(None, P, P, P, P, 2, M, 128, 128, P, None),
    "grouped_fp8_gemm_swiglu": lambda f, M: f(None, P, P, 8, P, P, P, 2, M, 128, 128, P, P, None),
    "grouped_fp8_gemm_swiglu_keep": lambda f, M: f(None, P, P, 8, P, P, P, 2, M, 128, 128, P, P, P, None),
    "fp8_quant_128x1_grouped": lambda f, M: f(None, 128, P, 8, P, 2, M, 128, P, P, M // 128 + 3, None),
    "grouped_fp8_wgrad": lambda f, M: f(None, P, P, P, M // 128 + 3, P, 2, M, 128, 128, P, None),
    "swiglu_backward_grouped": lambda f, M: f(None, P, P, 2, M, 128, P, P, P, P, M // 128 + 3, P, P, P, P, None),
    "grouped_int8_gemm": lambda f, M: f(None, P, P, 8, P, P, P, 2, M, 64, 64, P, None),
    "grouped_int8_gemm_swiglu": lambda f, M: f(None, P, P, 8, P, P, P, 2, M, 64, 64, P, None),
    "grouped_bf16_gemm": lambda f, M: f(None, P, 8, P, P, 2, M, 64, 64, P, None),
    "grouped_bf16_gemm_glu": lambda f, M: f(None, P, 8, P, P, 2, M, 64, 64, 0, P, None, None),
    "grouped_bf16_gemm_dgrad": lambda f, M: f(None, P, P, 2, M, 64, 64, P, None),
    "grouped_bf16_gemm_dgrad_glu": lambda f, M: f(None, P, P, P, 2, M, 64, 64, 0, P, None),
    "grouped_bf16_wgrad": lambda f, M: f(None, P, P, 8, P, 2, M, 64, 64, P, None),
}


@pytest.mark.parametrize("name", CALLS)
def test_rows(name):
    call = lambda M: CALLS[name](getattr(L.lib(), name), M)
    assert call((1 << 31) - 255) == L.MOE_ERR_UNSUPPORTED and "M_total" in L.last_error()
    assert call((1 << 31) - 1) == L.MOE_ERR_UNSUPPORTED
    assert call((1 << 31) - 256) == L.MOE_ERR_INVALID and "null" in L.last_error()


def test_every_call_with_groups_is_here():
    assert set(CALLS) == {n for n in L.SIGNATURES if n.startswith("grouped_") or n.endswith("_grouped")}

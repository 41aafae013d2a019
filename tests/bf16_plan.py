"""The library's choice of a kernel for a grouped bf16 product, asked from the
header that the launch itself uses (compiled here for the host)."""
import ctypes
import functools
import os
import subprocess
import tempfile

from conftest import ROOT

MODES = ["gemm", "glu", "dgrad", "dgrad_glu", "wgrad"]
PLANS = ["wide", "mid", "split16x64", "split16x16", "split64x64", "split64x32", "split64x16"]

SOURCE = r"""
#include "bf16_plan.h"
extern "C" int choice(int mode, int gather, int64_t A_rows, int64_t G, int64_t M, int64_t N, int64_t K,
                      int64_t cus) {
  return moe::bf16::plan(moe::bf16::Shape{(moe::bf16::Mode)mode, gather != 0, A_rows, G, M, N, K}, cus);
}
"""


@functools.lru_cache(None)
def _choice():
    with tempfile.TemporaryDirectory() as d:
        src, lib = os.path.join(d, "plan.cpp"), os.path.join(d, "plan.so")
        with open(src, "w") as f:
            f.write(SOURCE)
        subprocess.run(["g++", "-std=c++17", "-shared", "-fPIC", "-I",
                        os.path.join(ROOT, "fp8_block_scaled_bias_amd", "csrc"), src, "-o", lib], check=True)
        fn = ctypes.CDLL(lib).choice
    fn.argtypes = [ctypes.c_int] * 2 + [ctypes.c_int64] * 6
    return fn


def plan(mode, G, M_total, N, K, gather=False, a_rows=None, cus=256):
    """N, K: of the weights (glu: N = I)."""
    a_rows = M_total if a_rows is None else a_rows
    return PLANS[_choice()(MODES.index(mode), int(gather), a_rows, G, M_total, N, K, cus)]

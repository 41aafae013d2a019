"""The library's choice of a kernel for a grouped int8 product, asked from the
header that the launch itself uses (compiled here for the host)."""
import ctypes
import functools
import os
import subprocess
import tempfile

from conftest import ROOT

PLANS = ["wide", "mid", "flow", "split16x64", "split16x16", "split64x64", "split64x32", "split64x16"]

SOURCE = r"""
#include "int8_plan.h"
extern "C" int choice(int swiglu, int gather, int64_t A_rows, int64_t G, int64_t M, int64_t N, int64_t K,
                      int64_t cus) {
  return moe::int8::plan(moe::int8::Shape{swiglu != 0, gather != 0, A_rows, G, M, N, K}, cus);
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


def plan(swiglu, gather, a_rows, G, M_total, N, K, cus=256):
    """N: columns of the output."""
    return PLANS[_choice()(int(swiglu), int(gather), a_rows, G, M_total, N, K, cus)]

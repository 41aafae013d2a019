"""The bf16 grouped products on shapes for which the rule takes each kernel,
checked against FP64."""
import numpy as np
import pytest

import fp8_block_scaled_bias_amd as M
from bf16_cases import Case
from gpu_common import log

pytestmark = pytest.mark.gpu

# many groups: 16 of them uneven, empty ones at both ends and inside, whole
# tiles and one over and short; one, two and more K blocks
UNEVEN = [0, 300, 1, 0, 256, 64, 65, 0, 17, 200, 5, 129, 63, 2, 97, 0]
EVEN = [24] * 16


@pytest.mark.parametrize("gather", [False, True])
@pytest.mark.parametrize("K", [8, 64, 72, 128, 200, 448])
def test_wide_gemm(K, gather):
    log(f"[bf16 plans] wide gemm K={K} gather={gather}")
    Case(UNEVEN, 4104, K, 21, gather).gemm("wide gemm")


@pytest.mark.parametrize("act", [M.ACT_SILU, M.ACT_GELU])
@pytest.mark.parametrize("K,keep", [(64, True), (136, False), (520, True)])
def test_wide_glu(K, keep, act):
    log(f"[bf16 plans] wide glu K={K} keep={keep}")
    Case(UNEVEN, 2056, K, 22, act == M.ACT_SILU).glu(act, keep, "wide glu")
    Case(EVEN, 2056, K, 22, act == M.ACT_GELU).glu(act, keep, "wide glu even")


@pytest.mark.parametrize("N", [8, 72, 256, 328])
def test_wide_dgrad(N):
    log(f"[bf16 plans] wide dgrad N={N}")
    Case(UNEVEN, N, 4104, 23).dgrad("wide dgrad")
    Case(UNEVEN, N, 4104, 24).dgrad_glu(M.ACT_GELU, "wide dgrad glu")


@pytest.mark.parametrize("gather", [False, True])
@pytest.mark.parametrize("N,K", [(1032, 1032), (264, 2304), (2048, 520)])
def test_wide_wgrad(N, K, gather):
    log(f"[bf16 plans] wide wgrad N={N} K={K} gather={gather}")
    Case(UNEVEN, N, K, 25, gather).wgrad("wide wgrad")


def test_wide_wgrad_of_one_long_group():
    Case([1, 2, 1500, 0], 2056, 2048, 26, True).wgrad("long group")

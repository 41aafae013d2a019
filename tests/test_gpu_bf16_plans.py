"""The bf16 grouped products on shapes for which the rule takes each kernel,
checked against FP64."""
import numpy as np
import pytest
import torch

import fp8_block_scaled_bias_amd as M
from bf16_cases import Case, check, offsets, up, values
from bf16_plan import plan
from gpu_common import bf16_values_host, dev, log
from oracle import bf16 as OB

pytestmark = pytest.mark.gpu

# many groups: 16 of them uneven, empty ones at both ends and inside, whole
# tiles and one over and short; one, two and more K blocks
UNEVEN = [0, 300, 1, 0, 256, 64, 65, 0, 17, 200, 5, 129, 63, 2, 97, 0]
EVEN = [160] * 16


def taken(want, mode, case):
    assert plan(mode, case.G, case.M, case.N, case.K, case.index is not None, case.a_rows) == want
    return case


@pytest.mark.parametrize("gather", [False, True])
@pytest.mark.parametrize("K", [8, 64, 72, 128, 200, 448])
def test_wide_gemm(K, gather):
    log(f"[bf16 plans] wide gemm K={K} gather={gather}")
    taken("wide", "gemm", Case(UNEVEN * 2, 4360, K, 21, gather, behind=2000)).gemm("wide gemm")


@pytest.mark.parametrize("act", [M.ACT_SILU, M.ACT_GELU])
@pytest.mark.parametrize("K,keep", [(64, True), (136, False), (520, True)])
def test_wide_glu(K, keep, act):
    log(f"[bf16 plans] wide glu K={K} keep={keep}")
    taken("wide", "glu", Case(UNEVEN * 2, 2184, K, 22, act == M.ACT_SILU, behind=2000)).glu(act, keep, "wide glu")
    taken("wide", "glu", Case(EVEN, 2056, K, 22, act == M.ACT_GELU)).glu(act, keep, "wide glu even")


@pytest.mark.parametrize("N", [8, 72, 256, 328])
def test_wide_dgrad(N):
    log(f"[bf16 plans] wide dgrad N={N}")
    taken("wide", "dgrad", Case(UNEVEN * 2, N, 4360, 23, behind=2000)).dgrad("wide dgrad")
    taken("wide", "dgrad_glu", Case(UNEVEN * 2, N, 4360, 24, behind=2000)).dgrad_glu(M.ACT_GELU, "wide dgrad glu")


@pytest.mark.parametrize("gather", [False, True])
@pytest.mark.parametrize("N,K", [(1032, 1032), (392, 2304), (2048, 520)])
def test_wide_wgrad(N, K, gather):
    log(f"[bf16 plans] wide wgrad N={N} K={K} gather={gather}")
    taken("wide", "wgrad", Case(UNEVEN, N, K, 25, gather)).wgrad("wide wgrad")


def test_wide_wgrad_of_one_long_group():
    taken("wide", "wgrad", Case([1, 2, 1500, 0], 2056, 2048, 26, True)).wgrad("long group")


@pytest.mark.parametrize("gather", [False, True])
@pytest.mark.parametrize("K", [8, 56, 64, 264, 1032])
@pytest.mark.parametrize("name,counts,N,glu", [
    ("split16x64", [3, 0, 16, 1], 4168, False), ("split16x64", [9, 1, 0, 16], 2088, True),
    ("split16x16", [1], 72, False), ("split16x16", [11], 136, True), ("split16x16", [0, 5, 40, 0], 264, False),
    ("split16x16", [2, 0, 33], 72, True),
    ("split64x64", [63], 16384, False), ("split64x64", [20, 100], 4096, True),
    ("split64x32", [65], 4360, False), ("split64x16", [17], 136, True), ("split64x16", [50, 0, 130], 200, False),
])
def test_register_kernels(name, counts, N, glu, K, gather):
    case = taken(name, "glu" if glu else "gemm", Case(counts, N, K, 27, gather, behind=1))
    log(f"[bf16 plans] {name} {counts} N={N} K={K} glu={glu} gather={gather}")
    if glu:
        case.glu(M.ACT_GELU if gather else M.ACT_SILU, keep=K != 64, label=name)
    else:
        case.gemm(name)


@pytest.mark.parametrize("gather", [False, True])
@pytest.mark.parametrize("K", [8, 64, 200, 328])
def test_mid_kernel(K, gather):
    log(f"[bf16 plans] mid K={K} gather={gather}")
    taken("mid", "gemm", Case(UNEVEN, 1032, K, 28, gather)).gemm("mid gemm")
    taken("mid", "glu", Case(UNEVEN, 520, K, 28, gather)).glu(M.ACT_SILU, True, "mid glu")
    taken("mid", "dgrad", Case(UNEVEN, K, 1032, 28)).dgrad("mid dgrad")
    taken("mid", "dgrad_glu", Case(UNEVEN, K, 520, 28)).dgrad_glu(M.ACT_SILU, "mid dgrad glu")
    taken("mid", "wgrad", Case(UNEVEN, K, 392, 28, gather)).wgrad("mid wgrad")


def test_one_group_holds_most_rows():
    """A small average and one long group, in the kernel of few rows and in tiles."""
    taken("split16x64", "gemm", Case([0, 0, 40, 0, 0], 4104, 136, 29)).gemm("one of five")
    taken("mid", "gemm", Case([1] * 7 + [250] + [0] * 60, 1096, 136, 29)).gemm("one of many")


def test_offsets_past_32_bits():
    """Gathered rows more than 4 GiB into A: their kernels take 64-bit places."""
    k = 4096
    rows = (1 << 31) // k + 40
    rng = np.random.default_rng(30)
    a = torch.zeros((rows, k), dtype=torch.bfloat16, device="cuda")
    last = values(rng, (32, k))
    a[rows - 32:] = up(last)
    N = 1544
    b = values(rng, (1, N, k), k ** -0.5)
    for want, R in (("mid", 700), ("split64x16", 200), ("split16x16", 7)):
        idx = rows - 32 + rng.integers(0, 32, R)
        out = torch.empty((R, N), dtype=torch.bfloat16, device="cuda")
        assert plan("gemm", 1, R, N, k, True, rows) == want
        M.grouped_bf16_gemm(a, dev(idx.astype(np.int32)), up(b), dev(offsets([R])), 1, R, N, k, out)
        check(bf16_values_host(out), *OB.products(last[idx - rows + 32], b, offsets([R])), "past 32 bits")
    # the weight gradient of the same rows
    R = 300
    idx = rows - 32 + rng.integers(0, 32, R)
    dy = values(rng, (R, 520))
    dw = torch.empty((1, 520, k), device="cuda")
    assert plan("wgrad", 1, R, 520, k, True, rows) == "mid"
    M.grouped_bf16_wgrad(up(dy), a, dev(idx.astype(np.int32)), dev(offsets([R])), 1, R, 520, k, dw)
    ref, err = OB.wgrad(dy, last[idx - rows + 32], offsets([R]))
    assert (np.abs(dw.cpu().numpy() - ref) <= err + 2.0 ** -24 * np.abs(ref)).all()

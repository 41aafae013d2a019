"""Every kernel of the grouped int8 products, plain and with SwiGLU, gathered and
not, at sizes that end inside its tiles; each test asks which kernel its sizes
take, so that a moved border shows."""
import numpy as np
import pytest
import torch

import fp8_block_scaled_bias_amd as M
from gpu_common import bf16_values_host, host, log
from int8_plan import plan
from oracle import int8 as OI
from test_gpu_int8 import case, check, check_swiglu, run

pytestmark = pytest.mark.gpu

# rows of the groups: empty ones, tiles that are full, one row over, nearly empty
RAGGED = [0, 257, 1, 256, 130, 0, 0, 513, 64, 255, 17, 128, 129, 300, 2, 33] * 4
SOME = [0, 257, 1, 256, 130, 63, 200, 129]
FEW = [1, 0, 3, 16, 17, 2, 0, 4, 1, 5, 0, 7, 2, 3, 1, 2] * 8    # 4 a group

# kernel -> (rows of the groups, N plain, I with SwiGLU or None, every K)
CASES = {
    "wide": (RAGGED, 1032, 520, (144, 240, 256, 272, 400, 1040)),
    "mid": (SOME, 1032, 520, (16, 112, 128, 144, 272, 1040)),
    "flow": (FEW, 1032, 520, (16, 128, 144, 400, 1040)),
    "split16x64": (FEW[:40], 1032, 520, (16, 128, 144, 400, 2064)),
    "split16x16": ([9, 0, 2], 1032, 520, (16, 128, 144, 400, 2064)),
    "split64x64": ([100, 0, 1, 150], 4088, 2040, (16, 128, 144, 400, 2064)),
    "split64x32": ([30], 8200, None, (16, 128, 144, 400, 2064)),
    "split64x16": ([64, 5, 0, 61], 1032, 520, (16, 128, 144, 400, 2064)),
}


def cus():
    return torch.cuda.get_device_properties(0).multi_processor_count


@pytest.mark.parametrize("gather", [False, True], ids=["rows", "gathered"])
@pytest.mark.parametrize("kernel,K", [(name, K) for name, c in CASES.items() for K in c[3]])
def test_every_kernel(kernel, K, gather):
    counts, N, I, _ = CASES[kernel]
    R, G = sum(counts), len(counts)
    behind = 5    # rows of no group, left as they were
    for swiglu, cols in ((0, N), (1, I)):
        if cols is None:
            continue
        log(f"[int8 {kernel}] N={cols} K={K} swiglu={swiglu} gather={gather}")
        c = case(counts, 2 * cols if swiglu else cols, K, [K, cols, R], gather, extra_rows=behind)
        assert plan(swiglu, gather, len(c[1]), G, R + behind, cols, K, cus()) == kernel
        p = OI.products(c[1], c[3], c[2], c[4], c[0], c[5])
        fn = M.grouped_int8_gemm_swiglu if swiglu else M.grouped_int8_gemm
        out = run(fn, *c, R + behind, cols, K)
        got = bf16_values_host(out)[:R]
        if swiglu:
            check_swiglu(got, p, f"{kernel} swiglu")
        else:
            check(got, p, 4 * 2.0 ** -24, kernel)
        assert (host(out.view(torch.int16))[R:] == 0x4321).all()


@pytest.mark.parametrize("swiglu", [0, 1])
def test_one_group_holds_most_rows(swiglu):
    """Few rows on average, nearly all of them one group's."""
    counts = [1] * 60 + [700] + [0] * 39
    N, K, R = 1032 // (1 + swiglu) // 8 * 8, 400, 760
    assert plan(swiglu, 0, R, len(counts), R, N, K, cus()) in ("flow", "split16x64")
    c = case(counts, N * (1 + swiglu), K, [swiglu], False)
    p = OI.products(c[1], c[3], c[2], c[4], c[0])
    fn = M.grouped_int8_gemm_swiglu if swiglu else M.grouped_int8_gemm
    out = bf16_values_host(run(fn, *c, R, N, K))[:R]
    if swiglu:
        check_swiglu(out, p, "skewed")
    else:
        check(out, p, 4 * 2.0 ** -24, "skewed")


@pytest.mark.parametrize("kernel", ["wide", "mid"])
@pytest.mark.parametrize("swiglu", [0, 1])
def test_offsets_short_of_the_rows(kernel, swiglu):
    """The last group ends far before M_total, by whole tiles of every kernel."""
    counts, N, I, _ = CASES[kernel]
    K, R, behind = 272, sum(counts), 700
    cols = I if swiglu else N
    c = case(counts, 2 * cols if swiglu else cols, K, [K, 1], True, extra_rows=behind)
    assert plan(swiglu, 1, len(c[1]), len(counts), R + behind, cols, K, cus()) == kernel
    p = OI.products(c[1], c[3], c[2], c[4], c[0], c[5])
    out = run(M.grouped_int8_gemm_swiglu if swiglu else M.grouped_int8_gemm, *c, R + behind, cols, K)
    got = bf16_values_host(out)[:R]
    check_swiglu(got, p, kernel) if swiglu else check(got, p, 4 * 2.0 ** -24, kernel)
    assert (host(out.view(torch.int16))[R:] == 0x4321).all()


@pytest.mark.parametrize("kernel", ["wide", "mid"])
@pytest.mark.parametrize("swiglu", [0, 1])
def test_indices_out_of_range_are_clamped(kernel, swiglu):
    counts, N, I, _ = CASES[kernel]
    K, R, cols = 272, sum(counts), I if swiglu else N
    offs, a, b, sa, sb, index = case(counts, 2 * cols if swiglu else cols, K, [K, 2], True)
    index[::7] = 2 ** 31 - 1
    index[3::11] = -1
    index[5:20] = 2
    clamped = np.where((index < 0) | (index >= len(a)), len(a) - 1, index)
    assert plan(swiglu, 1, len(a), len(counts), R, cols, K, cus()) == kernel
    p = OI.products(a, sa, b, sb, offs, clamped)
    fn = M.grouped_int8_gemm_swiglu if swiglu else M.grouped_int8_gemm
    out = run(fn, offs, a, b, sa, sb, index, R, cols, K)
    got = bf16_values_host(out)[:R]
    check_swiglu(got, p, kernel) if swiglu else check(got, p, 4 * 2.0 ** -24, kernel)

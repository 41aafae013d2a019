"""The bf16 grouped products (projections, gated activation, input and weight
gradients) against FP64, at the sizes and groups where they can go wrong."""
import numpy as np
import pytest
import torch

import fp8_block_scaled_bias_amd as M
from bf16_cases import Case, check, up, values
from gpu_common import bf16_values_host, dev, host, log
from oracle import bf16 as OB

pytestmark = pytest.mark.gpu

# (rows of the groups, N, K, gather): one token, empty groups at both ends and
# inside, tiles that are whole, one over and one short, odd N and K
SHAPES = [
    ([1], 8, 8, False),
    ([1], 64, 512, True),
    ([0, 3, 0, 17, 0], 72, 72, False),
    ([130, 0, 1, 127], 136, 264, True),
    ([64, 65, 63, 0], 128, 128, False),
    ([256, 255, 257], 256, 192, True),
    ([33], 1416, 88, False),
    ([5, 300, 2, 2, 0, 0, 7, 64], 520, 200, True),
    ([1100], 264, 320, False),
]


@pytest.mark.parametrize("counts,N,K,gather", SHAPES)
def test_gemm(counts, N, K, gather):
    log(f"[bf16 gemm] {counts} N={N} K={K} gather={gather}")
    Case(counts, N, K, 1, gather).gemm("gemm")


@pytest.mark.parametrize("act", [M.ACT_SILU, M.ACT_GELU])
@pytest.mark.parametrize("counts,N,K,gather", SHAPES)
def test_gemm_glu(counts, N, K, gather, act):
    log(f"[bf16 glu] {counts} I={N} K={K} gather={gather} act={act}")
    Case(counts, N, K, 2, gather).glu(act, keep=(N + act) % 16 == 0, label="glu")


@pytest.mark.parametrize("counts,N,K,gather", SHAPES)
def test_dgrad(counts, N, K, gather):
    log(f"[bf16 dgrad] {counts} N={N} K={K}")
    Case(counts, N, K, 3).dgrad("dgrad")


@pytest.mark.parametrize("act", [M.ACT_SILU, M.ACT_GELU])
@pytest.mark.parametrize("counts,N,K,gather", SHAPES)
def test_dgrad_glu(counts, N, K, gather, act):
    log(f"[bf16 dgrad glu] {counts} N={N} I={K} act={act}")
    Case(counts, N, K, 4).dgrad_glu(act, "dgrad glu")


@pytest.mark.parametrize("counts,N,K,gather", SHAPES)
def test_wgrad(counts, N, K, gather):
    log(f"[bf16 wgrad] {counts} N={N} K={K} gather={gather}")
    Case(counts, N, K, 5, gather).wgrad("wgrad")


def test_exact_on_whole_numbers():
    """Whole numbers whose sums fp32 holds: every layout and index shows."""
    rng = np.random.default_rng(11)
    counts, N, K = [70, 0, 5, 200], 136, 152
    offs = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    R, G = int(offs[-1]), len(counts)
    a = rng.integers(-8, 9, (R, K)).astype(float)
    b = rng.integers(-8, 9, (G, N, K)).astype(float)
    dy = rng.integers(-8, 9, (R, N)).astype(float)
    dw = torch.empty((G, N, K), device="cuda")
    M.grouped_bf16_wgrad(up(dy), up(a), None, dev(offs), G, R, N, K, dw)
    assert np.array_equal(host(dw), OB.wgrad(dy, a, offs)[0])
    c = torch.empty((R, N), dtype=torch.bfloat16, device="cuda")
    M.grouped_bf16_gemm(up(a), None, up(b), dev(offs), G, R, N, K, c)
    from oracle.formats import bf16_round
    assert np.array_equal(bf16_values_host(c), bf16_round(OB.products(a, b, offs)[0]))
    da = torch.empty((R, K), dtype=torch.bfloat16, device="cuda")
    M.grouped_bf16_gemm_dgrad(up(dy), up(b), dev(offs), G, R, N, K, da)
    assert np.array_equal(bf16_values_host(da), bf16_round(OB.dgrad(dy, b, offs)[0]))


def test_infinities_stay_where_they_belong():
    """One row, one weight row, rows behind the last group and the memory next
    to the operands hold NaN: only results they take part in do."""
    rng = np.random.default_rng(12)
    counts, N, K = [9, 40, 3], 72, 72   # no size a multiple of a K block
    offs = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    R, G, behind = int(offs[-1]), 3, 5
    a, b = values(rng, (R, K)), values(rng, (G, N, K))
    dy = values(rng, (R, N))

    def inside(v, lead):
        """v as the middle of a NaN-filled tensor."""
        t = torch.full((v.shape[0] + 2 * lead,) + v.shape[1:], float("nan"), dtype=torch.bfloat16, device="cuda")
        t[lead:lead + v.shape[0]] = up(v)
        return t[lead:lead + v.shape[0] + (behind if v.shape[0] == R else 0)]
    ta, tb, td, to = inside(a, 8), inside(b, 1), inside(dy, 8), dev(offs)
    out = torch.empty((R + behind, N), dtype=torch.bfloat16, device="cuda")
    M.grouped_bf16_gemm(ta, None, tb, to, G, R + behind, N, K, out)
    check(bf16_values_host(out)[:R], *OB.products(a, b, offs), "gemm")
    da = torch.empty((R + behind, K), dtype=torch.bfloat16, device="cuda")
    M.grouped_bf16_gemm_dgrad(td, tb, to, G, R + behind, N, K, da)
    check(bf16_values_host(da)[:R], *OB.dgrad(dy, b, offs), "dgrad")
    dw = torch.empty((G, N, K), device="cuda")
    M.grouped_bf16_wgrad(td, ta, None, to, G, R + behind, N, K, dw)
    ref, err = OB.wgrad(dy, a, offs)
    assert (np.abs(host(dw) - ref) <= err + 2.0 ** -24 * np.abs(ref)).all()
    # one NaN in a row, one in a weight row
    a2, b2 = a.copy(), b.copy()
    ta[11, 5], tb[1, 7, 3] = float("nan"), float("inf")
    M.grouped_bf16_gemm(ta, None, tb, to, G, R + behind, N, K, out)
    got = bf16_values_host(out)[:R]
    bad = ~np.isfinite(got)
    expect = np.zeros_like(bad)
    expect[11], expect[9:49, 7] = True, True
    assert np.array_equal(bad, expect)
    check(np.where(expect, 0, got), *[np.where(expect, 0, v) for v in OB.products(a2, b2, offs)], "others")


def test_saturated_gates():
    """Gates far out on both sides: finite results, slopes of 0 and 1."""
    for act in (M.ACT_SILU, M.ACT_GELU):
        R, N, I = 8, 8, 16
        gu = np.zeros((R, 2 * I))
        gu[:, :I] = np.resize([-3e38, -1e20, -90.0, -17.0, -16.0, 16.0, 17.0, 90.0, 1e10, 0.0, -0.0, 1e-30, 5.0, -5.0,
                               88.5, -88.5], I)
        gu[:, I:] = 1.0
        from oracle.formats import bf16_round
        gu = bf16_round(gu).astype(np.float64)
        dc, w = np.zeros((R, N)), np.zeros((1, N, I))
        dc[:, 0], w[0, 0] = 1.0, 1.0
        out = torch.empty((R, 2 * I), dtype=torch.bfloat16, device="cuda")
        M.grouped_bf16_gemm_dgrad_glu(up(dc), up(w), up(gu), dev(np.array([0, R], np.int32)), 1, R, N, I, act, out)
        got = bf16_values_host(out)
        assert np.isfinite(got).all()
        ref = OB.glu_backward(gu, np.ones((R, I)), act)
        assert (np.abs(got - ref) <= 2.0 ** -8 * np.abs(ref) + 2.0 ** -20).all(), act


def test_wgrad_of_no_rows():
    dw = torch.full((3, 16, 8), float("nan"), device="cuda")
    z = torch.zeros((0, 16), dtype=torch.bfloat16, device="cuda")
    M.grouped_bf16_wgrad(z, torch.zeros((0, 8), dtype=torch.bfloat16, device="cuda"), None,
                         torch.zeros(4, dtype=torch.int32, device="cuda"), 3, 0, 16, 8, dw)
    assert (host(dw) == 0).all()
    # rows, but none of them in a group
    one = torch.ones((5, 16), dtype=torch.bfloat16, device="cuda")
    dw.fill_(float("nan"))
    M.grouped_bf16_wgrad(one, one[:, :8].contiguous(), None, torch.zeros(4, dtype=torch.int32, device="cuda"), 3, 5,
                         16, 8, dw)
    assert (host(dw) == 0).all()


def test_index_past_the_end_reads_the_last_row():
    rng = np.random.default_rng(13)
    a, b = values(rng, (4, 64)), values(rng, (1, 32, 64))
    idx = np.array([0, 3, 7, -1, 2], np.int32)
    out = torch.empty((5, 32), dtype=torch.bfloat16, device="cuda")
    M.grouped_bf16_gemm(up(a), dev(idx), up(b), dev(np.array([0, 5], np.int32)), 1, 5, 32, 64, out)
    check(bf16_values_host(out), *OB.products(a[np.array([0, 3, 3, 3, 2])], b, np.array([0, 5])), "clamped")

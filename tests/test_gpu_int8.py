"""The int8 quantisers and grouped products against the whole-number oracle:
codes and scales exactly, products within the roundings of their outputs."""
import numpy as np
import pytest
import torch

import fp8_block_scaled_bias_amd as M
from gpu_common import bf16_dev, bf16_values_host, dev, host, log
from oracle import int8 as OI
from oracle.formats import bf16_value_from_bits

pytestmark = pytest.mark.gpu


def bf16_bits(v):
    return torch.from_numpy(np.asarray(v, np.float32)).to(torch.bfloat16).view(torch.int16).numpy().view(np.uint16)


def hard_rows(K, rng):
    """Rows with ties, zeros, subnormal and very large values."""
    v = (rng.standard_normal((8, K)) * np.exp(rng.standard_normal((8, 1)))).astype(np.float32)
    v[1] = (np.arange(K) % 253 - 126) * 0.5       # all ties at scale 1 ...
    v[1, 0] = 127.0
    v[2] = v[1] * np.float32(2.0 ** -20)           # ... and at another power of two
    v[3] = 0
    v[4] = rng.standard_normal(K) * 1e-39          # subnormal
    v[5] = 0
    v[5, K // 2] = -1e-40
    v[6] = rng.standard_normal(K) * 1e37
    v[7] = -0.0
    v[7, K - 1] = 3e-3
    return v


@pytest.mark.parametrize("M_,K,ld", [(1, 8, 8), (1, 7168, 7168), (3, 24, 40), (130, 128, 136), (67, 2048, 2048),
                                     (200, 7168, 7176), (5, 8200, 8200), (2, 40000, 40000)])
def test_quant_rows(M_, K, ld):
    rng = np.random.default_rng([M_, K])
    x = (rng.standard_normal((M_, ld)) * np.exp(rng.standard_normal((M_, 1)) * 2)).astype(np.float32)
    x[: min(8, M_), :K] = hard_rows(K, rng)[: min(8, M_)]
    bits = bf16_bits(x)
    log(f"[int8 rows] M={M_} K={K} ld={ld}")
    q = torch.full((M_ + 1, K), 99, dtype=torch.int8, device="cuda")
    s = torch.full((M_ + 1,), np.nan, device="cuda")
    M.int8_quant_rows(bf16_dev(bits), M_, K, ld, q, s)
    rq, rs = OI.quant_rows(bf16_value_from_bits(bits[:, :K]))
    assert np.array_equal(host(s)[:M_], rs) and np.array_equal(host(q)[:M_], rq)
    assert (host(q)[M_] == 99).all() and np.isnan(host(s)[M_])   # the row behind the last


def test_quant_rows_every_bf16_against_many_scales():
    """Every finite bf16 value below a row's largest, at 64 largest values."""
    rng = np.random.default_rng(0)
    pos = np.arange(0x0080, 0x7F00, dtype=np.uint16)
    tops = rng.choice(pos[pos > 0x2000], 64, replace=False)
    K = 0x1000
    rows = []
    for top in tops:
        v = (top - np.minimum(np.arange(K), top - 1)).astype(np.uint16)
        v[1::2] |= 0x8000
        rows.append(v)
    bits = np.stack(rows)
    q = torch.empty(bits.shape, dtype=torch.int8, device="cuda")
    s = torch.empty(len(tops), device="cuda")
    M.int8_quant_rows(bf16_dev(bits), len(tops), K, K, q, s)
    rq, rs = OI.quant_rows(bf16_value_from_bits(bits))
    assert np.array_equal(host(s), rs) and np.array_equal(host(q), rq)


@pytest.mark.parametrize("G,N,K", [(1, 1, 8), (2, 9, 24), (3, 40, 1024), (2, 130, 7168), (1, 3, 9000)])
def test_quant_channels(G, N, K):
    rng = np.random.default_rng([N, K])
    w = (rng.standard_normal((G, N, K)) * 0.02).astype(np.float32)
    flat = w.reshape(G * N, K)
    n = min(8, G * N)
    flat[:n] = hard_rows(K, rng)[:n]
    if G * N > 8:
        flat[8] = np.float32(1e-45)
    log(f"[int8 channels] G={G} N={N} K={K}")
    q = torch.empty((G, N, K), dtype=torch.int8, device="cuda")
    s = torch.empty((G, N), device="cuda")
    M.int8_quant_channels(dev(w), G, N, K, q, s)
    rq, rs = OI.quant_rows(w)
    assert np.array_equal(host(s), rs) and np.array_equal(host(q), rq)


def case(counts, N, K, seed, gather, extra_rows=0, all_low=False):
    rng = np.random.default_rng(seed)
    G, R = len(counts), int(sum(counts))
    offs = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    a_rows = max(1, R // 2) if gather else R + extra_rows
    a = rng.integers(-127, 128, (a_rows, K)).astype(np.int8)
    b = rng.integers(-127, 128, (G, N, K)).astype(np.int8)
    if all_low:
        a[:], b[:] = -128, -128
    sa = np.exp(rng.standard_normal(a_rows)).astype(np.float32) * np.float32(0.02)
    sb = rng.uniform(0.5, 1.5, (G, N)).astype(np.float32) * np.float32(0.02 / np.sqrt(K))
    index = rng.integers(0, a_rows, R + extra_rows).astype(np.int32) if gather else None
    return offs, a, b, sa, sb, index


def run(fn, offs, a, b, sa, sb, index, M_total, N, K):
    out = bf16_dev(np.full((M_total + 1, N), 0x4321, np.uint16))
    fn(dev(a), dev(sa), None if index is None else dev(index), dev(b), dev(sb), dev(offs), len(offs) - 1,
       M_total, N, K, out)
    return out


def check(got, ref, rel, label):
    """One bf16 rounding (2^-8 of the value) on top of the fp32 ones."""
    d = np.abs(got.astype(np.float64) - ref)
    tol = (2.0 ** -8 + rel) * np.abs(ref) + 2.0 ** -133
    assert (d <= tol).all(), f"{label}: worst {np.max(d - tol)} at {np.argwhere(d > tol)[:4].tolist()}"


def check_swiglu(got, p, label):
    """silu(g) u from products p = [g, u].  g and u are off by 4 roundings each
    (2^-24); silu turns a relative error d of its argument into |1 + g (1 -
    sigmoid(g))| d, at most 1.3 d for g > 0 and (1 + |g|) d for g < 0; then exp
    (2 roundings of at most half its value), an addition, a quotient, a
    product: 8 in all; then the rounding to bf16.  Below g = -88 exp(-g)
    overflows and silu is 0, where the exact one is under 88 e^-88 < 2^-118."""
    I = p.shape[1] // 2
    ref, g = OI.swiglu(p), np.abs(p[:, :I])
    tol = ((2.0 ** -8 + (4 * (1 + np.minimum(g, 90)) + 12) * 2.0 ** -24) * np.abs(ref)
           + 2.0 ** -118 * np.abs(p[:, I:]) + 2.0 ** -133)
    d = np.abs(got.astype(np.float64) - ref)
    assert (d <= tol).all(), f"{label}: worst {np.max(d - tol)} at {np.argwhere(d > tol)[:4].tolist()}"


GROUPS = {
    "one row": [1], "dense": [70], "decode": [0, 3, 0, 1, 16, 17, 0, 40],
    "ragged": [5, 0, 130, 64, 1, 33, 300], "prefill": [260, 257, 0, 700, 1],
    "empty": [0, 0, 0, 2], "many": [1, 2, 0] * 90,
}


@pytest.mark.parametrize("groups", list(GROUPS))
@pytest.mark.parametrize("N,K", [(8, 16), (24, 48), (136, 208), (256, 1024), (264, 1040), (520, 144)])
@pytest.mark.parametrize("gather", [False, True])
def test_grouped_gemm_and_swiglu(groups, N, K, gather):
    counts = GROUPS[groups]
    if groups == "many" and N * K > 300000:
        pytest.skip("size: the many small groups run at the smaller matrices")
    R = sum(counts)
    log(f"[int8 gemm] {groups} N={N} K={K} gather={gather}")
    c = case(counts, N, K, [N, K, R], gather, extra_rows=3)
    p = OI.products(c[1], c[3], c[2], c[4], c[0], c[5])
    # fp32: conversion of the sum, product of the scales, their product
    out = run(M.grouped_int8_gemm, *c, R + 3, N, K)
    got = bf16_values_host(out)
    check(got[:R], p, 4 * 2.0 ** -24, "gemm")
    # rows of no group are left as they were
    assert (host(out.view(torch.int16))[R:] == 0x4321).all()
    if N % 16 == 0:
        I = N // 2
        out = run(M.grouped_int8_gemm_swiglu, *c, R + 3, I, K)
        check_swiglu(bf16_values_host(out)[:R], p, "swiglu")
        assert (host(out.view(torch.int16))[R:] == 0x4321).all()


@pytest.mark.parametrize("counts,N,K", [([1], 4096, 7168), ([9, 0, 2], 1008, 7168), ([600, 300], 256, 4112),
                                        ([1500], 1040, 2064), ([128] * 9, 512, 768)])
def test_larger_products(counts, N, K):
    R = sum(counts)
    log(f"[int8 gemm] counts={counts[:4]} N={N} K={K}")
    c = case(counts, N, K, [N, K], False)
    p = OI.products(c[1], c[3], c[2], c[4], c[0], c[5])
    check(bf16_values_host(run(M.grouped_int8_gemm, *c, R, N, K))[:R], p, 4 * 2.0 ** -24, "gemm")
    c = case(counts, N, K, [N, K, 1], True)
    p = OI.products(c[1], c[3], c[2], c[4], c[0], c[5])
    I = N // 2
    check_swiglu(bf16_values_host(run(M.grouped_int8_gemm_swiglu, *c, R, I, K))[:R], p, "swiglu")


@pytest.mark.parametrize("rows", [1, 20, 300])
def test_longest_sum(rows):
    """All codes -128 at the largest K: the sum is 2^31 - 2^18, still positive."""
    K = 131072 - 16
    c = case([rows], 8, K, 3, False, all_low=True)
    p = OI.products(c[1], c[3], c[2], c[4], c[0], c[5])
    check(bf16_values_host(run(M.grouped_int8_gemm, *c, rows, 8, K))[:rows], p, 4 * 2.0 ** -24, "gemm")


def test_indices_past_the_rows_are_clamped_and_repeat():
    counts, N, K = [4, 30, 0, 300], 64, 128
    offs, a, b, sa, sb, index = case(counts, N, K, 9, True)
    index[::7] = 2 ** 31 - 1
    index[3::11] = -1
    index[5:20] = 2
    clamped = np.where((index < 0) | (index >= len(a)), len(a) - 1, index)
    p = OI.products(a, sa, b, sb, offs, clamped)
    out = run(M.grouped_int8_gemm, offs, a, b, sa, sb, index, sum(counts), N, K)
    check(bf16_values_host(out)[:sum(counts)], p, 4 * 2.0 ** -24, "gemm")


def test_saturated_gate_and_zero_scales():
    """Gates far from zero (silu is 0 or the gate itself) and zero scales."""
    counts, I, K = [3, 40], 16, 64
    offs, a, b, sa, sb, index = case(counts, 2 * I, K, 4, False)
    sb[:] *= 3e4
    sa[5] = 0
    p = OI.products(a, sa, b, sb, offs, index)
    assert np.abs(p[:, :I]).max() > 500
    out = bf16_values_host(run(M.grouped_int8_gemm_swiglu, offs, a, b, sa, sb, index, 43, I, K))[:43]
    assert np.isfinite(out).all()
    check_swiglu(out, p, "saturated")
    assert (out[5] == 0).all()


def test_streams_and_graph_replay():
    """Two calls on two streams at once, then both captured and replayed."""
    cs = [case([20, 0, 50], 128, 256, 1, False), case([7, 400], 128, 256, 2, False)]
    on = [[dev(x) for x in (c[1], c[3], c[2], c[4], c[0])] for c in cs]
    outs = [torch.empty((sum(np.diff(c[0])), 128), dtype=torch.bfloat16, device="cuda") for c in cs]
    refs = [OI.products(c[1], c[3], c[2], c[4], c[0]) for c in cs]

    def call(i, stream):
        a, sa, b, sb, offs = on[i]
        M.grouped_int8_gemm(a, sa, None, b, sb, offs, len(offs) - 1, outs[i].shape[0], 128, 256, outs[i], stream)

    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(4):
        for i in (0, 1):
            call(i, streams[i])
    torch.cuda.synchronize()
    for i in (0, 1):
        check(bf16_values_host(outs[i]), refs[i], 4 * 2.0 ** -24, f"stream {i}")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(0, torch.cuda.current_stream())
        call(1, torch.cuda.current_stream())
    for rep in range(3):
        for o in outs:
            o.zero_()
        graph.replay()
        torch.cuda.synchronize()
        for i in (0, 1):
            check(bf16_values_host(outs[i]), refs[i], 4 * 2.0 ** -24, f"replay {rep}")
        call(rep % 2, None)
        torch.cuda.synchronize()


@pytest.mark.parametrize("R,a_rows,N,K,gather", [
    (1048700, 1048700, 8, 4096, False),    # rows of A past 2^32 bytes
    (300, 1048700, 136, 4096, True),       # gathered from there
    (20, 1048700, 24, 4096, True),
    (1048700, 1048700, 2056, 144, False),  # the output past 2^32 bytes
    (33560000, 1000, 64, 16, True),
])
def test_offsets_past_32_bits(R, a_rows, N, K, gather):
    """Two groups, the second from an odd row on; sampled rows, the last ones
    among them."""
    log(f"[int8 far] R={R} A={a_rows} N={N} K={K} gather={gather}")
    gen = torch.Generator(device="cuda").manual_seed(5)
    a = torch.randint(-127, 128, (a_rows, K), dtype=torch.int8, device="cuda", generator=gen)
    b = torch.randint(-127, 128, (2, N, K), dtype=torch.int8, device="cuda", generator=gen)
    sa = torch.rand((a_rows,), device="cuda", generator=gen) + 0.5
    sb = torch.rand((2, N), device="cuda", generator=gen) + 0.5
    index = None
    if gather:
        index = torch.randint(0, a_rows, (R,), dtype=torch.int32, device="cuda", generator=gen)
        index[-7:] = a_rows - 1 - torch.arange(7, dtype=torch.int32, device="cuda")
    cut = R // 2 + 1
    out = torch.zeros((R, N), dtype=torch.bfloat16, device="cuda")
    M.grouped_int8_gemm(a, sa, index, b, sb, dev(np.array([0, cut, R], np.int32)), 2, R, N, K, out)
    rows = np.unique(np.concatenate([np.arange(0, R, max(1, R // 97)), np.arange(cut - 3, cut + 3),
                                     np.arange(R - 9, R)]))
    pick = torch.from_numpy(rows).cuda()
    src = pick if index is None else index[pick].long()
    offs = np.array([0, int((rows < cut).sum()), len(rows)], np.int32)
    p = OI.products(host(a[src]), host(sa[src]), host(b), host(sb), offs)
    check(bf16_values_host(out[pick].contiguous()), p, 4 * 2.0 ** -24, "gemm")
    del a, out
    torch.cuda.empty_cache()


def test_quantised_rows_past_32_bits():
    M_, K = 300_007, 8192   # 4.9 GB of bf16, 2.46 GB of codes
    x = torch.empty((M_, K), dtype=torch.bfloat16, device="cuda")
    pick = np.array([0, 1, 131071, 131072, 262143, 262144, M_ - 2, M_ - 1])
    x.normal_(generator=torch.Generator(device="cuda").manual_seed(6))
    q = torch.empty((M_, K), dtype=torch.int8, device="cuda")
    s = torch.empty((M_,), device="cuda")
    log(f"[int8 rows far] M={M_} K={K}")
    M.int8_quant_rows(x, M_, K, K, q, s)
    at = torch.from_numpy(pick).cuda()
    rq, rs = OI.quant_rows(host(x[at].float()))
    assert np.array_equal(host(s[at]), rs) and np.array_equal(host(q[at]), rq)
    del x, q
    torch.cuda.empty_cache()


@pytest.mark.parametrize("rows,behind", [(0, 3), (1, 0), (1, 15), (16, 0), (9, 30), (60, 4)])
@pytest.mark.parametrize("gather", [False, True])
def test_one_group_of_few_rows(rows, behind, gather):
    """One group (a linear layer) whose rows fit a tile, with rows behind it."""
    N, K = 272, 400
    log(f"[int8 one group] {rows}+{behind} gather={gather}")
    c = case([rows], N, K, [rows, behind], gather, extra_rows=behind)
    p = OI.products(c[1], c[3], c[2], c[4], c[0], c[5])
    out = run(M.grouped_int8_gemm, *c, rows + behind, N, K)
    check(bf16_values_host(out)[:rows], p, 4 * 2.0 ** -24, "gemm")
    assert (host(out.view(torch.int16))[rows:] == 0x4321).all()
    out = run(M.grouped_int8_gemm_swiglu, *c, rows + behind, N // 2, K)
    check_swiglu(bf16_values_host(out)[:rows], p, "swiglu")
    assert (host(out.view(torch.int16))[rows:] == 0x4321).all()


@pytest.mark.parametrize("M_,K", [(300, 4096), (256, 4096), (512, 8192), (513, 7168), (513, 8200), (512, 16384),
                                  (2048, 520), (2051, 2048), (2047, 1024)])
def test_quant_rows_by_every_number_of_waves(M_, K):
    """Rows by one wave, four and sixteen, at both sides of each border."""
    rng = np.random.default_rng([M_, K])
    bits = bf16_bits(np.concatenate([hard_rows(K, rng), rng.standard_normal((M_ - 8, K)).astype(np.float32)]))
    q = torch.full((M_, K), 99, dtype=torch.int8, device="cuda")
    s = torch.full((M_,), -1.0, device="cuda")
    log(f"[int8 rows] M={M_} K={K}")
    M.int8_quant_rows(bf16_dev(bits), M_, K, K, q, s)
    rq, rs = OI.quant_rows(bf16_value_from_bits(bits).astype(np.float32))
    assert np.array_equal(host(s), rs) and np.array_equal(host(q), rq)

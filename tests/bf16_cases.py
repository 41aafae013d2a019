"""Operands and checks shared by the GPU tests of the bf16 grouped products."""
import numpy as np

import fp8_block_scaled_bias_amd as M
from gpu_common import bf16_dev, bf16_values_host, dev, host
from oracle import bf16 as OB
from oracle.formats import bf16_bits_from_value as bits_of, bf16_round, bf16_value_from_bits

U = 2.0 ** -24


def values(rng, shape, sigma=1.0):
    return bf16_round(rng.standard_normal(shape) * sigma).astype(np.float64)


def up(v):
    return bf16_dev(bits_of(v))


def offsets(counts):
    return np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)


def check(got, ref, err, label):
    """|got - ref| within err (of the fp32 evaluation) and one bf16 rounding."""
    d = np.abs(got.astype(np.float64) - ref)
    tol = err + 2.0 ** -8 * (np.abs(ref) + err) + 2.0 ** -133
    bad = ~(d <= tol)
    assert not bad.any(), f"{label}: {bad.sum()} off, worst {np.nanmax(d - tol)} at {np.argwhere(bad)[:4].tolist()}"


def act_errors(g, eg, act):
    """Bounds on the fp32 evaluation of act(g) and its slope where g itself is
    off by eg.  Both have slopes of at most 1.2 (act) and 1.2 (its slope: |act''|
    <= 0.5 for SiLU, 0.8 for GELU).  z carries 5 roundings, so exp(-z) is off
    by (5 |z| + 2) roundings relative to itself, and s = 1 / (1 + exp(-z)) by
    that times 1 - s, and 3; |z| (1 - s) <= 0.3 for z > 0 and |z| s is what is
    left of it for z < 0.  act = g s has one more, the slope's second term g s
    (1 - s) dz five more, with 1 - s off by the same absolute amount as s: in
    all at most 16 (1 + |z|) roundings of the sizes |act| and s + |g| s (1 +
    dz), and where s rounds to 1 the term that 1 - s loses, 2^-24 |g| dz."""
    a, slope, z = OB.activation(g, act)
    s = OB._logistic(z)
    dz = np.ones_like(g) if act == OB.SILU else 1.6 * (1 + 0.135 * np.minimum(np.abs(g), 16) ** 2)
    n = 16 * (1 + np.minimum(np.abs(z), 700)) * U
    lost = 2.0 ** -126 * (1 + np.abs(g))
    ea = 1.2 * eg + n * np.abs(a) + lost
    es = 1.2 * eg + n * (s + np.abs(g) * s * (1 - s) * dz) + 4 * U * np.abs(np.clip(g, -16, 16)) * s * dz + lost * (1 + dz)
    return ea, es


def check_glu(h, p, e, act, label):
    I = p.shape[1] // 2
    g, u, eg, eu = p[:, :I], p[:, I:], e[:, :I], e[:, I:]
    a, _, _ = OB.activation(g, act)
    ea, _ = act_errors(g, eg, act)
    check(h, a * u, ea * (np.abs(u) + eu) + np.abs(a) * eu + 2 * U * np.abs(a * u), label)


def check_dglu(got, gu, dh, e, act, label):
    I = gu.shape[1] // 2
    g, u = gu[:, :I], gu[:, I:]
    a, slope, _ = OB.activation(g, act)
    ea, es = act_errors(g, 0.0, act)
    size = np.abs(dh) + e
    eg = e * np.abs(u * slope) + size * np.abs(u) * es + 4 * U * np.abs(dh * u * slope)
    eu = e * np.abs(a) + size * ea + 4 * U * np.abs(dh * a)
    check(got, OB.glu_backward(gu, dh, act), np.concatenate([eg, eu], axis=1), label)


class Case:
    """Groups of given sizes; rows behind the last group hold a mark."""

    def __init__(self, counts, N, K, seed, gather=False, behind=3):
        self.rng = rng = np.random.default_rng([seed, N, K, *counts])
        self.counts, self.N, self.K = counts, N, K
        self.offs, self.G = offsets(counts), len(counts)
        self.R = int(self.offs[-1])
        self.M = self.R + behind
        self.a_rows = max(1, self.R // 2) if gather else self.M
        self.index = rng.integers(0, self.a_rows, self.M).astype(np.int32) if gather else None
        self.d_index = None if self.index is None else dev(self.index)
        self.d_offs = dev(self.offs)

    def marked(self, N, dtype=None):
        return bf16_dev(np.full((self.M, N), 0x4321, np.uint16))

    def result(self, t):
        bits = bf16_values_host(t)
        assert (bits[self.R:] == bf16_value_from_bits(np.uint16(0x4321))).all(), "rows behind the last group"
        return bits[:self.R]

    def gemm(self, label):
        a, b = values(self.rng, (self.a_rows, self.K)), values(self.rng, (self.G, self.N, self.K), self.K ** -0.5)
        out = self.marked(self.N)
        M.grouped_bf16_gemm(up(a), self.d_index, up(b), self.d_offs, self.G, self.M, self.N, self.K, out)
        check(self.result(out), *OB.products(a, b, self.offs, self.index), label)

    def glu(self, act, keep, label):
        a = values(self.rng, (self.a_rows, self.K), 2.0)
        b = values(self.rng, (self.G, 2 * self.N, self.K), self.K ** -0.5)
        out, gu = self.marked(self.N), self.marked(2 * self.N) if keep else None
        M.grouped_bf16_gemm_glu(up(a), self.d_index, up(b), self.d_offs, self.G, self.M, self.N, self.K, act, out, gu)
        p, e = OB.products(a, b, self.offs, self.index)
        check_glu(self.result(out), p, e, act, label)
        if keep:
            check(self.result(gu), p, e, label + " kept")

    def dgrad(self, label):
        dc, w = values(self.rng, (self.M, self.N)), values(self.rng, (self.G, self.N, self.K), self.N ** -0.5)
        out = self.marked(self.K)
        M.grouped_bf16_gemm_dgrad(up(dc), up(w), self.d_offs, self.G, self.M, self.N, self.K, out)
        check(self.result(out), *OB.dgrad(dc, w, self.offs), label)

    def dgrad_glu(self, act, label):
        dc, w = values(self.rng, (self.M, self.N)), values(self.rng, (self.G, self.N, self.K), self.N ** -0.5)
        gu = values(self.rng, (self.M, 2 * self.K), 3.0)
        out = self.marked(2 * self.K)
        M.grouped_bf16_gemm_dgrad_glu(up(dc), up(w), up(gu), self.d_offs, self.G, self.M, self.N, self.K, act, out)
        dh, e = OB.dgrad(dc, w, self.offs)
        check_dglu(self.result(out), gu[:self.R], dh, e, act, label)

    def wgrad(self, label):
        dy, a = values(self.rng, (self.M, self.N)), values(self.rng, (self.a_rows, self.K))
        out = dev(np.full((self.G, self.N, self.K), np.nan, np.float32))
        M.grouped_bf16_wgrad(up(dy), up(a), self.d_index, self.d_offs, self.G, self.M, self.N, self.K, out)
        ref, err = OB.wgrad(dy, a, self.offs, self.index)
        d = np.abs(host(out).astype(np.float64) - ref)
        assert (d <= err + U * np.abs(ref)).all(), f"{label}: worst {np.max(d - err)}"

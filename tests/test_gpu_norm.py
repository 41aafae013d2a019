"""The norms before and after a block, their codes and gradients against FP64,
within bounds of an fp32 evaluation."""
import numpy as np
import pytest
import torch

import fp8_block_scaled_bias_amd as M
from bf16_cases import U, check, up, values
from gpu_common import bf16_values_host, dev, host, log
from oracle import norm as ON
from oracle.formats import e4m3_decode

pytestmark = pytest.mark.gpu

EPS = 1e-6
F32, BF16 = torch.float32, torch.bfloat16


def stream(rng, shape, dtype, sigma=1.0):
    """Values of the residual stream and their tensor."""
    if dtype == BF16:
        v = values(rng, shape, sigma)
        return v, up(v)
    v = (rng.standard_normal(shape) * sigma).astype(np.float32)
    return v.astype(np.float64), dev(v)


def get(t):
    return bf16_values_host(t) if t.dtype == BF16 else host(t).astype(np.float64)


def check_as(t, ref, err, label):
    """Within err and one rounding to the tensor's type."""
    if t.dtype == BF16:
        return check(get(t), ref, err, label)
    d = np.abs(get(t) - ref)
    tol = err + U * np.abs(ref) + 2.0 ** -149
    assert (d <= tol).all(), f"{label}: worst {np.max(d - tol)} at {np.argwhere(d > tol)[:4].tolist()}"


def check_e4m3(codes, scales, v, e, label):
    """1x128 codes of values v off by e: the scale within its maximum's error
    and two roundings; a code within half a step of the value (2^-4 of it, or
    half the smallest step, 2^-10 scales) and the value's own error."""
    T, H = v.shape
    tiles = np.abs(v).reshape(T, -1, 128)
    s, top = host(scales).astype(np.float64), tiles.max(axis=2)
    es = (e.reshape(tiles.shape).max(axis=2) + 2 * U * top) / 448
    zero = top == 0
    assert (s[zero] == 1).all() and (np.abs(s - top / 448)[~zero] <= es[~zero]).all(), f"{label}: scales"
    wide = np.repeat(s, 128, axis=1)
    got = e4m3_decode(host(codes)).reshape(T, H) * wide
    tol = (2.0 ** -4 + 4 * U) * np.abs(v) + 2.0 ** -10 * wide * (1 + 2.0 ** -20) + 2 * e
    assert (np.abs(got - v) <= tol).all(), f"{label}: codes, worst {np.max(np.abs(got - v) - tol)}"


def rows_of(rng, T, H, dtype):
    """Rows of different sizes; one of zeros and one of very small values."""
    v, _ = stream(rng, (T, H), dtype)
    v = v * 2.0 ** rng.integers(-6, 7, (T, 1))
    if T > 2:
        v[1] = 0
        v[2] = v[2] * 2.0 ** -40
    return v, up(v) if dtype == BF16 else dev(v.astype(np.float32))


SIZES = [(1, 8), (3, 64), (5, 520), (4, 128), (2, 8192), (3, 8200), (2, 16384), (130, 1024), (7, 7168), (600, 256)]


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("T,H", SIZES)
def test_norm(T, H, dtype):
    rng = np.random.default_rng([T, H])
    for quant in (M.QUANT_NONE, M.QUANT_INT8) + ((M.QUANT_E4M3,) if H % 128 == 0 else ()):
        with_add, with_weight = quant != M.QUANT_INT8, quant != M.QUANT_NONE
        log(f"[norm] T={T} H={H} {dtype} quant={quant}")
        v, x = rows_of(rng, T, H, dtype)
        add = sum_out = None
        if with_add:
            add = up(values(rng, (T, H), 0.3))
            if T > 2:
                add[1] = 0
            total = (x.float().cpu() + add.float().cpu()).to(dtype)   # one fp32 addition, one rounding
            v, sum_out = (total.float().numpy().astype(np.float64), torch.empty_like(x))
        w32 = (1 + 0.2 * rng.standard_normal(H)).astype(np.float32)
        weight = dev(w32) if with_weight else None
        n = torch.full((T + 1, H), 7.0, dtype=BF16, device="cuda")
        rstd = torch.empty(T, device="cuda")
        codes = scales = None
        if quant == M.QUANT_E4M3:
            codes = torch.empty((T, H), dtype=torch.uint8, device="cuda")
            scales = torch.empty((T, H // 128), device="cuda")
        elif quant == M.QUANT_INT8:
            codes = torch.empty((T, H), dtype=torch.int8, device="cuda")
            scales = torch.empty(T, device="cuda")
        M.moe_norm(x, add, weight, T, H, EPS, sum_out, n, rstd, quant, codes, scales)
        ref, err, r, er = ON.norm(v, w32.astype(np.float64) if with_weight else 1.0, EPS)
        check(bf16_values_host(n)[:T], ref, err, "n")
        assert (bf16_values_host(n)[T] == 7).all()
        assert (np.abs(host(rstd) - r) <= er * r).all(), "rstd"
        if with_add:
            assert np.array_equal(get(sum_out), v), "sum"
        if quant == M.QUANT_E4M3:
            check_e4m3(codes, scales, ref, err, "codes")
        elif quant == M.QUANT_INT8:
            top, s = np.abs(ref).max(axis=1), host(scales).astype(np.float64)
            some = top > 0
            assert (s[~some] == 1).all()
            assert (np.abs(s - top / 127)[some] <= (err.max(axis=1) + 3 * U * top)[some] / 127).all()
            q = host(codes).astype(np.float64)
            tol = s[:, None] * (0.5 + 127 * 2 * U) + err
            assert (np.abs(q * s[:, None] - ref) <= tol).all() and np.abs(q).max() <= 127


def test_norm_in_place_and_optional_outputs():
    rng = np.random.default_rng(3)
    T, H = 9, 264
    for dtype in (F32, BF16):
        _, x = stream(rng, (T, H), dtype)
        add = up(values(rng, (T, H)))
        n, s = torch.empty((T, H), dtype=BF16, device="cuda"), torch.empty_like(x)
        M.moe_norm(x, add, None, T, H, EPS, s, n)
        again, n2 = x.clone(), torch.empty_like(n)
        M.moe_norm(again, add, None, T, H, EPS, again, n2)
        assert torch.equal(again, s) and torch.equal(n, n2)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("T,H", SIZES + [(1100, 72)])
def test_norm_backward(T, H, dtype):
    rng = np.random.default_rng([T, H, 1])
    log(f"[norm backward] T={T} H={H} {dtype}")
    v, x = rows_of(rng, T, H, dtype)
    w32 = (1 + 0.2 * rng.standard_normal(H)).astype(np.float32)
    dn = values(rng, (T, H))
    r32 = (1 / np.sqrt((v * v).mean(axis=1) + EPS)).astype(np.float32)
    ws_bytes = M.moe_norm_backward_workspace_bytes(T, H)
    ws = torch.full((ws_bytes,), 0xFF, dtype=torch.uint8, device="cuda")   # (NaN as fp32)
    for scale, weight in ((1.0, w32), (-0.25, None)):
        res, d_res = stream(rng, (T, H), dtype) if weight is not None else (np.zeros((T, H)), None)
        dx = torch.empty_like(x)
        dw = torch.full((H,), float("nan"), device="cuda")
        M.moe_norm_backward(up(dn), x, None if weight is None else dev(weight), dev(r32), d_res, scale, T, H, dx, dw,
                            ws, ws_bytes)
        ref, err, rw, ew = ON.norm_backward(dn, v, 1.0 if weight is None else weight.astype(np.float64),
                                            r32.astype(np.float64), res, scale)
        check_as(dx, ref, err, "dx")
        assert (np.abs(host(dw) - rw) <= ew + U * np.abs(rw)).all(), "d_weight"
        # in place over d_res, without d_weight, the same bits
        if d_res is not None:
            M.moe_norm_backward(up(dn), x, dev(weight), dev(r32), d_res, scale, T, H, d_res, None, None, 0)
            assert torch.equal(d_res, dx)


COMBINE = [(1, 1, 8, 0, 1), (3, 8, 128, 1, 1), (5, 2, 520, 1, 0), (2, 8, 8192, 1, 1), (2, 3, 8200, 0, 1), (1, 8, 16384, 1, 1),
           (64, 6, 1024, 1, 1), (600, 4, 256, 1, 1), (9, 8, 7168, 1, 0), (530, 1, 64, 0, 0)]


class Block:
    """A token batch at the end of a block."""

    def __init__(self, T, k, H, shared, dtype, seed=5):
        rng = self.rng = np.random.default_rng([T, k, H, seed])
        self.T, self.k, self.H, self.shared = T, k, H, shared
        self.D = values(rng, (T * (k + shared), H), 0.7)
        if T > 2:
            self.D[T * k:] *= 2.0 ** -8
        self.perm = rng.permutation(T * k).astype(np.int32)
        w = rng.random((T, k)).astype(np.float32)
        self.w = (w / w.sum(axis=1, keepdims=True)).astype(np.float32)
        if T > 2:
            self.w[0, 0] = 0      # a choice of weight 0
            if not shared:
                self.w[2] = 0     # a token of nothing at all
        self.sw = rng.random(T).astype(np.float32) if shared else None
        self.weight = (1 + 0.2 * rng.standard_normal(H)).astype(np.float32)
        self.x, self.d_x = stream(rng, (T, H), dtype)
        self.dD = up(self.D)
        self.S = self.dD[T * k:] if shared else None

    def rows(self, gated):
        sw = None if not self.shared else self.sw.astype(np.float64) if gated else np.ones(self.T)
        return ON.gather(self.D, self.perm, self.w.astype(np.float64), sw, self.T, self.k)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("T,k,H,shared,norm", COMBINE)
def test_combine_norm(T, k, H, shared, norm, dtype):
    b = Block(T, k, H, shared, dtype)
    for gated, weighted in ((0, 1), (shared, 0)):
        log(f"[combine norm] T={T} k={k} H={H} shared={shared} norm={norm} {dtype} gated={gated}")
        y = torch.full((T + 1, H), 9.0, dtype=dtype, device="cuda")
        rstd = torch.full((T,), -1.0, device="cuda")
        M.moe_combine_norm(b.dD, dev(b.perm), dev(b.w), b.S, dev(b.sw) if gated else None, b.d_x, 0.5, norm,
                           dev(b.weight) if weighted else None, EPS, 2.0, T, k, H, y, rstd)
        rows, w = b.rows(gated)
        ref, err, r = ON.combine_norm(rows, w, b.x, 0.5, norm, b.weight.astype(np.float64) if weighted else 1.0, EPS, 2.0)
        check_as(y[:T], ref, err, "y")
        assert (get(y[T:]) == 9).all()
        got = host(rstd)
        assert (np.abs(got - r[0]) <= r[1] * r[0]).all() if norm else (got == -1).all()
        # in place over the residual, the same bits
        x2 = b.d_x.clone()
        M.moe_combine_norm(b.dD, dev(b.perm), dev(b.w), b.S, dev(b.sw) if gated else None, x2, 0.5, norm,
                           dev(b.weight) if weighted else None, EPS, 2.0, T, k, H, x2)
        assert torch.equal(x2, y[:T])


def test_combine_norm_without_norm_is_moe_combine():
    """norm 0, no weight, scales 0 and 1: the bits of moe_combine."""
    b = Block(37, 8, 1032, 1, BF16)
    y, ref = (torch.empty((37, 1032), dtype=BF16, device="cuda") for _ in range(2))
    M.moe_combine(b.dD, dev(b.perm), dev(b.w), b.S, 37, 8, 1032, ref)
    M.moe_combine_norm(b.dD, dev(b.perm), dev(b.w), b.S, None, b.d_x, 0.0, 0, None, EPS, 1.0, 37, 8, 1032, y)
    assert torch.equal(y, ref)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("T,k,H,shared,norm", COMBINE)
def test_combine_norm_backward(T, k, H, shared, norm, dtype):
    b = Block(T, k, H, shared, dtype)
    R = T * (k + shared)
    dy, d_dy = stream(b.rng, (T, H), dtype, 0.02)
    ws_bytes = M.moe_combine_norm_backward_workspace_bytes(T, H)
    ws = torch.full((ws_bytes,), 0xFF, dtype=torch.uint8, device="cuda")
    for gated, weighted in ((0, 1), (shared, 0)):
        log(f"[combine norm backward] T={T} k={k} H={H} shared={shared} norm={norm} {dtype} gated={gated}")
        coded = H % 128 == 0
        dD = torch.full((R + 1, H), 5.0, dtype=BF16, device="cuda")
        dw = torch.full((T, k), float("nan"), device="cuda")
        dsw = torch.full((T,), float("nan"), device="cuda") if gated else None
        dweight = torch.full((H,), float("nan"), device="cuda")
        codes = torch.empty((R, H), dtype=torch.uint8, device="cuda") if coded else None
        scales = torch.empty((R, H // 128), device="cuda") if coded else None
        M.moe_combine_norm_backward(d_dy, dev(b.perm), dev(b.w), b.dD, shared, dev(b.sw) if gated else None, norm,
                                    dev(b.weight) if weighted else None, EPS, 2.0, T, k, H, dD, dw, dsw, codes, scales,
                                    dweight, ws, ws_bytes)
        rows, w = b.rows(gated)
        ref = ON.combine_norm_backward(dy, rows, w, norm, b.weight.astype(np.float64) if weighted else np.ones(H), EPS, 2.0)

        def layout(v):
            out = np.zeros((R, H))
            out[b.perm] = v[:, :k].reshape(T * k, H)
            if shared:
                out[T * k:] = v[:, k]
            return out
        want, err = (layout(v) for v in ref["rows"])
        check(bf16_values_host(dD)[:R], want, err, "dD")
        assert (bf16_values_host(dD)[R] == 5).all()
        dot, e = ref["w"]
        assert (np.abs(host(dw) - dot[:, :k]) <= e[:, :k] + U * np.abs(dot[:, :k])).all(), "d_topk_w"
        if gated:
            assert (np.abs(host(dsw) - dot[:, k]) <= e[:, k] + U * np.abs(dot[:, k])).all(), "d_shared_w"
        rw, ew = ref["weight"]
        assert (np.abs(host(dweight) - rw) <= ew + U * np.abs(rw)).all(), "d_weight"
        if coded:
            check_e4m3(codes, scales, want, err, "codes")


def test_indices_outside_the_rows():
    """They read the last routed row and are not written."""
    b = Block(6, 2, 256, 1, BF16)
    bad = b.perm.copy()
    bad[3], bad[8] = 12, -1
    y = torch.empty((6, 256), dtype=BF16, device="cuda")
    M.moe_combine_norm(b.dD, dev(bad), dev(b.w), b.S, None, b.d_x, 1.0, 1, dev(b.weight), EPS, 1.0, 6, 2, 256, y)
    clamped = bad.copy()
    clamped[[3, 8]] = 11
    rows, w = ON.gather(b.D, clamped, b.w.astype(np.float64), np.ones(6), 6, 2)
    ref, err, _ = ON.combine_norm(rows, w, b.x, 1.0, 1, b.weight.astype(np.float64), EPS, 1.0)
    check(get(y), ref, err, "y")
    dD = torch.full((18 + 4, 256), 5.0, dtype=BF16, device="cuda")
    dw = torch.empty((6, 2), device="cuda")
    dy = up(values(b.rng, (6, 256)))
    M.moe_combine_norm_backward(dy, dev(bad), dev(b.w), b.dD, 1, None, 1, None, EPS, 1.0, 6, 2, 256, dD, dw, None, None,
                                None, None, None, 0)
    got = bf16_values_host(dD)
    free = sorted(set(range(12)) - set(bad.tolist()))
    assert (got[free] == 5).all() and (got[18:] == 5).all() and np.isfinite(got).all()


def test_empty_batches():
    z = torch.empty((0, 64), dtype=BF16, device="cuda")
    e = torch.empty(0, device="cuda")
    i = torch.empty(0, dtype=torch.int32, device="cuda")
    dw = torch.full((64,), float("nan"), device="cuda")
    M.moe_norm(z, None, None, 0, 64, EPS, None, z)
    M.moe_norm_backward(z, z, None, e, None, 1.0, 0, 64, z, dw, None, 0)
    assert (host(dw) == 0).all()
    M.moe_combine_norm(z, i, e, None, None, z, 1.0, 1, None, EPS, 1.0, 0, 2, 64, z)
    dw.fill_(float("nan"))
    M.moe_combine_norm_backward(z, i, e, z, 0, None, 1, None, EPS, 1.0, 0, 2, 64, z, e, None, None, None, dw, None, 0)
    assert (host(dw) == 0).all()

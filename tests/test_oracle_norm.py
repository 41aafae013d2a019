"""The FP64 oracle of the norms around a block against plain loops and
differences (CPU)."""
import math

import numpy as np
import pytest

from oracle import norm as ON


def test_norm_hand_worked():
    v = np.array([[3.0, -4.0], [0.0, 0.0]])
    n, _, r, _ = ON.norm(v, np.array([1.0, 2.0]), 0.5)
    # mean square 12.5: rstd = 1 / sqrt(13); a row of zeros keeps 0
    np.testing.assert_allclose(n, [[3 / math.sqrt(13), -8 / math.sqrt(13)], [0, 0]], rtol=1e-15)
    np.testing.assert_allclose(r, [1 / math.sqrt(13), math.sqrt(2)], rtol=1e-15)


def test_norm_backward_against_differences():
    rng = np.random.default_rng(1)
    T, H, eps, h = 3, 5, 1e-3, 1e-6
    v, w, dn, res = (rng.standard_normal(s) for s in ((T, H), H, (T, H), (T, H)))
    r = ON.norm(v, w, eps)[2]
    dx, _, dw, _ = ON.norm_backward(dn, v, w, r, res, 0.7)
    loss = lambda v, w: (dn * ON.norm(v, w, eps)[0]).sum() + 0.7 * (res * v).sum()  # noqa: E731
    for t in range(T):
        for i in range(H):
            d = np.zeros((T, H))
            d[t, i] = h
            assert math.isclose(dx[t, i], (loss(v + d, w) - loss(v - d, w)) / (2 * h), rel_tol=1e-6, abs_tol=1e-8)
    for i in range(H):
        d = np.zeros(H)
        d[i] = h
        assert math.isclose(dw[i], (loss(v, w + d) - loss(v, w - d)) / (2 * h), rel_tol=1e-6, abs_tol=1e-8)


@pytest.mark.parametrize("use_norm", [0, 1])
def test_combine_against_loops_and_differences(use_norm):
    rng = np.random.default_rng(2)
    T, k, H, eps, scale, h = 3, 2, 4, 1e-3, 0.5, 1e-6
    D, w, sw = rng.standard_normal((T * k + T, H)), rng.random((T, k)), rng.random(T)
    perm, weight, x = rng.permutation(T * k), rng.standard_normal(H), rng.standard_normal((T, H))
    dy = rng.standard_normal((T, H))

    def y_of(D, w, sw, weight):
        out = np.zeros((T, H))
        for t in range(T):
            z = sum(w[t, j] * D[perm[t * k + j]] for j in range(k)) + sw[t] * D[T * k + t]
            if use_norm:
                z = z / math.sqrt((z ** 2).mean() + eps)
            out[t] = 2.0 * x[t] + scale * z * weight
        return out
    rows, ws = ON.gather(D, perm, w, sw, T, k)
    y, _, r = ON.combine_norm(rows, ws, x, 2.0, use_norm, weight, eps, scale)
    np.testing.assert_allclose(y, y_of(D, w, sw, weight), rtol=1e-12)
    assert (r is None) == (not use_norm)
    got = ON.combine_norm_backward(dy, rows, ws, use_norm, weight, eps, scale)
    loss = lambda *a: (dy * y_of(*a)).sum()  # noqa: E731
    args = [D, w, sw, weight]

    def diff(which, at):
        lo, hi = [v.copy() for v in args], [v.copy() for v in args]
        lo[which][at] -= h
        hi[which][at] += h
        return (loss(*hi) - loss(*lo)) / (2 * h)
    near = lambda a, b: math.isclose(a, b, rel_tol=1e-6, abs_tol=1e-8)  # noqa: E731
    for t in range(T):
        for j in range(k):
            assert near(got["w"][0][t, j], diff(1, (t, j)))
            for i in range(H):
                assert near(got["rows"][0][t, j, i], diff(0, (perm[t * k + j], i)))
        assert near(got["w"][0][t, k], diff(2, t))
        for i in range(H):
            assert near(got["rows"][0][t, k, i], diff(0, (T * k + t, i)))
    for i in range(H):
        assert near(got["weight"][0][i], diff(3, i))


def test_bounds_hold_for_fp32():
    """The bounds hold for a plain fp32 evaluation on the CPU."""
    rng = np.random.default_rng(4)
    T, H, eps = 6, 700, 1e-6
    f = np.float32
    v, w, dn = (rng.standard_normal(s).astype(f) for s in ((T, H), H, (T, H)))
    n, en, r, er = ON.norm(v.astype(float), w.astype(float), eps)
    r32 = f(1) / np.sqrt((v * v).mean(axis=1, dtype=f) + f(eps))
    assert (np.abs(r32 - r) <= er * r).all()
    assert (np.abs((v * r32[:, None]) * w - n) <= en).all()
    dx, ex, dw, ew = ON.norm_backward(dn.astype(float), v.astype(float), w.astype(float), r32.astype(float),
                                      np.zeros((T, H)), 1.0)
    hat, g = v * r32[:, None], dn * w
    got = r32[:, None] * (g - hat * (g * hat).mean(axis=1, dtype=f, keepdims=True))
    assert (np.abs(got - dx) <= ex).all() and (np.abs((dn * hat).sum(axis=0, dtype=f) - dw) <= ew).all()

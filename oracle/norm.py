"""The norms before and after a block and their gradients in FP64, with bounds
on an FP32 evaluation that sums in any order of at most `ADDS` additions one
after the other."""
import numpy as np

U = 2.0 ** -24
ADDS = 96


def _mean(v, e):
    """Row means of v whose values are off by e, and their bound."""
    n = v.shape[1]
    return v.sum(axis=1, keepdims=True) / n, (e + ADDS * U * np.abs(v)).sum(axis=1, keepdims=True) / n


def rstd(v, eps, e=0.0):
    """1 / sqrt(mean v^2 + eps) [T, 1] and its relative bound (v off by e)."""
    m, em = _mean(v * v, 2 * np.abs(v) * e + U * v * v)
    return 1 / np.sqrt(m + eps), em / (2 * (m + eps)) + 4 * U


def norm(v, weight, eps):
    """n [T, H], its bound, rstd [T] and its relative bound."""
    r, er = rstd(v, eps)
    n = v * r * weight
    return n, np.abs(n) * (er + 3 * U), r[:, 0], er[:, 0]


def norm_backward(dn, v, weight, r, d_res, res_scale):
    """dx, its bound, d_weight, its bound; r [T]: rstd as given."""
    r = r[:, None]
    hat, g = v * r, dn * weight
    mean, em = _mean(g * hat, 3 * U * np.abs(g * hat))
    core = r * (g - hat * mean)
    ec = r * (3 * U * np.abs(g) + np.abs(hat) * (em + 4 * U * np.abs(mean)))
    dx = core + res_scale * d_res
    e = ec + 3 * U * (np.abs(core) + np.abs(res_scale * d_res))
    T = v.shape[0]
    return dx, e, (dn * hat).sum(axis=0), (ADDS + T / 512 + 2) * U * np.abs(dn * hat).sum(axis=0)


def gather(D, inv_perm, w, shared_w, T, k):
    """The token's rows [T, k (+ 1), H] and their weights."""
    rows = D[inv_perm].reshape(T, k, -1)
    w = w.reshape(T, k)
    if shared_w is not None:
        rows = np.concatenate([rows, D[T * k:][:, None]], axis=1)
        w = np.concatenate([w, shared_w[:, None]], axis=1)
    return rows, w


def _sum(rows, w):
    p = rows * w[:, :, None]
    return p.sum(axis=1), (w.shape[1] + 1) * U * np.abs(p).sum(axis=1)


def combine_norm(rows, w, residual, residual_scale, use_norm, weight, eps, scale):
    """y, its bound, rstd and its relative bound (None without the norm)."""
    z, ez = _sum(rows, w)
    r, er = rstd(z, eps, ez) if use_norm else (np.ones((len(z), 1)), np.zeros((len(z), 1)))
    b = z * r * weight
    eb = np.abs(r * weight) * ez + np.abs(b) * (er + 3 * U)
    y = residual_scale * residual + scale * b
    e = abs(scale) * eb + 3 * U * (np.abs(residual_scale * residual) + np.abs(scale * b))
    return y, e, (r[:, 0], er[:, 0]) if use_norm else None


def combine_norm_backward(dy, rows, w, use_norm, weight, eps, scale):
    """Gradients and their bounds: rows [T, m, H], w [T, m], weight [H]."""
    z, ez = _sum(rows, w)
    g = scale * dy
    gw = g * weight
    if use_norm:
        r, er = rstd(z, eps, ez)
        hat = z * r
        eh = r * ez + np.abs(hat) * (er + 2 * U)
        mean, em = _mean(gw * hat, np.abs(gw) * eh + 4 * U * np.abs(gw * hat))
        em = em + np.abs(mean) * (er + 4 * U)
        core = gw - hat * mean
        dz = r * core
        e = r * (4 * U * np.abs(gw) + np.abs(hat) * em + np.abs(mean) * eh + 2 * U * np.abs(hat * mean)) \
            + np.abs(dz) * (er + 3 * U)
    else:
        hat, eh, dz, e = z, ez, gw, 3 * U * np.abs(gw)
    T = len(z)
    d_weight = (g * hat).sum(axis=0)
    ew = (np.abs(g) * eh + (ADDS + T / 512 + 3) * U * np.abs(g * hat)).sum(axis=0)
    dw = (rows * dz[:, None]).sum(axis=2)
    edw = (np.abs(rows) * (e + ADDS * U * np.abs(dz))[:, None]).sum(axis=2)
    spread = dz[:, None] * w[:, :, None]
    return dict(rows=(spread, np.abs(w[:, :, None]) * e[:, None] + 2 * U * np.abs(spread)), w=(dw, edw),
                weight=(d_weight, ew))

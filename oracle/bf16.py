"""Grouped products of unquantised matrices, the gated activations and their
backward, in FP64; the products also with bounds on an FP32 evaluation."""
import numpy as np

SILU, GELU = 0, 1
U = 2.0 ** -24      # FP32 unit roundoff


def _groups(offsets):
    for g in range(len(offsets) - 1):
        if offsets[g + 1] > offsets[g]:
            yield g, slice(int(offsets[g]), int(offsets[g + 1]))


def _sum(terms, a, b):
    """a @ b and a bound on its evaluation in FP32 in any order.  Each of its
    `terms` products may be cut to 24 bits below its largest neighbour, and each
    addition rounded or cut: 2^-23 of the products' sum each."""
    s = np.abs(a) @ np.abs(b)
    return a @ b, 2 * terms * 2 * U * s


def products(a, b, offsets, index=None):
    """C = A B^T of each group's rows: [R, N] and its bound."""
    R, N = int(offsets[-1]), b.shape[1]
    c, e = np.zeros((R, N)), np.zeros((R, N))
    for g, rows in _groups(offsets):
        src = a[rows] if index is None else a[index[rows]]
        c[rows], e[rows] = _sum(a.shape[1], src, b[g].T)
    return c, e


def dgrad(dc, w, offsets):
    """dA = dC W of each group's rows: [R, K] and its bound."""
    R, K = int(offsets[-1]), w.shape[2]
    c, e = np.zeros((R, K)), np.zeros((R, K))
    for g, rows in _groups(offsets):
        c[rows], e[rows] = _sum(w.shape[1], dc[rows], w[g])
    return c, e


def wgrad(dy, a, offsets, index=None):
    """dW_g = dY_g^T A_g: [G, N, K] and its bound."""
    G = len(offsets) - 1
    c = np.zeros((G, dy.shape[1], a.shape[1]))
    e = np.zeros_like(c)
    for g, rows in _groups(offsets):
        src = a[rows] if index is None else a[index[rows]]
        c[g], e[g] = _sum(src.shape[0], dy[rows].T, src)
    return c, e


def _logistic(z):
    t = np.exp(-np.abs(z))
    return np.where(z >= 0, 1 / (1 + t), t / (1 + t))


def activation(g, act):
    """act(g), its slope, and the argument z of its logistic function."""
    z, dz = g, np.ones_like(g)
    if act == GELU:
        r = 2 * np.sqrt(2 / np.pi)
        z, dz = r * (g + 0.044715 * g ** 3), r * (1 + 3 * 0.044715 * g ** 2)
    s, s1 = _logistic(z), _logistic(-z)
    return g * s, s + g * s * s1 * dz, z


def glu(gu, act):
    I = gu.shape[1] // 2
    return activation(gu[:, :I], act)[0] * gu[:, I:]


def glu_backward(gu, dh, act):
    """[dg | du] for the gradient dh of glu(gu)."""
    I = gu.shape[1] // 2
    a, slope, _ = activation(gu[:, :I], act)
    return np.concatenate([dh * gu[:, I:] * slope, dh * a], axis=1)

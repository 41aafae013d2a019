"""8-bit integer quantisation by rows and the grouped product with a scale for
each token and each output channel, in whole numbers and FP64."""
import numpy as np


def quant_rows(v):
    """v [..., K] fp32 values -> codes int8, scales fp32 (amax times the fp32
    1 / 127; 1 if that is 0).  The FP64 quotient of two fp32 numbers is never rounded onto or
    over a tie, so its rounding to a whole number is that of the exact one."""
    v = np.asarray(v, np.float32)
    s = np.abs(v).max(axis=-1) * (np.float32(1) / np.float32(127))
    s = np.where(s == 0, np.float32(1), s).astype(np.float32)
    q = np.rint(v.astype(np.float64) / s.astype(np.float64)[..., None])
    return np.clip(q, -127, 127).astype(np.int8), s


def products(a, sa, b, sb, offsets, index=None):
    """[offsets[-1], N] FP64 products of the groups' rows."""
    R, N = int(offsets[-1]), b.shape[1]
    out = np.zeros((R, N))
    for g in range(len(offsets) - 1):
        rows = np.arange(offsets[g], offsets[g + 1])
        src = rows if index is None else index[rows]
        # whole numbers below 2^53: exact in FP64 in any order
        acc = a[src].astype(np.float64) @ b[g].astype(np.float64).T
        out[rows] = acc * (sa[src].astype(np.float64)[:, None] * sb[g].astype(np.float64)[None, :])
    return out


def swiglu(p):
    """silu(gate) * up of products [R, 2I]."""
    I = p.shape[1] // 2
    g, u = p[:, :I], p[:, I:]
    z = np.exp(-np.abs(g))
    return g * np.where(g >= 0, 1.0 / (1.0 + z), z / (1.0 + z)) * u

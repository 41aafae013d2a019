"""The gate on given logits and its gradient, in FP64, token by token.

s = softmax or sigmoid of the logits; experts are ordered by s + bias (by the
logit itself without a bias), within the kept groups; ties go to the lower
index; a logit or bias of -inf excludes its expert (chosen only when nothing
else is left).  The formulas are those of include/moe_fp8.h, moe_gate.
"""
import numpy as np

SOFTMAX, SIGMOID = 0, 1


def gate_scores(logits, score):
    l = np.asarray(logits, np.float64)
    s = np.zeros_like(l)
    for t in range(l.shape[0]):
        there = l[t] > -np.inf
        if not there.any():
            continue
        if score == SOFTMAX:
            e = np.exp(l[t, there] - l[t, there].max())
            s[t, there] = e / e.sum()
        else:
            x = l[t, there]
            z = np.exp(-np.abs(x))
            s[t, there] = np.where(x >= 0, 1.0 / (1.0 + z), z / (1.0 + z))
    return s


def gate(logits, bias, score, n_group, topk_group, group_top, k, renormalize, scale):
    l = np.asarray(logits, np.float64)
    T, E = l.shape
    size = E // n_group
    s = gate_scores(l, score)
    b = np.zeros(E) if bias is None else np.asarray(bias, np.float64)
    excluded = ~(l > -np.inf) | ~(b > -np.inf)[None, :]
    with np.errstate(invalid="ignore"):
        v = l if bias is None else s + b
        pair = s + b
    idx = np.zeros((T, k), np.int32)
    w = np.zeros((T, k))
    for t in range(T):
        worth = []
        for g in range(n_group):
            of = v[t] if group_top == 1 else pair[t]
            members = sorted((of[e] for e in range(g * size, (g + 1) * size) if not excluded[t, e]),
                             reverse=True)
            worth.append(sum(members[:group_top]) if members else -np.inf)
        kept = sorted(range(n_group), key=lambda g: (-worth[g], g))[:topk_group]
        cand = [e for g in kept for e in range(g * size, (g + 1) * size)]
        cand.sort(key=lambda e: (excluded[t, e], 0.0 if excluded[t, e] else -v[t, e], e))
        idx[t] = sorted(cand[:k])
        w[t] = s[t, idx[t]]
        if renormalize:
            total = w[t].sum()
            w[t] = w[t] / total if total > 0 else 0.0
    counts = np.bincount(idx.ravel(), minlength=E).astype(np.int32)
    return dict(idx=idx, w=scale * w, counts=counts, scores=s)


def gate_backward(logits, score, renormalize, scale, idx, dw, ds=None):
    l = np.asarray(logits, np.float64)
    s = gate_scores(l, score)
    T, E = s.shape
    # sigmoid: 1 - s and s (1 - s) from exp(-|l|), as 1 - s itself has few bits
    # where s is near 1
    with np.errstate(invalid="ignore"):
        z = np.exp(-np.abs(l))
    rest = np.where(l >= 0, z, 1.0) / (1.0 + z)
    g = np.zeros((T, E)) if ds is None else np.array(ds, np.float64)
    extra = np.zeros((T, E))
    for t in range(T):
        named = [(int(e), scale * float(d)) for e, d in zip(idx[t], dw[t]) if 0 <= e < E]
        total = sum(s[t, e] for e, _ in named)
        mean = sum(d * (s[t, e] / total) for e, d in named) if total > 0 else 0.0
        for e, d in named:
            if not renormalize:
                g[t, e] += d
            elif total > 0:
                # ds_e (d - mean) / total, times s_e; its part of a softmax's
                # sum over the row is 0
                extra[t, e] += s[t, e] / total * (d - mean) * (1.0 if score == SOFTMAX else rest[t, e])
    if score == SIGMOID:
        return g * z / (1.0 + z) ** 2 + extra
    return s * (g - (g * s).sum(axis=1, keepdims=True)) + extra

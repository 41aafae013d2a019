"""moe_gate, moe_gate_backward, moe_router_logits and its backward against the
FP64 oracle: choices and counts exactly, weights and gradients within bounds
counted from the fp32 roundings."""
import numpy as np
import pytest
import torch

import fp8_block_scaled_bias_amd as M
from gpu_common import dev, host, log
from oracle import gate as OG

pytestmark = pytest.mark.gpu

U = 2.0 ** -24   # fp32 rounding: half a step, relative


def as_logits(l, kind):
    """Device logits of the type and the values they hold."""
    t = dev(np.asarray(l, np.float32))
    t = t if kind == "f32" else t.to(torch.bfloat16)
    return t, t.float().cpu().numpy().astype(np.float64)


def run_gate(logits, bias, score, n_group, topk_group, group_top, k, renorm, scale, scores=True,
             stream=None):
    T, E = logits.shape
    idx = torch.full((T, k), -7, dtype=torch.int32, device="cuda")
    w = torch.full((T, k), np.nan, dtype=torch.float32, device="cuda")
    counts = torch.full((E,), -7, dtype=torch.int32, device="cuda")
    s = torch.full((T, E), np.nan, dtype=torch.float32, device="cuda") if scores else None
    M.moe_gate(logits, T, E, None if bias is None else dev(np.asarray(bias, np.float32)), score, n_group,
               topk_group, group_top, k, renorm, scale, idx, w, counts, stream, scores=s)
    return host(idx), host(w), host(counts), None if s is None else host(s)


def score_bound(l, score):
    """Relative error of an fp32 score.  softmax: the difference to the
    largest logit is off by half a step, U * D, which exp turns into a
    relative error; exp itself 2 U, twice (element and sum), the sum's up to
    16 + 6 additions and the quotient.  sigmoid: exp 2 U plus one addition and
    the quotient."""
    if score == OG.SIGMOID:
        return 6 * U
    fin = np.where(np.isfinite(l), l, 0.0)
    D = float((fin.max(axis=1) - fin.min(axis=1)).max()) if l.size else 0.0
    return (2 * (min(D, 104.0) + 2) + 24) * U


def check(l_host, bias, got, args, label):
    score, n_group, topk_group, group_top, k, renorm, scale = args
    ref = OG.gate(l_host, bias, score, n_group, topk_group, group_top, k, renorm, scale)
    idx, w, counts, s = got
    assert np.array_equal(idx, ref["idx"]), f"{label}: choices differ at {np.argwhere(idx != ref['idx'])[:4]}"
    assert np.array_equal(counts, ref["counts"]), label
    tol = score_bound(l_host, score)
    tiny = 2.0 ** -125   # fp32 results below the normal range
    # the weight: the score, k - 1 additions, quotient and scale
    wt = (2 * tol + (k + 3) * U) if renorm else tol + U
    assert (np.abs(w - ref["w"]) <= wt * np.abs(ref["w"]) + tiny).all(), label
    if s is not None:
        assert (np.abs(s - ref["scores"]) <= tol * ref["scores"] + tiny).all(), label


SHAPES = [  # T, E, n_group, topk_group, group_top, k
    (1, 1, 1, 1, 1, 1), (1, 2, 2, 1, 2, 1), (5, 7, 7, 3, 2, 2), (3, 60, 1, 1, 1, 4), (64, 16, 4, 2, 2, 4),
    (65, 64, 8, 4, 2, 8), (257, 256, 8, 4, 2, 8), (130, 160, 8, 3, 1, 6), (77, 256, 1, 1, 1, 8),
    (33, 130, 5, 2, 2, 3), (19, 512, 16, 5, 2, 8), (9, 1000, 1, 1, 1, 7), (17, 1024, 32, 7, 2, 8),
]


@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "-".join(map(str, s)))
@pytest.mark.parametrize("score", [OG.SOFTMAX, OG.SIGMOID])
@pytest.mark.parametrize("kind", ["f32", "bf16"])
def test_gate(shape, score, kind):
    T, E, n_group, topk_group, group_top, k = shape
    rng = np.random.default_rng([T, E, score])
    logits, lh = as_logits(rng.standard_normal((T, E)) * 1.7, kind)
    for bias in (None, (rng.uniform(-1, 1, E) * (0.01 if score else 0.5 / E)).astype(np.float32)):
        for renorm, scale in ((1, 1.0), (0, 2.5)):
            log(f"[gate] {shape} score={score} {kind} bias={bias is not None} renorm={renorm}")
            args = (score, n_group, topk_group, group_top, k, renorm, scale)
            got = run_gate(logits, bias, *args)
            check(lh, bias, got, args, str(args))


@pytest.mark.parametrize("E,n_group", [(256, 8), (160, 8), (60, 1), (1024, 4)])
def test_gate_ties_and_exclusions(E, n_group):
    """Few distinct values (ties inside and across groups), -inf and the
    type's lowest value in rows, rows of nothing else."""
    rng = np.random.default_rng(E)
    T = 40
    l = rng.integers(-2, 3, (T, E)).astype(np.float32)
    l[5:15][rng.random((10, E)) < 0.9] = -np.inf
    l[15] = -np.inf
    l[16, 1:] = -np.inf
    l[17] = -3.4e38
    l[18, ::2] = -3.4e38
    l[19] = 0.0
    l[20, : E // 2] = -np.inf
    l[21, ::2] = -0.0
    zero = np.zeros(E, np.float32)
    some = zero.copy()
    some[rng.random(E) < 0.3] = -np.inf
    for kind in ("f32", "bf16"):
        logits, lh = as_logits(l, kind)
        for score in (OG.SOFTMAX, OG.SIGMOID):
            for bias in (None, zero, some):
                for top in (1, 2):
                    args = (score, n_group, max(1, n_group // 2), top, 6, 1, 1.0)
                    log(f"[gate ties] E={E} {kind} score={score} bias={bias is not None} top={top}")
                    check(lh, bias, run_gate(logits, bias, *args), args, f"{kind} {args}")


@pytest.mark.parametrize("E", [32, 256])
@pytest.mark.parametrize("score", [OG.SOFTMAX, OG.SIGMOID])
def test_gate_order_below_fp32(score, E):
    """Biases that make every score + bias the same up to an fp32 rounding:
    the order is that of the exact sums."""
    rng = np.random.default_rng(E + score)
    for trial in range(12):
        l = (rng.standard_normal((1, E)) * 1.5).astype(np.float32)
        s = OG.gate_scores(l, score)
        bias = (0.9 - s[0]).astype(np.float32)
        logits, lh = as_logits(np.repeat(l, 3, axis=0), "f32")
        for n_group, topk, top in ((1, 1, 1), (8, 3, 2)):
            args = (score, n_group, topk, top, 6, 0, 1.0)
            check(lh, bias, run_gate(logits, bias, *args), args, f"trial {trial} {args}")


def test_gate_unspecified_rows_stay_in_range():
    """NaN and +inf logits: the ids are still k different experts."""
    E, k = 64, 8
    l = np.random.default_rng(0).standard_normal((6, E)).astype(np.float32)
    l[0] = np.nan
    l[1, ::3] = np.nan
    l[2, 5] = np.inf
    l[3] = np.inf
    l[4, 0] = -np.inf
    logits, _ = as_logits(l, "f32")
    for score in (OG.SOFTMAX, OG.SIGMOID):
        for bias in (None, np.zeros(E, np.float32)):
            for n_group in (1, 8):
                idx, _, counts, _ = run_gate(logits, bias, score, n_group, max(1, n_group // 2), 2, k, 1, 1.0)
                assert (idx >= 0).all() and (idx < E).all() and (np.diff(idx, axis=1) > 0).all()
                assert counts.sum() == 6 * k


def test_gate_large_batch_and_empty():
    T, E, k = 16384, 256, 8
    rng = np.random.default_rng(3)
    l = rng.standard_normal((T, E)).astype(np.float32) * 1.7
    logits, lh = as_logits(l, "f32")
    bias = rng.uniform(-0.01, 0.01, E).astype(np.float32)
    log("[gate] T=16384")
    args = (OG.SIGMOID, 8, 4, 2, k, 1, 2.5)
    idx, w, counts, _ = run_gate(logits, bias, *args, scores=False)
    part = np.arange(0, T, 37)
    ref = OG.gate(lh[part], bias, *args)
    assert np.array_equal(idx[part], ref["idx"])
    assert np.array_equal(counts, np.bincount(idx.ravel(), minlength=E))
    idx2, w2, counts2, _ = run_gate(logits, bias, *args, scores=False)
    assert np.array_equal(idx, idx2) and np.array_equal(w, w2) and np.array_equal(counts, counts2)
    _, _, counts, _ = run_gate(logits[:0], bias, *args)
    assert (counts == 0).all()


def test_gate_more_tokens_than_a_grid_holds():
    """A workgroup takes several rounds of tokens, some of which need the order
    of 64 bits (equal scores + bias at the border) in each."""
    T, E, k = 70001, 64, 6
    rng = np.random.default_rng(8)
    l = rng.standard_normal((T, E)).astype(np.float32)
    l[::5] = np.round(l[::5] * 2) / 2
    logits, lh = as_logits(l, "f32")
    bias = np.zeros(E, np.float32)
    log("[gate] T=70001")
    args = (OG.SOFTMAX, 8, 4, 2, k, 1, 1.0)
    got = run_gate(logits, bias, *args)
    assert np.array_equal(got[2], np.bincount(got[0].ravel(), minlength=E))
    part = np.unique(np.concatenate([np.arange(0, T, 41), np.arange(65520, 65560), np.arange(T - 20, T)]))
    ref = OG.gate(lh[part], bias, *args)
    assert np.array_equal(got[0][part], ref["idx"])
    # weights: as in check()
    tol = 2 * score_bound(lh, OG.SOFTMAX) + (k + 3) * U
    assert (np.abs(got[1][part] - ref["w"]) <= tol * ref["w"]).all()


def run_backward(logits, score, k, renorm, scale, idx, dw, ds):
    T, E = logits.shape
    dl = torch.full((T, E), np.nan, dtype=logits.dtype, device="cuda")
    M.moe_gate_backward(logits, T, E, score, k, renorm, scale, dev(idx.astype(np.int32)),
                        dev(dw.astype(np.float32)), dl,
                        d_scores=None if ds is None else dev(ds.astype(np.float32)))
    return host(dl.float()).astype(np.float64)


def backward_bound(lh, score, renorm, scale, idx, dw, ds, kind):
    """Per element: every ds is a few products and sums of the scores (each
    off by score_bound) and of dw; the sums over the row have up to 16 + 6
    additions of terms that do not cancel in their error."""
    s = OG.gate_scores(lh, score)
    T, E = s.shape
    mag = np.zeros((T, E)) if ds is None else np.abs(ds)
    for t in range(T):
        named = [(int(e), abs(scale * d)) for e, d in zip(idx[t], dw[t]) if 0 <= e < E]
        total = sum(s[t, e] for e, _ in named)
        mean = sum(d * s[t, e] for e, d in named) / total if total > 0 else 0.0
        for e, d in named:
            mag[t, e] += d if not renorm else (d + mean) / total if total > 0 else 0.0
    rel = 4 * score_bound(lh, score) + 40 * U
    if score == OG.SIGMOID:
        size = mag * s   # 1 - s is off by U, not by a part of itself
    else:
        size = s * (mag + (mag * s).sum(axis=1, keepdims=True))
    return rel * size + 2.0 ** -125


@pytest.mark.parametrize("shape", [(1, 1, 1), (1, 2, 2), (3, 60, 4), (70, 64, 8), (65, 256, 8), (31, 160, 6),
                                   (33, 130, 3), (5, 512, 8), (6, 1000, 7), (4, 1024, 8)])
@pytest.mark.parametrize("score", [OG.SOFTMAX, OG.SIGMOID])
@pytest.mark.parametrize("kind", ["f32", "bf16"])
def test_gate_backward(shape, score, kind):
    T, E, k = shape
    rng = np.random.default_rng([T, E, score])
    logits, lh = as_logits(rng.standard_normal((T, E)) * 1.7, kind)
    idx = np.stack([np.sort(rng.choice(E, k, replace=False)) for _ in range(T)])
    dw = rng.standard_normal((T, k)).astype(np.float32)
    for renorm in (0, 1):
        for ds in (None, (rng.standard_normal((T, E)) * 0.1).astype(np.float32)):
            log(f"[gate backward] {shape} score={score} {kind} renorm={renorm}")
            got = run_backward(logits, score, k, renorm, 1.5, idx, dw, ds)
            ref = OG.gate_backward(lh, score, renorm, 1.5, idx, dw, ds)
            tol = backward_bound(lh, score, renorm, 1.5, idx, dw, ds, kind)
            if kind == "bf16":
                tol = tol * (1 + 2.0 ** -8) + 2.0 ** -8 * np.abs(ref) + 2.0 ** -133
            assert (np.abs(got - ref) <= tol).all(), np.abs(got - ref).max()


def test_gate_backward_odd_rows():
    """Ids out of range, ids named twice, -inf logits, a row of nothing else."""
    rng = np.random.default_rng(8)
    T, E, k = 6, 96, 4
    l = rng.standard_normal((T, E)).astype(np.float32)
    l[1, 10:] = -np.inf
    l[2] = -np.inf
    logits, lh = as_logits(l, "f32")
    idx = np.stack([np.sort(rng.choice(E, k, replace=False)) for _ in range(T)])
    idx[0] = [-1, 3, 3, E]
    idx[1] = [0, 1, 50, 60]
    idx[3] = [-5, E, E + 7, 2 ** 31 - 1]
    dw = rng.standard_normal((T, k)).astype(np.float32)
    for score in (OG.SOFTMAX, OG.SIGMOID):
        for renorm in (0, 1):
            got = run_backward(logits, score, k, renorm, 2.0, idx, dw, None)
            ref = OG.gate_backward(lh, score, renorm, 2.0, idx, dw, None)
            assert (np.abs(got - ref) <= backward_bound(lh, score, renorm, 2.0, idx, dw, None, "f32")).all()
            assert (got[2] == 0).all() and (got[3] == 0).all()


def test_gate_backward_against_differences():
    """The GPU gradient against differences of the GPU's own weights."""
    rng = np.random.default_rng(4)
    T, E, k = 4, 32, 3
    l = rng.standard_normal((T, E)).astype(np.float32)
    # clear margins, so that a step of 2^-6 does not change the choice
    top = np.argsort(-l, axis=1)[:, :k]
    np.put_along_axis(l, top, np.take_along_axis(l, top, 1) + 2, axis=1)
    dw = rng.standard_normal((T, k))
    for score in (OG.SOFTMAX, OG.SIGMOID):
        for renorm in (0, 1):
            args = (score, 1, 1, 1, k, renorm, 1.0)
            idx, _, _, _ = run_gate(dev(l), None, *args)
            g = run_backward(dev(l), score, k, renorm, 1.0, idx, dw, None)
            h = 2.0 ** -6
            step = rng.choice([-1.0, 1.0], (T, E)).astype(np.float32)
            ip, wp, _, _ = run_gate(dev(l + h * step.astype(np.float32)), None, *args)
            im, wm, _, _ = run_gate(dev(l - h * step.astype(np.float32)), None, *args)
            assert np.array_equal(ip, idx) and np.array_equal(im, idx)
            got = ((wp.astype(np.float64) - wm) * dw).sum(axis=1) / (2 * h)
            # each weight is off by under 2^-18 (fp32); the third derivative of
            # a score along a step of all +-1 is at most 8, of a ratio 64
            tol = np.abs(dw).sum(axis=1) * (2.0 ** -18 / h + 64 * h * h / 6)
            assert (np.abs(got - (g * step).sum(axis=1)) <= tol).all()


@pytest.mark.parametrize("T,H,E", [(3, 256, 16), (200, 1024, 64), (2100, 512, 160), (130, 256, 512)])
def test_router_logits_and_backward(T, H, E):
    rng = np.random.default_rng([T, E])
    x = dev(rng.standard_normal((T, H)).astype(np.float32)).to(torch.bfloat16)
    C = (rng.standard_normal((E, H)) * 0.05).astype(np.float32)
    xh = x.float().cpu().numpy().astype(np.float64)
    wsb = max(16, M.moe_route_workspace_bytes(T, H, E))
    ws = torch.empty(wsb, dtype=torch.uint8, device="cuda")
    logits = torch.full((T, E), np.nan, device="cuda")
    M.moe_router_logits(x, T, H, dev(C), E, logits, ws, wsb)
    got, ref = host(logits), xh @ C.astype(np.float64).T
    size = np.abs(xh) @ np.abs(C.astype(np.float64)).T
    # exact products; at most 3 H additions, each off by U of a partial sum
    # no larger than the sum of the sizes (64 counts their usual growth)
    assert (np.abs(got - ref) <= 64 * U * size).all()
    dl = rng.standard_normal((T, E)).astype(np.float32)
    dxin = dev(rng.standard_normal((T, H)).astype(np.float32)).to(torch.bfloat16)
    wsb = max(16, M.moe_router_backward_dense_workspace_bytes(T, H, E))
    ws = torch.empty(wsb, dtype=torch.uint8, device="cuda")
    for given in (None, dxin):
        dx = torch.empty((T, H), dtype=torch.bfloat16, device="cuda")
        dC = torch.full((E, H), np.nan, device="cuda")
        M.moe_router_logits_backward(x, dev(C), dev(dl), T, H, E, given, dx, dC, ws, wsb)
        d64, base = dl.astype(np.float64), 0 if given is None else host(given.float()).astype(np.float64)
        rx, rC = base + d64 @ C, d64.T @ xh
        bx = (E + 2) * U * (np.abs(base) + np.abs(d64) @ np.abs(C))
        assert (np.abs(host(dx.float()) - rx) <= 2.0 ** -8 * np.abs(rx) + 1.01 * bx).all()
        assert (np.abs(host(dC) - rC) <= (T + 2) * U * (np.abs(d64).T @ np.abs(xh))).all()
    M.moe_router_logits_backward(x[:0], dev(C), dev(dl)[:0], 0, H, E, None, x[:0], dC, ws, wsb)
    assert (host(dC) == 0).all()


def test_gate_graph_replays_on_its_stream():
    """Forward and backward captured together, replayed between eager calls."""
    T, E, k = 300, 128, 6
    rng = np.random.default_rng(6)
    logits = dev(rng.standard_normal((T, E)).astype(np.float32))
    args = (OG.SOFTMAX, 1, 1, 1, k, 1, 1.0)
    idx = torch.empty((T, k), dtype=torch.int32, device="cuda")
    w, counts = torch.empty((T, k), device="cuda"), torch.empty(E, dtype=torch.int32, device="cuda")
    dw, dl = dev(rng.standard_normal((T, k)).astype(np.float32)), torch.empty((T, E), device="cuda")

    def both():
        M.moe_gate(logits, T, E, None, *args[:5], 1, 1.0, idx, w, counts)
        M.moe_gate_backward(logits, T, E, OG.SOFTMAX, k, 1, 1.0, idx, dw, dl)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        both()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        both()
    for rep in range(3):
        l = rng.standard_normal((T, E)).astype(np.float32)
        logits.copy_(dev(l))
        graph.replay()
        torch.cuda.synchronize()
        got = [host(t).copy() for t in (idx, w, counts, dl)]
        both()
        for a, b in zip(got, (idx, w, counts, dl)):
            assert np.array_equal(a, host(b)), rep
        check(l.astype(np.float64), None, (got[0], got[1], got[2], None), args, f"replay {rep}")

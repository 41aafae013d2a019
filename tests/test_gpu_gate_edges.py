"""moe_gate and moe_gate_backward where fp32 comes to its limits: large biases that
cancel in a group's sum, scores below fp32's range, saturated scores."""
import numpy as np
import pytest
import torch

import fp8_block_scaled_bias_amd as M
from gpu_common import dev, host, log
from oracle import gate as OG
from test_gpu_gate import run_backward, run_gate

pytestmark = pytest.mark.gpu

U = 2.0 ** -24   # fp32 rounding: half a step, relative


@pytest.mark.parametrize("size", [64.0, 1024.0, 65536.0])
@pytest.mark.parametrize("E,n_group", [(16, 8), (64, 8), (40, 10), (512, 32)])
@pytest.mark.parametrize("score", [OG.SOFTMAX, OG.SIGMOID])
def test_biases_that_cancel_in_a_group(score, E, n_group, size):
    """A group's two best have biases of opposite sign: their sum is small, its
    rounding errors are those of the large ones.  The scores differ so little
    that sums in fp32 would order the groups wrongly."""
    T, k, per = 1500, min(8, n_group // 2), E // n_group
    rng = np.random.default_rng([E, int(size), score])
    spread = 4 * size * 2.0 ** -23          # of the scores: a few steps of fp32 at `size`
    slope = 0.25 if score == OG.SIGMOID else 1.0 / E
    l = (rng.standard_normal((T, E)) * min(1.0, spread / slope)).astype(np.float32)
    bias = np.full((n_group, per), -2 * size, np.float32)
    bias[:, 0], bias[:, 1] = size, -size
    args = (score, n_group, k, 2, k, 0, 1.0)
    ref = OG.gate(l, bias.ravel(), *args)
    log(f"[gate cancel] E={E} groups={n_group} size={size} score={score}")
    idx, _, counts, _ = run_gate(dev(l), bias.ravel(), *args, scores=False)
    wrong = (idx != ref["idx"]).any(axis=1)
    assert not wrong.any(), f"{wrong.sum()} of {T} tokens"
    assert np.array_equal(counts, ref["counts"])


def test_infinite_biases():
    """Biases of +inf, -inf and the type's largest values: k different ids."""
    E, k = 64, 8
    l = np.random.default_rng(0).standard_normal((40, E)).astype(np.float32)
    for bias in ([np.inf] * 3 + [0] * 61, [np.inf, -np.inf] * 32, [3.4e38, -3.4e38] * 32, [3.4e38] * 64):
        for n_group, top in ((1, 1), (8, 1), (8, 2)):
            for score in (OG.SOFTMAX, OG.SIGMOID):
                idx, _, counts, _ = run_gate(dev(l), np.array(bias, np.float32), score, n_group,
                                             max(1, n_group // 2), top, k, 1, 1.0)
                assert (idx >= 0).all() and (idx < E).all() and (np.diff(idx, axis=1) > 0).all()
                assert counts.sum() == 40 * k


def test_sigmoid_gradient_of_saturated_scores():
    """s (1 - s) where s is near 1 or near 0, to a few roundings of itself."""
    E, k = 96, 4
    l = np.concatenate([np.linspace(-86, 86, E), [0.0] * E, np.tile([10, -10, 20, -20, 40, -40], 16),
                        np.linspace(12, 20, E)]).reshape(4, E).astype(np.float32)
    rng = np.random.default_rng(1)
    idx = np.stack([np.sort(rng.choice(E, k, replace=False)) for _ in range(4)])
    dw, ds = rng.standard_normal((4, k)).astype(np.float32), rng.standard_normal((4, E)).astype(np.float32)
    for given in (None, ds):
        got = run_backward(dev(l), OG.SIGMOID, k, 0, 1.5, idx, dw, given)
        ref = OG.gate_backward(l, OG.SIGMOID, 0, 1.5, idx, dw, given)
        # the slope: exp 2, 1 + z, its reciprocal 1.5, both twice, two products:
        # 9; then scale * dw 1 and the product 1, relative.  ds + scale * dw:
        # one more, of the sum's parts, which may cancel
        z = np.exp(-np.abs(l.astype(np.float64)))
        part = np.zeros((4, E)) if given is None else np.abs(given).astype(np.float64)
        for t in range(4):
            part[t, idx[t]] += 1.5 * np.abs(dw[t])
        assert (np.abs(got - ref) <= U * (11 * np.abs(ref) + 2 * part * z / (1 + z) ** 2) + 2.0 ** -149).all()


LOWS = (-60.0, -86.0, -88.0, -95.0, -100.0, -110.0, -150.0)


def low_choices(score, k, E=64):
    """Rows whose k chosen logits lie far below zero (and below the row's
    largest): their scores are subnormal or 0 in fp32.  Chosen: ids 3, 10, ..."""
    rng = np.random.default_rng(k)
    l = rng.standard_normal((7, E)).astype(np.float32)
    chosen = 3 + 7 * np.arange(k)
    for t, low in enumerate(LOWS):
        l[t, chosen] = low - np.arange(k) * 0.75
    l[1, chosen[0]] = -60.0   # a spread of 26 to 31 between the choices
    return l, np.tile(chosen, (7, 1))


def nothing(l, idx, score):
    """Rows whose chosen scores have to count as 0 in fp32, and those where they
    may: under half of 2^-149 and, for a softmax, under 2^-126."""
    most = np.take_along_axis(OG.gate_scores(l, score), idx, 1).max(axis=1)
    return most < 0.99 * 2.0 ** -150, most < (1.01 * 2.0 ** -126 if score == OG.SOFTMAX else 2.0 ** -148)


def share_bound(l, idx, score):
    """Relative error of s_j / S.  exp(l - m) by exp2: (2.2 |l - m| + 2) roundings
    (the difference, its product with log2 e and that constant, each a part of
    |l - m|; exp2 itself).  Scores of a sum above 2^-64 are those of the row
    (m its largest logit) or sigmoids (6 roundings at any logit), others are
    relative to the largest choice.  The error of a score and of the sum, k - 1
    additions (three rounds of them, at most 8), 1 / sum and the quotient."""
    c = np.take_along_axis(l, idx, 1).astype(np.float64)
    low = np.take_along_axis(OG.gate_scores(l, score), idx, 1).sum(axis=1) < 1.001 * 2.0 ** -64
    normal = 6.0 if score == OG.SIGMOID else 2.2 * (l.max(axis=1) - c.min(axis=1)) + 2
    each = np.where(low, 2.2 * (c.max(axis=1) - c.min(axis=1)) + 2, normal)
    return (2 * each + 11)[:, None] * U


@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("k", [1, 2, 8])
@pytest.mark.parametrize("score", [OG.SOFTMAX, OG.SIGMOID])
def test_renormalised_gradient_of_scores_below_fp32(score, k, kind):
    l, idx = low_choices(score, k)
    logits = dev(l) if kind == "f32" else dev(l).to(torch.bfloat16)
    l = host(logits.float())
    rng = np.random.default_rng(2)
    dw = rng.standard_normal((7, k)).astype(np.float32)
    ds = rng.standard_normal((7, l.shape[1])).astype(np.float32)
    for given in (None, ds):
        got = run_backward(logits, score, k, 1, 1.5, idx, dw, given)
        ref = OG.gate_backward(l, score, 1, 1.5, idx, dw, given)
        assert np.isfinite(got).all()
        # p_j (dw_j - mean): the shares' errors in it and in the mean, and five
        # roundings (scale * dw, the product and sum of the mean, difference,
        # product), times 1 - s_j (6 roundings)
        p = np.exp(np.take_along_axis(l, idx, 1).astype(np.float64))
        p /= p.sum(axis=1, keepdims=True)     # all far below 0: s = exp(l)
        a = 1.5 * np.abs(dw)
        part = np.zeros(l.shape)
        np.put_along_axis(part, idx, p * (a + (a * p).sum(axis=1, keepdims=True)), axis=1)
        tol = (3 * share_bound(l, idx, score) + 14 * U) * part + 2.0 ** -149
        if given is not None:
            # s (ds - sum ds s) of logits within 5 of the largest or under
            # e^-60: 2 |l - m| + 2 roundings of exp, 10 of the sum, quotient
            s = OG.gate_scores(l, score)
            size = s * (np.abs(ds) + (s * np.abs(ds)).sum(axis=1, keepdims=True))
            tol = tol + 80 * U * size + 2.0 ** -125
        if kind == "bf16":
            tol = tol * (1 + 2.0 ** -8) + 2.0 ** -8 * np.abs(ref) + 2.0 ** -134
        # without the choices' part
        rest = ref - OG.gate_backward(l, score, 1, 1.5, idx, dw, None)
        must, may = nothing(l, idx, score)
        ok = (np.abs(got - ref) <= tol).all(axis=1)
        empty = (np.abs(got - rest) <= tol).all(axis=1)
        assert np.where(must, empty, ok | (may & empty)).all(), (ok, empty, must, may)


@pytest.mark.parametrize("k", [1, 2, 8])
@pytest.mark.parametrize("score", [OG.SOFTMAX, OG.SIGMOID])
@pytest.mark.parametrize("tie", [False, True])
def test_renormalised_weights_of_scores_below_fp32(score, k, tie):
    """A bias chooses experts whose scores are subnormal or 0 in fp32: the weights
    are still their shares.  tie: one more expert ties at the border, so that the
    order is looked at in 64 bits."""
    l, idx = low_choices(score, k)
    bias = np.zeros(l.shape[1], np.float32)
    bias[idx[0]] = 4.0
    if tie:
        bias[-1] = 4.0
        l[:, -1] = -170.0
    args = (score, 1, 1, 1, k, 1, 1.5)
    ref = OG.gate(l, bias, *args)
    assert np.array_equal(ref["idx"], idx)
    got, w, counts, _ = run_gate(dev(l), bias, *args)
    assert np.array_equal(got, idx) and np.array_equal(counts, ref["counts"])
    must, may = nothing(l, idx, score)
    ok = (np.abs(w - ref["w"]) <= (share_bound(l, idx, score) + 2 * U) * ref["w"] + 2.0 ** -149).all(axis=1)
    empty = (w == 0).all(axis=1)
    assert np.where(must, empty, ok | (may & empty)).all(), (ok, empty, must, may)
    # every logit -inf: weights 0
    _, w, _, _ = run_gate(dev(np.full_like(l, -np.inf)), bias, *args)
    assert (w == 0).all()


def test_more_tokens_than_one_launch_holds():
    """Two experts, 2^28 + 77 tokens: sixteen threads a token are more than 2^32."""
    T, E = (1 << 28) + 77, 2
    log(f"[gate] T={T}")
    logits = torch.empty((T, E), dtype=torch.bfloat16, device="cuda")
    logits.normal_(generator=torch.Generator(device="cuda").manual_seed(3))
    idx = torch.full((T, 1), -7, dtype=torch.int32, device="cuda")
    w = torch.full((T, 1), np.nan, device="cuda")
    counts = torch.empty(E, dtype=torch.int32, device="cuda")
    M.moe_gate(logits, T, E, None, OG.SOFTMAX, 1, 1, 1, 1, 0, 1.0, idx, w, counts)
    dl = torch.full((T, E), np.nan, dtype=torch.bfloat16, device="cuda")
    M.moe_gate_backward(logits, T, E, OG.SOFTMAX, 1, 0, 1.0, idx, w, dl)
    torch.cuda.synchronize()
    assert int(counts.sum()) == T
    first = (logits[:, :1] >= logits[:, 1:]).to(torch.int32)   # a tie goes to the lower index
    assert torch.equal(idx, 1 - first)
    del first
    rows = np.unique(np.concatenate([np.arange(0, T, T // 997), np.arange(2 ** 25 - 3, 2 ** 25 + 3),
                                     np.arange(2 ** 28 - 3, 2 ** 28 + 3), np.arange(T - 40, T)]))
    at = torch.from_numpy(rows).cuda()
    l = host(logits[at].float())
    ref = OG.gate(l, None, OG.SOFTMAX, 1, 1, 1, 1, 0, 1.0)
    assert np.array_equal(host(idx[at]), ref["idx"])
    # exp, sum, quotient, product of logits within 12 of each other
    assert (np.abs(host(w[at]) - ref["w"]) <= 40 * U * ref["w"]).all()
    want = OG.gate_backward(l, OG.SOFTMAX, 0, 1.0, ref["idx"], host(w[at]))
    # w s (1 - s): w off by its bound, the difference by the parts' roundings
    assert (np.abs(host(dl[at].float()) - want) <= 2.0 ** -8 * np.abs(want) + 200 * U).all()
    assert bool(torch.isfinite(dl).all())


@pytest.mark.parametrize("score", [OG.SOFTMAX, OG.SIGMOID])
def test_weights_and_gradient_are_0_in_the_same_rows(score):
    """Whether every chosen score is 0 in fp32 does not depend on how the order was
    found, and the gradient takes the rows whose weights are 0 as such."""
    k, E = 4, 64
    l, idx = low_choices(score, k)
    l = np.concatenate([l, l[:1], l[:1], l[:1]])
    idx = np.concatenate([idx, idx[:3]])
    l[7:10, idx[0]] = np.array([-84.5, -91.0, -104.5])[:, None]
    plain, tied = np.zeros(E, np.float32), np.zeros(E, np.float32)
    plain[idx[0]] = tied[idx[0]] = tied[-1] = 4.0
    l[:, -1] = -170.0
    empty = []
    for bias in (plain, tied):
        got, w, _, _ = run_gate(dev(l), bias, score, 1, 1, 1, k, 1, 1.0)
        assert np.array_equal(got, idx)
        empty.append((w == 0).all(axis=1))
    assert np.array_equal(empty[0], empty[1]), empty
    dw = np.arange(1, 4 * len(l) + 1, dtype=np.float32).reshape(-1, 4) ** 2
    dl = run_backward(dev(l), score, k, 1, 1.0, idx, dw, None)
    assert np.array_equal((np.take_along_axis(dl, idx, 1) == 0).all(axis=1), empty[0]), empty

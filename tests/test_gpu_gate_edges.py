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

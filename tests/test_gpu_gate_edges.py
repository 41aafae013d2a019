"""moe_gate and moe_gate_backward where fp32 comes to its limits: large biases that
cancel in a group's sum, scores below fp32's range, saturated scores."""
import numpy as np
import pytest
import torch

import fp8_block_scaled_bias_amd as M
from gpu_common import dev, host, log
from oracle import gate as OG
from test_gpu_gate import run_gate

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

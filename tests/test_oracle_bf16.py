"""The FP64 oracle of the bf16 experts against plain loops and differences (CPU)."""
import math

import numpy as np
import pytest
import torch

from oracle import bf16 as OB


def test_products_against_loops():
    rng = np.random.default_rng(3)
    offs, K, N = np.array([0, 2, 2, 5]), 4, 3
    a, b = rng.integers(-4, 5, (6, K)).astype(float), rng.integers(-4, 5, (3, N, K)).astype(float)
    idx = np.array([5, 0, 1, 1, 4])
    for index in (None, idx):
        c, e = OB.products(a, b, offs, index)
        for r in range(5):
            g = 0 if r < 2 else 2
            src = r if index is None else index[r]
            for n in range(N):
                assert c[r, n] == sum(a[src, k] * b[g, n, k] for k in range(K))
                assert e[r, n] == 2 ** -22 * K * sum(abs(a[src, k] * b[g, n, k]) for k in range(K))
    dc = rng.integers(-4, 5, (5, N)).astype(float)
    d, _ = OB.dgrad(dc, b, offs)
    w, _ = OB.wgrad(dc, a, offs, idx)
    assert (w[1] == 0).all()
    # both are the derivatives of <dC, C>
    h = 0.5   # the product is linear: any step is exact
    for r, k in ((0, 1), (4, 3)):
        a2 = a[idx].copy()
        a2[r, k] += h
        diff = (dc * (OB.products(a2, b, offs)[0] - OB.products(a[idx], b, offs)[0])).sum() / h
        assert diff == d[r, k]
    for g, n, k in ((0, 2, 1), (2, 0, 3)):
        b2 = b.copy()
        b2[g, n, k] += h
        diff = (dc * (OB.products(a, b2, offs, idx)[0] - OB.products(a, b, offs, idx)[0])).sum() / h
        assert diff == w[g, n, k]


@pytest.mark.parametrize("act", [OB.SILU, OB.GELU])
def test_activation(act):
    g = np.concatenate([np.linspace(-12, 12, 97), [0.0]])
    a, slope, _ = OB.activation(g, act)
    t = torch.from_numpy(g)
    ref = torch.nn.functional.silu(t) if act == OB.SILU else torch.nn.functional.gelu(t, approximate="tanh")
    np.testing.assert_allclose(a, ref.numpy(), rtol=1e-10, atol=1e-14)
    h = 1e-6
    diff = (OB.activation(g + h, act)[0] - OB.activation(g - h, act)[0]) / (2 * h)
    np.testing.assert_allclose(slope, diff, rtol=1e-6, atol=1e-8)
    assert a[-1] == 0 and slope[-1] == 0.5
    big, s, _ = OB.activation(np.array([-1e4, 1e4]), act)
    assert big[0] == 0 and s[0] == 0 and big[1] == 1e4 and s[1] == 1


def test_gelu_known_value():
    # 0.5 * (1 + tanh(sqrt(2 / pi) * 1.044715)) at g = 1
    assert math.isclose(float(OB.activation(np.array([1.0]), OB.GELU)[0][0]),
                        0.5 * (1 + math.tanh(math.sqrt(2 / math.pi) * 1.044715)), rel_tol=1e-14)


@pytest.mark.parametrize("act", [OB.SILU, OB.GELU])
def test_glu_backward_against_differences(act):
    rng = np.random.default_rng(7)
    gu, dh = rng.standard_normal((3, 8)) * 2, rng.standard_normal((3, 4))
    d = OB.glu_backward(gu, dh, act)
    h = 1e-6
    for r in range(3):
        for c in range(8):
            e = np.zeros_like(gu)
            e[r, c] = h
            diff = (dh * (OB.glu(gu + e, act) - OB.glu(gu - e, act))).sum() / (2 * h)
            assert math.isclose(d[r, c], diff, rel_tol=1e-5, abs_tol=1e-8)

"""The FP64 gate and int8 oracles against hand-worked rows, differences and
whole-number arithmetic (CPU)."""
import fractions

import numpy as np
import pytest

from oracle import gate as OG
from oracle import int8 as OI


def test_gate_hand_worked():
    # softmax of ln(1), ln(2), ln(3), ln(4): 0.1, 0.2, 0.3, 0.4
    l = np.log([[1.0, 2.0, 3.0, 4.0]])
    r = OG.gate(l, None, OG.SOFTMAX, 1, 1, 1, 2, 1, 2.0)
    assert r["idx"].tolist() == [[2, 3]]
    np.testing.assert_allclose(r["w"], [[6 / 7, 8 / 7]], rtol=1e-15)
    # a bias moves the choice and not the weight
    r = OG.gate(l, np.array([0.35, 0, 0, 0]), OG.SOFTMAX, 1, 1, 1, 2, 0, 1.0)
    assert r["idx"].tolist() == [[0, 3]]
    np.testing.assert_allclose(r["w"], [[0.1, 0.4]], rtol=1e-15)
    assert r["counts"].tolist() == [1, 0, 0, 1]
    # two groups: top-1 keeps the second (0.4), top-2 too (0.7 against 0.3)
    assert OG.gate(l, None, OG.SOFTMAX, 2, 1, 1, 1, 0, 1.0)["idx"].tolist() == [[3]]
    # sigmoid(0) = 1/2 everywhere: ties to the lower index and group
    z = np.zeros((1, 6))
    r = OG.gate(z, None, OG.SIGMOID, 3, 2, 2, 3, 0, 1.0)
    assert r["idx"].tolist() == [[0, 1, 2]] and (r["w"] == 0.5).all()


def test_gate_exclusion():
    l = np.array([[-np.inf, 1.0, -np.inf, 0.0], [-np.inf] * 4])
    r = OG.gate(l, None, OG.SOFTMAX, 1, 1, 1, 3, 1, 1.0)
    assert r["idx"].tolist() == [[0, 1, 3], [0, 1, 2]]
    assert r["w"][0, 0] == 0 and (r["w"][1] == 0).all()
    r = OG.gate(np.array([[3.0, 1.0, 0.0]]), np.array([-np.inf, 0, 0]), OG.SIGMOID, 1, 1, 1, 2, 0, 1.0)
    assert r["idx"].tolist() == [[1, 2]]


@pytest.mark.parametrize("score", [OG.SOFTMAX, OG.SIGMOID])
@pytest.mark.parametrize("renorm", [0, 1])
def test_gate_backward_against_differences(score, renorm):
    rng = np.random.default_rng(5)
    T, E, k, scale = 3, 9, 4, 1.7
    l = rng.standard_normal((T, E)) * 2
    idx = np.stack([np.sort(rng.choice(E, k, replace=False)) for _ in range(T)])
    dw, ds = rng.standard_normal((T, k)), rng.standard_normal((T, E))

    def loss(l):
        s = OG.gate_scores(l, score)
        w = np.take_along_axis(s, idx, 1)
        if renorm:
            w = w / w.sum(axis=1, keepdims=True)
        return (scale * w * dw).sum() + (s * ds).sum()

    got = OG.gate_backward(l, score, renorm, scale, idx, dw, ds)
    h = 1e-6
    for t in range(T):
        for e in range(E):
            d = np.zeros_like(l)
            d[t, e] = h
            # central differences: error h^2/6 |f'''| + 2^-53 |f| / h, far below 1e-8
            assert abs((loss(l + d) - loss(l - d)) / (2 * h) - got[t, e]) < 1e-8


def test_quant_rows_is_the_exact_rounding():
    rng = np.random.default_rng(1)
    v = rng.standard_normal((4, 64)).astype(np.float32)
    v[1] = np.arange(64, dtype=np.float32) * 0.5     # ties
    v[1, -1] = 127.0                                 # scale 1
    v[2] = 0
    v[3] *= np.float32(2.0) ** -130                  # subnormal scales
    q, s = OI.quant_rows(v)
    assert s[1] == 1 and s[2] == 1 and (q[2] == 0).all()
    assert q[1, :8].tolist() == [0, 0, 1, 2, 2, 2, 3, 4]
    for m in range(4):
        for a, b in zip(v[m], q[m]):
            assert round(fractions.Fraction(float(a)) / fractions.Fraction(float(s[m]))) == b


def test_products_and_swiglu():
    rng = np.random.default_rng(2)
    a = rng.integers(-127, 128, (5, 32)).astype(np.int8)
    b = rng.integers(-127, 128, (3, 4, 32)).astype(np.int8)
    sa, sb = np.full(5, 0.5, np.float32), np.full((3, 4), 0.25, np.float32)
    offs, index = [0, 2, 2, 4], np.array([4, 0, 0, 1])
    p = OI.products(a, sa, b, sb, offs, index)
    for r, g in ((0, 0), (1, 0), (2, 2), (3, 2)):
        want = [int(a[index[r]].astype(int) @ b[g, n].astype(int)) * 0.125 for n in range(4)]
        assert p[r].tolist() == want
    h = OI.swiglu(np.array([[0.0, 2.0, 3.0, -1.0]]))
    np.testing.assert_allclose(h, [[0.0, -2.0 / (1 + np.exp(-2.0))]], rtol=1e-15)

"""Pins of the trained scorer's oracle (oracle/scorer.py): hand-worked values, and gradients against differences."""
import math

import numpy as np
import pytest

from oracle import scorer as S


def test_embedding_by_hand():
    table = np.array([[1.0, 2.0], [3.0, -4.0]])
    assert S.embedding(table, [1, -1, 0, 2, 1], 0.5).tolist() == [[1.5, -2], [0, 0], [0.5, 1], [0, 0], [1.5, -2]]
    d, size, n = S.embedding_backward(np.array([[1.0, 2], [9, 9], [-3, 4], [9, 9], [1, 1]]), [1, -1, 0, 2, 1], 2, 0.5)
    assert d.tolist() == [[-1.5, 2], [1, 1.5]] and size.tolist() == [[1.5, 2], [1, 1.5]] and n.tolist() == [1, 2]


def test_row_by_hand():
    r = S.Row([0.0, math.log(2), -np.inf, np.nan, math.log(5)], 1.0)
    assert np.allclose(r.p, [1 / 8, 2 / 8, 0, 0, 5 / 8], rtol=1e-15)
    assert np.isclose(r.entropy, math.log(8) - 2 / 8 * math.log(2) - 5 / 8 * math.log(5), rtol=1e-15)
    assert r.top(4)[0].tolist() == [4, 1, 0, -1] and r.top(4)[1][3] == -np.inf
    assert np.allclose(S.Row([0.0, math.log(2)], 2.0).p, [1 / 5, 4 / 5])
    both = S.Row([np.inf, 1.0, np.inf], 1.0)
    assert both.p.tolist() == [0.5, 0, 0.5] and both.top(2)[0].tolist() == [0, 2]
    none = S.Row([-np.inf, np.nan], 1.0)
    assert none.entropy == 0 and not none.p.any() and none.top(1)[0].tolist() == [-1] and not none.backward(0, 1.0, 1.0).any()


@pytest.mark.parametrize("scale", [1.0, 0.3, 2.5])
def test_row_gradient_against_differences(scale):
    rng = np.random.default_rng(1)
    l = rng.normal(size=9)
    l[4] = -np.inf
    for token, d, dh in ((2, 1.3, -0.7), (4, 1.0, 0.4), (-1, 5.0, 1.0), (9, 5.0, -2.0)):
        got = S.Row(l, scale).backward(token, d, dh)
        for i in range(9):
            if i == 4:
                assert got[i] == (0 if token != 4 else 0)
                continue
            f = []
            for h in (1e-6, -1e-6):
                m = l.copy()
                m[i] += h
                r = S.Row(m, scale)
                shut = not (0 <= token < 9) or m[token] == -np.inf
                f.append((0 if shut else d * r.logp[token]) + dh * r.entropy)
            diff = (f[0] - f[1]) / 2e-6
            if token == 4:   # a shut token: its log probability is -inf for every logit; the formula's -d p stays
                diff -= scale * d * S.Row(l, scale).p[i]
            assert abs(got[i] - diff) < 1e-8


@pytest.mark.parametrize("act", ["none", "relu", "silu", "gelu"])
def test_gated_against_differences(act):
    rng = np.random.default_rng(2)
    R, K, N, M = 7, 5, 4, 3
    x, wg, wu, dh = rng.normal(size=(R, K)), rng.normal(size=(M, N, K)), rng.normal(size=(M, N, K)), rng.normal(size=(R, N))
    o = np.array([1, 4, 4, 6])   # rows 0 and 6 are no pair's, pair 1 has none
    h, g, u, *_ = S.gated(x, wg, wu, act, o)
    assert np.isnan(h[[0, 6]]).all() and np.isfinite(h[1:6]).all()
    dx, dg, du, *_ = S.gated_backward(dh, x, wg, wu, g, u, act, o)
    assert np.isnan(dx[[0, 6]]).all() and not dg[1].any()
    for a, got in ((x, dx), (wg, dg), (wu, du)):
        for i in np.ndindex(a.shape):
            if a is x and i[0] in (0, 6):
                continue
            keep, f = a[i], []
            for s in (1e-6, -1e-6):
                a[i] = keep + s
                f.append(float(np.nansum(S.gated(x, wg, wu, act, o)[0] * dh)))
            a[i] = keep
            assert abs((f[0] - f[1]) / 2e-6 - got[i]) < 1e-7


def test_activations_by_hand():
    v = np.array([-1000.0, -1.0, 0.0, 1.0, 1000.0])
    assert np.allclose(S.activation(v, "silu")[0], [0, -1 / (1 + math.e), 0, math.e / (1 + math.e), 1000], atol=1e-300)
    assert np.allclose(S.activation(v, "gelu")[0], [0, -0.15865525393145705, 0, 0.8413447460685429, 1000], rtol=1e-12)
    # Q(10) = phi(10) / 10 (1 - 1/100 + 3/10^4 - 15/10^6 + ..)
    q = math.exp(-50) / math.sqrt(2 * math.pi) / 10 * (1 - 1e-2 + 3e-4 - 15e-6 + 105e-8 - 945e-10)
    assert abs(S.activation(np.array([-10.0]), "gelu")[0][0] / (-10 * q) - 1) < 2e-8
    assert S.activation(v, "relu")[1].tolist() == [0, 0, 0, 1, 1]

"""Pins of the routed-expert oracle (oracle/experts.py): hand-worked values, gradients against differences,
and the sort against its definition."""
import numpy as np
import pytest

from oracle import experts as X


def test_route_by_hand():
    l = np.array([[0.0, np.log(2.0), np.log(2.0), np.log(3.0)]])
    ids, w, _ = X.route(l, 3, False)
    assert ids.tolist() == [[3, 1, 2]]   # the tie goes to the lower expert
    assert np.allclose(w, [[3 / 8, 2 / 8, 2 / 8]], rtol=1e-15)
    ids, w, _ = X.route(l, 3, True)
    assert np.allclose(w, [[3 / 7, 2 / 7, 2 / 7]], rtol=1e-15)


def test_route_shut_experts():
    l = np.array([[-np.inf, np.nan, 1.0], [-np.inf, -np.inf, np.nan], [np.inf, 0.0, np.inf]])
    ids, w, _ = X.route(l, 2, True)
    assert ids.tolist() == [[2, -1], [-1, -1], [0, 2]]
    assert w.tolist() == [[1.0, 0.0], [0.0, 0.0], [0.5, 0.5]]


@pytest.mark.parametrize("renormalise", [False, True])
def test_route_backward_against_differences(renormalise):
    rng = np.random.default_rng(1)
    l = rng.normal(size=(5, 9))
    l[0, 3] = -np.inf
    dw = rng.normal(size=(5, 4))
    ids, w, _ = X.route(l, 4, renormalise)
    d, _, _ = X.route_backward(l, ids, w, dw, renormalise)
    h = 1e-6
    for t in range(5):
        for e in range(9):
            if l[t, e] == -np.inf:
                assert d[t, e] == 0.0
                continue
            f = []
            for step in (h, -h):
                m = l.copy()
                m[t, e] += step
                i2, w2, _ = X.route(m, 4, renormalise)
                assert np.array_equal(i2, ids)   # the choice does not move for these inputs
                f.append(float(np.sum(w2 * dw)))
            assert abs((f[0] - f[1]) / (2 * h) - d[t, e]) < 1e-8


def test_sort_by_hand():
    off, order, pos = X.sort(np.array([[2, 0], [0, -1], [5, 2], [1, 0]]), 3)
    assert off.tolist() == [0, 3, 4, 6]
    assert order.tolist() == [1, 2, 7, 6, 0, 5, -1, -1]
    assert pos.tolist() == [[4, 0], [1, -1], [-1, 5], [3, 2]]


def test_exchange_gradients_are_transposes():
    """dispatch and combine are linear in the rows: their backwards satisfy <A x, r> = <x, A' r>."""
    rng = np.random.default_rng(2)
    T, K, D = 6, 3, 5
    _, _, pos = X.sort(rng.integers(-1, 4, (T, K)), 4)
    x, r = rng.normal(size=(T, D)), rng.normal(size=(T * K, D))
    w = rng.normal(size=(T, K))
    sent = X.dispatch(x, pos, np.zeros((T * K, D)))
    dx, _ = X.combine(r, pos, None)
    assert np.isclose(np.sum(sent * r), np.sum(x * dx), rtol=1e-12)
    dy = rng.normal(size=(T, D))
    y, _ = X.combine(r, pos, w)
    dr, dw, _ = X.combine_backward(dy, r, pos, w, np.zeros((T * K, D)))
    assert np.isclose(np.sum(y * dy), np.sum(dr * r), rtol=1e-12)
    assert np.isclose(np.sum(y * dy), np.sum(w * dw), rtol=1e-12)   # y is linear in w too


def test_linear_by_hand():
    # one output, 3 inputs, group 2 (the last one short): W = [0.5 (3 - 8), 0.5 (8 - 8), 2 (15 - 8)]
    q = X.unpack(np.array([[[0x83, 0x0F]]], np.uint8), 3)
    assert q.tolist() == [[[3, 8, 15]]]
    s = np.array([[[0.5, 2.0]]])
    y, mag = X.linear(np.array([[2.0, 100.0, -1.0]]), q, s, None, 2, None, None, False, np.zeros((1, 1)))
    assert y.tolist() == [[-5.0 - 14.0]]
    assert mag.tolist() == [[0.5 * (2 * 11 + 100 * 16) + 2.0 * 23]]
    z = np.array([[[3, 0]]], np.uint8)
    y, _ = X.linear(np.array([[2.0, 1.0, -1.0]]), q, s, z, 2, None, np.array([[30.0]]), True, np.zeros((1, 1)))
    assert y.tolist() == [[2.5 - 30.0 + 30.0]]


def test_linear_rows_by_expert():
    rng = np.random.default_rng(3)
    q = rng.integers(0, 16, (3, 4, 8)).astype(np.uint8)
    s = rng.normal(size=(3, 4, 1))
    x = rng.normal(size=(5, 8))
    y, _ = X.linear(x, q, s, None, 8, np.array([0, 2, 2, 4]), None, False, np.full((5, 4), 7.0))
    for r, e in ((0, 0), (1, 0), (2, 2), (3, 2)):
        assert np.allclose(y[r], ((q[e] - 8.0) * s[e]) @ x[r])
    assert np.all(y[4] == 7.0)

"""The layer oracle (oracle/layer.py) against closed forms, brute force and differences (CPU only)."""
import itertools
import math

import numpy as np
import pytest

from oracle import layer as ol


def test_route_by_hand():
    l = np.array([[1.0, 3.0, 2.0, 3.0], [0.0, 0.0, 0.0, 0.0], [-1.0, np.nan, -np.inf, 5.0]])
    ids, w = ol.route(l, 2)
    assert ids.tolist() == [[1, 3], [0, 1], [3, 0]]          # ties to the lower id; NaN and -inf never chosen
    assert np.allclose(w[:2], 0.5, rtol=0, atol=1e-15)
    assert np.allclose(w[2], [1 / (1 + math.exp(-6)), 1 / (1 + math.exp(6))], rtol=1e-14)
    m, row = ol.rows_of(ids, 4, 100)
    assert m.tolist() == [2, 2, 0, 2]
    assert row.tolist() == [[2, 4], [0, 3], [5, 1]]
    m, row = ol.rows_of(ids, 4, 8, cap=1)
    assert row.tolist() == [[1, 3], [0, -1], [-1, -1]]
    m, row = ol.rows_of(ids, 4, 9, seg_align=4)
    assert row.tolist() == [[4, 8], [0, 5], [-1, 1]]


def test_route_without_candidates():
    ids, w = ol.route(np.full((2, 4), -np.inf), 3)
    assert (ids == -1).all() and (w == 0).all()
    ids, w = ol.route(np.array([[np.inf, 1.0, np.inf, -np.inf]]), 4, "sigmoid")
    assert ids.tolist() == [[0, 2, 1, -1]] and w[0, 3] == 0


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("group_top", [1, 2])
def test_groups_against_brute_force(score, group_top):
    rng = np.random.default_rng(5)
    l, bias = rng.normal(size=(30, 12)), rng.normal(size=12) * 0.1
    ids, _ = ol.route(l, 3, score, bias=bias, n_groups=4, topk_groups=2, group_top=group_top)
    s = ol.scores(l, score) + bias
    for t in range(30):
        best = None
        for groups in itertools.combinations(range(4), 2):
            total = sum(np.sort(s[t, 3 * g:3 * g + 3])[-group_top:].sum() for g in groups)
            if best is None or total > best[0]:
                best = (total, groups)
        cand = [e for g in best[1] for e in range(3 * g, 3 * g + 3)]
        assert ids[t].tolist() == sorted(cand, key=lambda e: -s[t, e])[:3]


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [False, True])
def test_route_backward_against_differences(score, renorm):
    rng = np.random.default_rng(6)
    l, dw = rng.normal(size=(4, 9)), rng.normal(size=(4, 3))
    ids, _ = ol.route(l, 3, score, renorm=renorm, scale=2.5)

    def loss(x):
        s, total = ol.scores(x, score), 0.0
        for t in range(4):
            total += (ol.weights(x[t, ids[t]], s[t, ids[t]], score, renorm, 2.5) * dw[t]).sum()
        return total
    g = ol.route_backward(l, ids, dw, score, renorm, 2.5)
    h = 1e-6
    for t, e in itertools.product(range(4), range(9)):
        d = np.zeros_like(l)
        d[t, e] = h
        # central difference: h^2 / 6 times third derivatives (< 10 here), and rounding 1e-16 / h
        assert abs((loss(l + d) - loss(l - d)) / (2 * h) - g[t, e]) < 1e-8


def test_far_negative_sigmoids_keep_their_ratio():
    l = np.array([[-800.0, -801.0, -900.0]])
    _, w = ol.route(l, 2, "sigmoid")
    assert np.allclose(w[0], [1 / (1 + math.exp(-1)), 1 / (1 + math.e)], rtol=1e-12)


def test_combine_is_the_transpose_of_dispatch():
    rng = np.random.default_rng(7)
    row_of = np.array([[0, 3], [-1, 1], [2, 9]])             # 9 is past the rows
    x, v = rng.normal(size=(3, 5)), rng.normal(size=(4, 5))
    A = ol.dispatch(x, row_of, 4)
    out, _ = ol.combine(v, row_of, None, 4)
    assert np.isclose(sum((A[r] * v[r]).sum() for r in A), (out * x).sum(), rtol=1e-13)


def test_combine_backward_against_differences():
    rng = np.random.default_rng(8)
    row_of = np.array([[0, 3], [-1, 1]])
    Y, w, dout = rng.normal(size=(4, 5)), rng.normal(size=(2, 2)), rng.normal(size=(2, 5))
    dY, dw, _ = ol.combine_backward(dout, Y, w, row_of, 4)
    # the combination is linear in Y and in w: exact differences
    f = lambda y, ww: (ol.combine(y, row_of, ww, 4)[0] * dout).sum()   # noqa: E731
    for r, c in itertools.product(range(4), range(5)):
        d = np.zeros_like(Y)
        d[r, c] = 1
        assert np.isclose(f(Y + d, w) - f(Y, w), dY[r][c] if r in dY else 0, rtol=1e-9, atol=1e-12)
    for t, j in itertools.product(range(2), range(2)):
        d = np.zeros_like(w)
        d[t, j] = 1
        assert np.isclose(f(Y, w + d) - f(Y, w), dw[t, j], rtol=1e-9, atol=1e-12)


def test_swiglu_backward_against_differences():
    rng = np.random.default_rng(9)
    gu, dh = rng.normal(size=(2, 64)) * 2, rng.normal(size=(2, 32))
    d, h = ol.swiglu_backward(gu, dh)
    assert np.allclose(h, ol.swiglu(gu), rtol=1e-14)
    eps = 1e-6
    for r, c in itertools.product(range(2), range(64)):
        e = np.zeros_like(gu)
        e[r, c] = eps
        diff = ((ol.swiglu(gu + e) - ol.swiglu(gu - e)) * dh).sum() / (2 * eps)
        assert abs(diff - d[r, c]) < 1e-8
    # gate column 17 is column 33 of the interleaved order, its up column 49
    g, u = np.zeros((1, 32)), np.zeros((1, 32))
    g[0, 17], u[0, 17] = 1.0, 2.0
    v = ol.interleave(g, u)
    assert v[0, 33] == 1.0 and v[0, 49] == 2.0 and np.count_nonzero(v) == 2


def test_scales_and_token_groups():
    assert ol.scale_of(np.array([448.0, 0.0, 1.0, 449.0, 1e-44]), True).tolist() == [1.0, 1.0, 2.0 ** -8, 2.0, 2.0 ** -126]
    assert ol.scale_of(np.array([448.0, 0.0]), False).tolist() == [1.0, 1.0]
    assert ol.token_groups([130, 0, -5, 128, 1], 10 ** 6) == [(0, 128), (128, 130), (130, 258), (258, 259)]
    assert ol.token_groups([130, 200], 140) == [(0, 128), (128, 130), (130, 140)]

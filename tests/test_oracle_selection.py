"""The plain 64-bit selection operators: cases worked by hand, closed forms,
and the gradient against differences."""
import math

import numpy as np
import pytest

from oracle import selection as sel


def test_route_softmax_by_hand():
    # exp: 1, 2, 4, 1 over 8; the two 1/8 tie and the lower index comes first
    z = np.log([[1.0, 2.0, 4.0, 1.0]])
    ids, w, counts = sel.route(z, 3, renormalise=False)
    assert ids.tolist() == [[2, 1, 0]]
    np.testing.assert_allclose(w, [[0.5, 0.25, 0.125]], rtol=1e-15)
    assert counts.tolist() == [1, 1, 1, 0]
    _, w, _ = sel.route(z, 3, renormalise=True, scale=7.0)
    np.testing.assert_allclose(w, [[4.0, 2.0, 1.0]], rtol=1e-15)


def test_route_bias_is_for_the_choice_only():
    z = np.zeros((1, 4))
    ids, w, _ = sel.route(z, 2, score="sigmoid", bias=[0.0, 0.1, 0.3, 0.2], renormalise=False)
    assert ids.tolist() == [[2, 3]]
    np.testing.assert_array_equal(w, [[0.5, 0.5]])


def test_route_groups_by_hand():
    # sums of the best two: group 0: 0.9 + 0.1, group 1: 0.6 + 0.5
    s = np.array([[0.9, 0.1, 0.6, 0.5]])
    z = np.log(s / (1 - s))
    ids, _, _ = sel.route(z, 2, score="sigmoid", groups=2, kept_groups=1)
    assert ids.tolist() == [[2, 3]]
    ids, _, _ = sel.route(z, 2, score="sigmoid", groups=2, kept_groups=1, group_top=1)
    assert ids.tolist() == [[0, 1]]


def test_route_nothing_left():
    z = np.array([[-np.inf, np.nan, -np.inf, 1.0], [-np.inf] * 4, [0.0] * 4])
    ids, w, counts = sel.route(z, 2, live=[1, 1, 0])
    assert ids.tolist() == [[3, -1], [-1, -1], [-1, -1]]
    assert w.tolist() == [[1.0, 0.0], [0.0, 0.0], [0.0, 0.0]]
    assert counts.tolist() == [0, 0, 0, 1]


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renormalise", [False, True])
def test_route_gradient_against_differences(score, renormalise):
    rng = np.random.default_rng(5)
    z = rng.normal(size=(3, 9))
    ids, _, _ = sel.route(z, 4, score=score)
    g = rng.normal(size=(3, 4))
    grad, size = sel.route_backward(z, ids, g, score, renormalise, 1.5)
    assert np.all(np.abs(grad) <= size * (1 + 1e-12))

    def loss(y, t):
        s, _ = sel.expert_scores(y, score)
        w = s[ids[t]]
        return 1.5 * float((w / (w.sum() if renormalise else 1.0) * g[t]).sum())

    h = 1e-6
    for t in range(3):
        for j in range(9):
            up, down = z[t].copy(), z[t].copy()
            up[j] += h
            down[j] -= h
            # central differences: h^2 for the third derivative (at most about
            # ten times the weights'), 2^-52 / h for the values' rounding
            assert abs((loss(up, t) - loss(down, t)) / (2 * h) - grad[t, j]) < 1e-8


def test_adjust_by_hand():
    z = np.array([[2.0, -2.0, 3.0, 0.5, 1.0]], np.float32)
    out = sel.adjust(z, history=np.array([[0, 1, 2, 2, 9]]), history_len=[5], prompt_len=[2],
                     repetition=[2.0], presence=[0.25], frequency=[0.5],
                     bias_ids=np.array([[3, 3, -1]]), bias_values=np.array([[5.0, 1.0, 7.0]]),
                     allowed=np.array([[0b01111]]))
    assert out.tolist() == [[1.0, -4.0, 1.5 - 1.0 - 0.25, 1.5, -math.inf]]


def test_adjust_mask_rows():
    z = np.zeros((3, 2), np.float32)
    out = sel.adjust(z, allowed=np.array([[0b10]]), allowed_rows=np.array([0, -1, 1]))
    assert out.tolist() == [[-math.inf, 0.0], [0.0, 0.0], [-math.inf, -math.inf]]


def test_pick_by_hand():
    z = np.log(np.array([[1.0, 4.0, 2.0, 1.0]])).repeat(5, 0).astype(np.float32)
    u = [0.0, 0.49, 0.51, 0.76, 0.99]
    ids, lp = sel.pick(z, u, 4)
    assert ids.tolist() == [1, 1, 2, 0, 3]
    np.testing.assert_allclose(lp, np.log([0.5, 0.5, 0.25, 0.125, 0.125]), atol=1e-7)
    assert sel.pick(z, u, 4, top_p=[0.6] * 5)[0].tolist() == [1, 1, 1, 2, 2]
    assert sel.pick(z, u, 4, min_p=[0.6] * 5)[0].tolist() == [1] * 5
    assert sel.pick(z, u, 2)[0].tolist() == [1, 1, 1, 2, 2]
    assert sel.pick(z, u, 4, temperature=[0.0] * 5)[0].tolist() == [1] * 5


def test_pick_nothing_left():
    z = np.array([[-np.inf, np.nan], [np.inf, 0.0]], np.float32)
    ids, lp = sel.pick(z, [0.5, 0.9], 2)
    assert ids.tolist() == [-1, 0]
    assert lp.tolist() == [-math.inf, 0.0]

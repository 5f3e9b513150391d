"""The 64-bit reference of the router's gradient against central differences of the
reference of its weights (no GPU)."""
import numpy as np
import pytest

from tests import expert_ref as ref


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renormalize", [True, False])
def test_route_gradient_is_the_difference_quotient(score, renormalize):
    g = np.random.default_rng([70, len(score), renormalize])
    x = g.standard_normal((5, 12)) * 2
    x[1, 3:9] = -np.inf
    ids, _ = ref.route(x, 4, score)
    ids[2, 2:] = -1
    dw = g.standard_normal(ids.shape)
    dx = ref.route_backward(x, ids, dw, score, renormalize, 2.5)
    h = 1e-5
    for t in range(5):
        for e in range(12):
            if np.isneginf(x[t, e]):
                assert dx[t, e] == 0
                continue
            up, down = x.copy(), x.copy()
            up[t, e] += h
            down[t, e] -= h
            diff = ((ref.route_weights(up, ids, score, renormalize, 2.5)
                     - ref.route_weights(down, ids, score, renormalize, 2.5)) * dw).sum() / (2 * h)
            # third derivatives of the scores are below 1, the weights' factors below 10:
            # truncation 10 h^2, rounding 1e-15 / h
            assert abs(diff - dx[t, e]) < 4e-9


@pytest.mark.parametrize("score,top", [("sigmoid", -60.0), ("sigmoid", -95.0), ("softmax", -95.0)])
def test_route_gradient_of_small_scores(score, top):
    """The same where the scores are far below 1: the weights and their gradient are not."""
    g = np.random.default_rng([99, len(score), int(-top)])
    x = top - 5 * g.random((3, 8))
    x[:, 7] = top + 100 if score == "softmax" else top
    ids = np.tile(np.arange(4), (3, 1))
    dw = g.standard_normal(ids.shape)
    dx = ref.route_backward(x, ids, dw, score, True, 2.5)
    assert np.abs(dx).max() > 0.05
    h = 1e-5
    for t in range(3):
        for e in range(8):
            up, down = x.copy(), x.copy()
            up[t, e] += h
            down[t, e] -= h
            diff = ((ref.route_weights(up, ids, score, True, 2.5)
                     - ref.route_weights(down, ids, score, True, 2.5)) * dw).sum() / (2 * h)
            # truncation 10 h^2; the weights' rounding, with |x| near 100 in the exponent, 1e-13 / h
            assert abs(diff - dx[t, e]) < 4e-8

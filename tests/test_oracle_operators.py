"""The fp64 definitions of the training-step operators, pinned on the CPU: the gradients to
central differences of the forward definitions, the rest to hand-worked values."""
import numpy as np
import pytest

from oracle import operators as P


def test_embed_by_hand():
    table = np.array([[1.0, 2.0], [3.0, 4.0]])
    out = np.full((5, 2), 9.0)
    got = P.embed([1, 7, 0, -1], table, out, scale=2.0, token=7)
    np.testing.assert_array_equal(got, [[6, 8], [9, 9], [2, 4], [0, 0], [9, 9]])


def test_embed_backward_is_the_difference_quotient():
    rng = np.random.default_rng(1)
    ids = np.array([0, 3, 7, 3, 1, 3, 0, 99])
    table, d_out = rng.normal(size=(5, 3)), rng.normal(size=(8, 3))
    grad, mag = P.embed_backward(ids, d_out, 5, scale=1.5, token=7)

    def loss(t):
        return (P.embed(ids, t, np.zeros((8, 3)), 1.5, 7) * d_out).sum()

    h = 1e-5
    for t in range(5):
        for c in range(3):
            e = np.zeros_like(table)
            e[t, c] = h
            # the lookup is linear: the quotient is exact up to cancellation, 2^-52 * |loss| / h
            assert abs((loss(table + e) - loss(table - e)) / (2 * h) - grad[t, c]) < 1e-8
    assert (mag >= np.abs(grad) - 1e-15).all() and (grad[2] == 0).all()


def test_layernorm_by_hand():
    y, mean, rstd = P.layernorm(np.array([[1.0, 3.0]]), np.array([2.0, 1.0]), np.array([0.5, -0.5]), eps=0.0)
    np.testing.assert_allclose(y, [[-1.5, 0.5]])
    assert mean[0] == 2 and rstd[0] == 1


@pytest.mark.parametrize("rows,C", [(1, 2), (3, 5), (2, 1)])
def test_layernorm_backward_is_the_difference_quotient(rows, C):
    rng = np.random.default_rng(rows * 10 + C)
    x, d_y = rng.normal(size=(rows, C)), rng.normal(size=(rows, C))
    gamma, beta = rng.normal(size=C), rng.normal(size=C)
    _, mean, rstd = P.layernorm(x, gamma, beta)
    d_x, d_gamma, d_beta = P.layernorm_backward(x, mean, rstd, d_y, gamma)

    def loss(xx, g, b):
        return (P.layernorm(xx, g, b)[0] * d_y).sum()

    h = 1e-5

    def quotient(make):
        return (loss(*make(h)) - loss(*make(-h))) / (2 * h)

    # second-order quotient: h^2 times a third derivative, which stays below 1e3 here except
    # for rows of one element, where the loss does not depend on x at all
    for r in range(rows):
        for c in range(C):
            e = np.zeros_like(x)
            e[r, c] = 1.0
            assert abs(quotient(lambda t: (x + t * e, gamma, beta)) - d_x[r, c]) < 1e-6
    for c in range(C):
        e = np.zeros(C)
        e[c] = 1.0
        assert abs(quotient(lambda t: (x, gamma + t * e, beta)) - d_gamma[c]) < 1e-8
        assert abs(quotient(lambda t: (x, gamma, beta + t * e)) - d_beta[c]) < 1e-8


def test_clip_by_hand():
    norm, got = P.clip_grads([np.array([3.0]), np.array([0.0, 4.0])], 1.0)
    assert norm == 5.0
    np.testing.assert_allclose(got[0], 3.0 / 5.000001)
    np.testing.assert_allclose(got[1], [0.0, 4.0 / 5.000001])
    assert P.clip_grads([np.array([3.0])], 10.0)[1][0][0] == 3.0
    norm, got = P.clip_grads([np.array([np.inf, 1.0])], 1.0)
    assert norm == np.inf and np.isnan(got[0][0]) and got[0][1] == 0.0
    assert np.isnan(P.clip_grads([np.array([np.nan, 1.0])], 1.0)[1][0]).all()
    assert P.clip_grads([], 1.0)[0] == 0.0

"""The 64-bit definitions of the vocabulary reductions against hand-worked
values and against differences of their own losses (CPU)."""
from __future__ import annotations

import numpy as np
import pytest

from oracle import vocab as vo


def test_worked_row():
    # p = (1/2, 1/4, 1/4)
    x = np.log([[2.0, 1.0, 1.0]])
    logp, empty = vo.log_softmax(x)
    np.testing.assert_allclose(np.exp(logp), [[0.5, 0.25, 0.25]], rtol=1e-15)
    np.testing.assert_allclose(vo.entropy(logp), [1.5 * np.log(2)], rtol=1e-15)
    ids, lps = vo.top(x, logp, 4)
    assert ids.tolist() == [[0, 1, 2, -1]] and lps[0, 3] == -np.inf
    # q = (3/4 on 0, remaining 1/4): KL = 3/4 ln(3/2) + 1/4 ln(1/2)
    loss, _, _ = vo.distill(x, 1.0, np.array([[0]]), np.log([[0.75]]), True)
    np.testing.assert_allclose(loss, [0.75 * np.log(1.5) + 0.25 * np.log(0.5)], rtol=1e-14)
    # renormalised, the one listed token has all the mass
    loss, _, _ = vo.distill(x, 1.0, np.array([[0]]), np.log([[0.75]]), False)
    np.testing.assert_allclose(loss, [np.log(2)], rtol=1e-14)


def test_special_rows():
    inf = np.inf
    x = np.array([[-inf, -inf, -inf], [1.0, -inf, 1.0], [np.nan, 0, 0], [inf, 0, 0]])
    logp, empty = vo.log_softmax(x)
    assert empty.tolist() == [True, False, False, False]
    assert (logp[0] == -inf).all() and np.isnan(logp[2]).all() and np.isnan(logp[3]).all()
    np.testing.assert_allclose(logp[1, [0, 2]], np.log(0.5))
    assert vo.entropy(logp)[0] == 0
    assert vo.top(x, logp, 3)[0].tolist() == [[0, 1, 2], [0, 2, 1], [1, 2, 0], [0, 1, 2]]
    g = vo.logprobs_grad(x, 1.0, np.array([0, -100, 0, 0]), np.array([1.0, 1.0, 0.0, 0.0]), 0.0)
    assert (g == 0).all()


def central(f, x, v, h=1e-5):
    a, b = x.copy(), x.copy()
    a[:, v] += h
    b[:, v] -= h
    return (f(a) - f(b)) / (2 * h)


@pytest.mark.parametrize("temperature", [1.0, 0.7, 2.5])
def test_logprobs_gradient_is_the_difference(temperature):
    rng = np.random.default_rng(0)
    x, t = rng.standard_normal((4, 9)) * 2, np.array([0, 8, 3, -100])
    gl, gh = rng.standard_normal(4), rng.standard_normal(4)

    def f(y):
        logp, _ = vo.log_softmax(y, temperature)
        return gl * vo.logprobs(logp, t) + gh * vo.entropy(logp)

    g = vo.logprobs_grad(x, temperature, t, gl, gh)
    for v in range(9):
        np.testing.assert_allclose(g[:, v], central(f, x, v), atol=1e-8)


@pytest.mark.parametrize("tail", [False, True])
@pytest.mark.parametrize("temperature", [1.0, 2.5])
def test_distill_gradient_is_the_difference(tail, temperature):
    rng = np.random.default_rng(1)
    x = rng.standard_normal((3, 9)) * 2
    ids = np.array([[1, 4, 8], [0, -1, 0], [-1, 9, -100]])       # plain, repeated with padding, no teacher
    vals = np.log(np.array([[0.4, 0.3, 0.1], [0.2, 0.5, 0.3], [0.1, 0.1, 0.1]]))
    g = np.array([0.7, -1.3, 2.0])
    f = lambda y: g * vo.distill(y, temperature, ids, vals, tail)[0]
    got = vo.distill_grad(x, temperature, ids, vals, tail, g)
    assert (got[2] == 0).all() and f(x)[2] == 0
    for v in range(9):
        np.testing.assert_allclose(got[:, v], central(f, x, v), atol=1e-8)

"""The 64-bit definitions of oracle/layer.py pinned by hand and by differences (CPU)."""
from __future__ import annotations

import numpy as np
import pytest

from oracle import layer as lo


def test_norm_by_hand():
    # s = (3, 4): mean square 12.5
    s, rstd, y = lo.reduce_norm([np.array([[1.0, 2.0]]), np.array([[1.0, 1.0]])], np.array([0.0, 1.0]),
                                np.array([[1.0, 1.0]]), eps=0.0, offset=1.0)
    np.testing.assert_array_equal(s, [[3.0, 4.0]])
    np.testing.assert_allclose(rstd, [12.5 ** -0.5], rtol=1e-15)
    np.testing.assert_allclose(y, [[3 * 12.5 ** -0.5, 8 * 12.5 ** -0.5]], rtol=1e-15)
    np.testing.assert_allclose(lo.scales(y, 0), [[8 * 12.5 ** -0.5 / 448]], rtol=1e-15)
    np.testing.assert_array_equal(lo.scales(np.array([[0.0, 0.0, np.inf]]), 2)[0, :1], [2.0 ** -100])
    assert np.isnan(lo.scales(np.array([[0.0, 0.0, np.inf]]), 2)[0, 1])


@pytest.mark.parametrize("offset", [0.0, 1.0])
def test_norm_gradient_by_differences(offset):
    rng = np.random.default_rng(1)
    x, w, g, gs = rng.normal(size=(3, 7)), rng.normal(size=7), rng.normal(size=(3, 7)), rng.normal(size=(3, 7))
    eps = 1e-3

    def value(x, w):
        s, _, y = lo.reduce_norm([x], w, eps=eps, offset=offset)
        return (y * g).sum() + (s * gs).sum()

    dx, dw = lo.reduce_norm_backward(x, w, lo.reduce_norm([x], w, eps=eps)[1], g, gs, offset)
    h = 1e-6
    for i in np.ndindex(x.shape):
        d = np.zeros_like(x)
        d[i] = h
        assert abs((value(x + d, w) - value(x - d, w)) / (2 * h) - dx[i]) < 1e-8
    for i in range(7):
        d = np.zeros(7)
        d[i] = h
        assert abs((value(x, w + d) - value(x, w - d)) / (2 * h) - dw[i]) < 1e-8


def test_embedding_and_its_gradient_are_adjoint():
    rng = np.random.default_rng(2)
    tokens = np.array([3, -1, 0, 3, 9, 10, 4])
    table, g = rng.normal(size=(10, 4)), rng.normal(size=(7, 4))
    out, grad = lo.embedding(table, tokens, 2.5), lo.embedding_backward(g, tokens, 10, 2.5)
    np.testing.assert_array_equal(out[[1, 5]], 0.0)
    np.testing.assert_array_equal(out[3], table[3] * 2.5)
    np.testing.assert_allclose(grad[3], 2.5 * (g[0] + g[3]))
    np.testing.assert_allclose((out * g).sum(), (table * grad).sum())


def test_clip_by_hand():
    g = [np.array([3.0]), np.array([[0.0, 4.0]])]
    assert lo.grad_norm(g, 0.5) == 2.5
    norm, f = lo.clip(g, 1.0, eps=0.0)
    assert (norm, f) == (5.0, 0.2)
    assert lo.clip(g, 11.0, 2.0)[1] == 2.0
    assert lo.clip([np.zeros(2)], 0.0, eps=0.0)[1] == 1.0
    assert lo.clip([np.array([np.inf])], 1.0)[1] == 0.0
    assert np.isnan(lo.clip([np.array([np.nan])], 1.0)[1])

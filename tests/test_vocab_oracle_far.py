"""The 64-bit definitions of the vocabulary reductions far from zero (CPU)."""
from __future__ import annotations

import numpy as np
import pytest

from oracle import vocab as vo


@pytest.mark.parametrize("low", [-1e3, -65504.0, -1e30, float(np.finfo(np.float32).min)])
@pytest.mark.parametrize("temperature", [1.0, 2.0])
def test_unlisted_mass_far_below_the_listed(low, temperature):
    """Equal unlisted entries share -q_t g / T equally, however far down they are, and a row's gradient sums to 0."""
    x = np.full((1, 50), low)
    ids, q = np.array([[3, 20]]), np.array([[0.5, 0.2]])
    x[0, ids[0]] = [1.0, 0.0]
    g = vo.distill_grad(x, temperature, ids, np.log(q), True, np.array([0.7]))[0]
    rest = np.delete(g, ids[0])
    np.testing.assert_allclose(rest, -0.3 * 0.7 / temperature / 48, rtol=1e-12)
    np.testing.assert_allclose(g.sum(), 0.0, atol=1e-14)

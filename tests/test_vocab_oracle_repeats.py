"""Distillation lists that name an id twice, in the 64-bit definitions (CPU)."""
from __future__ import annotations

import numpy as np
import pytest

from oracle import vocab as vo


def test_two_halves_of_a_certain_token():
    x = np.array([[60.0, 0.0, 0.0]])
    loss, _, _ = vo.distill(x, 1.0, np.array([[0, 0]]), np.log([[0.5, 0.5]]), False)
    np.testing.assert_allclose(loss, [0.0], atol=1e-15)


@pytest.mark.parametrize("tail", [False, True])
def test_equals_the_merged_list(tail):
    rng = np.random.default_rng(0)
    x = rng.standard_normal((1, 9)) * 2
    q = np.array([[0.3, 0.1, 0.2, 0.15, 0.05]])
    a = vo.distill(x, 1.0, np.array([[4, 2, 4, -1, 2]]), np.log(q), tail)[0]
    b = vo.distill(x, 1.0, np.array([[2, 4]]), np.log([[0.15, 0.5]]), tail)[0]
    np.testing.assert_allclose(a, b, rtol=1e-13)
    assert a[0] > 0

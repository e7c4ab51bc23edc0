"""The binding's reading of rank buffers of any number of dimensions (CPU)."""
from __future__ import annotations

import pytest

torch = pytest.importorskip("torch")
ar = pytest.importorskip("reduce_scatter_amd", reason="libar.so not built")

from reduce_scatter_amd import _binding as b  # noqa: E402


def check(t, rows, width, pitch):
    return b._logit_table([t], ar.VocabShape(rows, [width], "f32", pitches=[pitch]), [])


def test_rows_that_no_pitch_describes():
    x = torch.zeros(2, 5, 8)                                     # [batch, position, vocabulary]
    bad = [
        (x[:, :-1], 8, 8, 8),                                    # the last position left out: two steps between rows
        (x.transpose(0, 1), 10, 8, 8),
        (x[:, :, :6], 10, 6, 6),                                 # padded rows, given the pitch of packed ones
        (x[:, ::2], 6, 8, 8),
        (torch.zeros(40, 2)[:, 0], 5, 8, 8),                     # one dimension, elements apart
        (torch.zeros(2, 5, 8, 2)[..., 0], 10, 8, 8),
        (torch.zeros(1, 16)[:, ::2], 1, 8, 8),                   # one row, elements apart
    ]
    for t, rows, width, pitch in bad:
        with pytest.raises(ValueError, match="strides"):
            check(t, rows, width, pitch)


def test_rows_at_one_pitch():
    x = torch.zeros(2, 5, 8)
    good = [
        (x, 10, 8, 8),
        (x[:, :, :6], 10, 6, 8),
        (x[1:, :-1], 4, 8, 8),                                   # one of the outer dimension
        (x[:, 2:3], 2, 8, 40),
        (x.view(-1), 10, 8, 8),
        (torch.zeros(10, 2, 4), 10, 8, 8),                       # a row in two dimensions, packed
        (torch.zeros(3, 1, 8), 3, 8, 8),
        (torch.zeros(1, 8), 1, 8, 8),
    ]
    for t, rows, width, pitch in good:
        check(t, rows, width, pitch)

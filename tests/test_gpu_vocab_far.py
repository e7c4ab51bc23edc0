"""Vocabulary reductions on logits far from zero: masks of any finite value at
any temperature, against the 64-bit definitions.

Tolerances of test_gpu_vocab_offset.py."""
from __future__ import annotations

import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)
pytest.importorskip("reduce_scatter_amd")

import test_gpu_vocab as base  # noqa: E402
from test_gpu_vocab_offset import Far, check_all_calls  # noqa: E402


FILLS = ["lowest", -1e9, -1e10, -1e20, -1e30]


# few rows on one workgroup each (kept in registers by the calls for both), few rows over several, many rows
@pytest.mark.parametrize("rows, widths", [(6, [700, 701]), (6, [60000]), (258, [1100, 1101])])
@pytest.mark.parametrize("temperature", [0.5, 1.0, 1.5, 2.0, 100.0])
@pytest.mark.parametrize("fill", FILLS)
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_masks_of_any_finite_value(dtype, fill, temperature, rows, widths):
    rng = np.random.default_rng(31)
    vocab = sum(widths)
    x = base.logits(rng, rows, vocab)
    low = torch.finfo(base.DT[dtype]).min if fill == "lowest" else fill
    for r in range(0, rows, 6):
        x[r] = low                                                        # uniform
        x[r + 1, :vocab // 3] = low                                       # whole leading vectors and tiles
        x[r + 2, torch.arange(vocab) // 32 % 2 == 0] = low                # whole vectors in between
        x[r + 3, vocab // 3:] = low                                       # the end
        x[r + 4, torch.arange(vocab) % (vocab // 9) != 1] = low           # nine or ten entries left
    x = x[:rows]
    d = Far(x, widths, dtype, temperature, 1, 0)
    best = np.argmax(d.x, 1)
    gl, gh = rng.standard_normal(rows), rng.standard_normal(rows)
    ids = np.stack([np.argsort(-row, kind="stable")[[0, 1, 3, 5, 8]] for row in d.x]).astype(np.int64)
    vals = np.log(np.array([0.4, 0.2, 0.1, 0.1, 0.05], dtype=np.float32))[None].repeat(rows, 0)
    check_all_calls(d, best, 9, gl, gh, ids, vals)


@pytest.mark.parametrize("temperature", [1e-4, 1e-9, 1e-20, 1e-30, 1e30])
@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
def test_extreme_temperatures(dtype, temperature):
    """Ordinary logits far apart in units of the temperature, where the largest takes all; or all but equal."""
    rng = np.random.default_rng(32)
    rows, vocab = 6, 3001
    x = base.logits(rng, rows, vocab)
    x[1, 5] = x[1, 2990] = 30.0                                           # a tie
    x[2] = 0.5                                                            # uniform
    x[3, :1500] = -8.0
    d = Far(x, [1500, 1501], dtype, temperature, 1, 0)
    gl, gh = rng.standard_normal((2, rows)) * temperature                 # gradients of about 1
    ids = np.stack([np.argsort(-row, kind="stable")[:2] for row in d.x]).astype(np.int64)
    # an entry without mass where the two differ (their divergence would be about 1 / T)
    vals = np.tile(np.array([[0.0, -np.inf]], dtype=np.float32), (rows, 1))
    vals[1:3] = np.log(np.float32(0.5))
    check_all_calls(d, np.argmax(d.x, 1), 5, gl, gh, ids, vals)

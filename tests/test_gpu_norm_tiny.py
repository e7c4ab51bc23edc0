"""Rows so small that 1 / sqrt(mean(s^2)) leaves fp32, which takes eps = 0: the
stored rstd is infinite, the normalised row is not.

Tolerance, u = 2^-24: s is exact here (one buffer); squares and their sum in 64
bits; the root's rounding to fp32 and three products, 4 u, and half a step of the
stored type."""
from __future__ import annotations

import numpy as np
import pytest

from oracle import layer as lo

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)
ar = pytest.importorskip("reduce_scatter_amd")

U = 2.0 ** -24
HALF = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}


@pytest.mark.parametrize("dtype", list(HALF))
@pytest.mark.parametrize("width", [5, 40, 300, 4096, 9001])
def test_rows_of_subnormal_numbers(width, dtype):
    g = torch.Generator(device="cuda").manual_seed(width)
    x = torch.randn(6, width, generator=g, device="cuda") * 1e-39
    x[1] = 0.0                                              # 0 * inf: the definition says NaN
    x[2], x[2, width // 2] = 0.0, -2.0 ** -133              # one entry
    x[3] = 2.0 ** -133                                      # the smallest number that both types hold
    x[4] *= 2.0 ** 8                                        # rstd just inside fp32
    x = x.to(dtype)
    w = torch.rand(width, generator=g, device="cuda") + 0.5
    sh = ar.NormShape(6, width, 1, dtype, weight_dtype="f32", eps=0.0)
    out, summed, rstd = torch.empty_like(x), torch.empty_like(x), torch.empty(6, device="cuda")
    q, sc = torch.empty(6, width, dtype=torch.float8_e4m3fn, device="cuda"), torch.empty(6, 1, device="cuda")
    ar.ar_reduce_norm([x], sh, w, out=out, summed=summed, rstd=rstd, out8=q, scales=sc)
    assert torch.equal(summed, x)
    _, r, y = lo.reduce_norm([x.double().cpu().numpy()], w.double().cpu().numpy(), eps=0.0)
    with np.errstate(all="ignore"):
        want_r = np.where(r > 3.4028235677973366e38, np.inf, r)
    got_r, got = rstd.double().cpu().numpy(), out.double().cpu().numpy()
    assert np.isinf(want_r[2:4]).all() and np.isinf(want_r[0])
    assert (np.isinf(got_r) == np.isinf(want_r)).all() and abs(got_r[4] - r[4]) <= 8 * U * r[4]
    assert np.isnan(got[1]).all()
    rows = [0, 2, 3, 4, 5]
    err = np.abs(got[rows] - y[rows])
    assert (err <= (1.01 * HALF[dtype] + 8 * U) * np.abs(y[rows])).all()
    top = np.abs(y[rows]).max(1)
    assert (np.abs(sc.double().cpu().numpy()[rows, 0] * 448 - top) <= 12 * U * top).all()
    each = q.double().cpu().numpy()[rows] * sc.double().cpu().numpy()[rows]
    assert (np.abs(each - y[rows]) <= (2.0 ** -4 + 16 * U) * np.abs(y[rows]) + 1.01 * 2.0 ** -10 * top[:, None] / 448).all()

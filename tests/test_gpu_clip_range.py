"""Clipping where the factor lies below the normal numbers of fp32 (norms past
2^126 times the limit), against the 64-bit definition (oracle/layer.py).

Tolerance, u = 2^-24: the factor's rounding and two of the product, u each, and
half a step of the stored type, of its subnormal numbers too."""
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
HALF = {torch.float32: (2.0 ** -24, 2.0 ** -150), torch.bfloat16: (2.0 ** -8, 2.0 ** -134)}


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("sizes", [[5000, 3], [2_000_000, 77]])        # partial sums added up by every workgroup; by a launch of their own
@pytest.mark.parametrize("max_norm, scale", [(1.0, 1.0), (1e-2, 1.0), (1e-6, 1.0), (1e-30, 1.0), (1.0, 2.0 ** -20), (1e-12, 1e6)])
def test_factors_below_the_normal_numbers(max_norm, scale, sizes, in_place):
    g = torch.Generator(device="cuda").manual_seed(4)
    grads = [((torch.rand(n, generator=g, device="cuda") * 2 - 1) * 3e38).to(t) for n, t in zip(sizes, HALF)]
    grads[0][:4] = torch.tensor([0.0, 1.0, 1e30, 1e-40])
    before = [t.double().cpu().numpy() for t in grads]
    norm, f = lo.clip(before, float(np.float32(max_norm)), scale, 0.0)
    assert f < 2.0 ** -126
    gl = ar.GradList(grads)
    outs = gl if in_place else ar.GradList([torch.empty_like(t) for t in grads])
    got = torch.empty(1, device="cuda")
    ar.ar_clip_grads(gl, outs, got, max_norm, scale=scale, eps=0.0,
                     workspace=torch.empty(ar.ar_grad_workspace(gl), dtype=torch.uint8, device="cuda"))
    assert got.item() == float("inf") if norm > 3.4028236e38 else abs(got.item() - norm) <= 1.01 * U * norm
    for b, o in zip(before, outs._tensors):
        want, (rel, tiny) = b * f, HALF[o.dtype]
        err = np.abs(o.double().cpu().numpy() - want)
        tol = (1.01 * rel + 3 * U) * np.abs(want) + 1.01 * tiny + 2.0 ** -150
        assert (err <= tol).all(), "%d off, worst %g of %g" % ((err > tol).sum(), err.max(), np.abs(want).max())

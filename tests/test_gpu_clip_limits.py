"""What clipping does at infinities, value by value: an infinite limit never
clips, whatever the norm; a finite one makes the finite gradients zero where one
is infinite, and that one NaN (infinity times 0)."""
from __future__ import annotations

import numpy as np
import pytest

from oracle import layer as lo

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)
ar = pytest.importorskip("reduce_scatter_amd")

INF = float("inf")


def clip(values, max_norm, sizes, scale=1.0):
    """Lists of 300 or two million numbers: the norm added up in the scaling launch, or by one of its own."""
    g = [torch.full((n,), 0.5, device="cuda") for n in sizes]
    g[1][:len(values)] = torch.tensor(values)
    gl, norm = ar.GradList(g), torch.empty(1, device="cuda")
    out = ar.GradList([torch.empty_like(t) for t in g])
    ar.ar_clip_grads(gl, out, norm, max_norm, scale=scale, workspace=torch.empty(ar.ar_grad_workspace(gl), dtype=torch.uint8, device="cuda"))
    return g, out._tensors, norm.item()


@pytest.mark.parametrize("sizes", [(200, 100), (2_000_000, 100)])
def test_limits(sizes):
    for bad in (INF, -INF):
        g, out, norm = clip([bad, 3.0], INF, sizes)
        assert norm == INF and all(torch.equal(a, b) for a, b in zip(g, out))
        g, out, norm = clip([bad, 3.0], INF, sizes, scale=0.25)
        assert norm == INF and all(torch.equal(a * 0.25, b) for a, b in zip(g, out))
        g, out, norm = clip([bad, 3.0], 1.0, sizes)
        assert norm == INF and out[1][0].isnan() and (out[1][1:] == 0).all() and (out[0] == 0).all()
    _, out, norm = clip([float("nan"), 3.0], INF, sizes)
    assert norm != norm and all(t.isnan().all() for t in out)
    # a norm past fp32 is no infinite one
    g, out, norm = clip([3e38, -3e38], 3e38, sizes)
    assert norm == INF
    want = np.array([3e38, -3e38]) * np.float64(np.float32(3e38)) / lo.grad_norm([t.double().cpu().numpy() for t in g])
    assert (np.abs(out[1][:2].double().cpu().numpy() - want) <= 4 * 2.0 ** -24 * np.abs(want)).all()
    g, out, norm = clip([3e38, -3e38], INF, sizes)
    assert norm == INF and all(torch.equal(a, b) for a, b in zip(g, out))

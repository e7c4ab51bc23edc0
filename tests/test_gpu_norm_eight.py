"""The 8-bit output bit for bit: in fp32 storage `out` is y itself, so `out8` has
to be e4m3 of the fp32 quotient y / scale and `scales` the fp32 quotient of the
largest |y| and 448, both to nearest even, with no tolerance."""
from __future__ import annotations

import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)
ar = pytest.importorskip("reduce_scatter_amd")


def eight(rows, width, group, size=1.0, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(rows, width, generator=g, device="cuda")
    w = (torch.rand(width, generator=g, device="cuda") + 0.5) * size
    sh = ar.NormShape(rows, width, 1, "f32", group=group)
    out, q, sc = torch.empty_like(x), torch.empty(rows, width, dtype=torch.float8_e4m3fn, device="cuda"), torch.empty(rows, sh.groups, device="cuda")
    ar.ar_reduce_norm([x], sh, w, out=out, out8=q, scales=sc)
    return out.cpu().numpy(), q.cpu(), sc.cpu().numpy()


@pytest.mark.parametrize("size", [1.0, 2.0 ** -90, 2.0 ** 100])
@pytest.mark.parametrize("rows, width, group", [(1024, 8192, 0), (1024, 8192, 128), (999, 5003, 0), (999, 5003, 512), (4096, 200, 32),
                                                (16384, 60, 0)])
def test_quotients(rows, width, group, size):
    y, q, sc = eight(rows, width, group, size, seed=rows + width)
    g = group or width
    most = np.stack([np.abs(y[:, c:c + g]).max(1) for c in range(0, width, g)], 1)
    want = np.maximum(most / np.float32(448), np.float32(2.0 ** -100))
    assert want.dtype == np.float32 and (sc == want).all()
    each = np.repeat(sc, g, 1)[:, :width]
    quotient = torch.from_numpy(y / each).to(torch.float8_e4m3fn)
    differ = int((q.view(torch.uint8) != quotient.view(torch.uint8)).sum())
    assert differ == 0, "%d of %d" % (differ, q.numel())

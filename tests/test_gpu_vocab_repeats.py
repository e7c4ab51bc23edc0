"""Distillation lists that name an id more than once: the same as one entry
with the sum of their probabilities."""
from __future__ import annotations

import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)
ar = pytest.importorskip("reduce_scatter_amd")

import test_gpu_vocab as base  # noqa: E402
from oracle import vocab as vo  # noqa: E402


def merged(ids, q):
    """Each row's distinct ids with their summed probabilities, -1 / 0 past them."""
    oi, oq = np.full_like(ids, -1), np.zeros(ids.shape)
    for r in range(len(ids)):
        u = np.unique(ids[r][ids[r] >= 0])
        oi[r, :len(u)] = u
        oq[r, :len(u)] = [q[r, ids[r] == i].sum() for i in u]
    return oi, oq


@pytest.mark.parametrize("rows, widths", [(3, [700, 701]), (3, [60000]), (258, [2101])])
@pytest.mark.parametrize("k, distinct", [(2, 1), (9, 3), (70, 40), (256, 100)])
@pytest.mark.parametrize("tail", [False, True])
def test_repeated_ids(tail, k, distinct, rows, widths):
    rng = np.random.default_rng(51)
    vocab = sum(widths)
    pool = np.stack([rng.permutation(vocab)[:distinct] for _ in range(rows)])
    ids = np.take_along_axis(pool, rng.integers(0, distinct, (rows, k)), 1).astype(np.int64)
    q = rng.dirichlet(np.ones(k), rows) * (0.9 if tail else 1.0)
    vals = np.log(q).astype(np.float32)
    x = base.logits(rng, rows, vocab)
    x[0, ids[0, 0]] = 60.0                                # p = 1 (k = 2: the divergence is ln of q's sum, at least 0)
    d = base.Data(x, widths, "f32")
    q = np.exp(vals.astype(np.float64))
    if not tail:
        q /= q.sum(1, keepdims=True)
    mi, mq = merged(ids, q)
    with np.errstate(divide="ignore"):
        mv = np.log(mq)
    # the definition with every id once, in 64 bits (renormalising what sums to 1 changes nothing)
    want = vo.distill(d.x, 1.0, mi, mv, tail)[0]
    assert (want > -1e-6).all()
    g = rng.standard_normal(rows)
    # an entry's share of the error of the merged logarithm is that of its own: the tolerance of the list as it is
    tol, gtol = base.distill_tols(d, ids, vals, tail, g)
    wg = vo.distill_grad(d.x, 1.0, mi, mv, tail, g.astype(np.float32).astype(np.float64))
    i, v, gg = (torch.from_numpy(a).cuda() for a in (ids, vals, g.astype(np.float32)))
    for fused in (True, False):
        loss, saved = torch.full((rows,), 55.0, device="cuda"), torch.full((rows, 4), 55.0, device="cuda")
        for s in d.gstore:
            s.fill_(77.0)
        if fused:
            ar.ar_distill_grad(d.bufs, d.grads, d.shape, i, v, loss, tail=tail, grad_loss=gg, workspace=d.workspace())
        else:
            ar.ar_distill(d.bufs, d.shape, i, v, loss, tail=tail, saved=saved, workspace=d.workspace())
            ar.ar_distill_backward(d.bufs, d.grads, d.shape, i, v, saved, tail=tail, grad_loss=gg)
        torch.cuda.synchronize()
        base.close(loss.cpu(), want, tol, "loss")
        base.close(d.gather_grads(), wg, np.nan_to_num(gtol) + base.half_step(wg, "f32"), "gradient")

"""Distillation with a tail where the student's unlisted mass is far below the
listed one: its sum has to keep its own reference, or the number of unlisted
entries, and with it their gradients, is lost.

Tolerances, u = 2^-24: an unlisted entry's share of the unlisted mass is e =
2^t / sum against the unlisted entries' own reference, (seq + 48 + 6 |z - m_t|) u
of itself as in test_gpu_vocab_offset.py; the remaining mass q_t = 1 - sum q
carries the rounding of the q.  ln p_t is a product of rounded factors plus
logarithms: 6 u of itself, and the sums'."""
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
from test_gpu_vocab_offset import Far  # noqa: E402

U = base.U


def distill(d, ids, vals, g, fused):
    """(loss, gradients, saved), the gradients into buffers that held something else."""
    i, v, gg = (torch.from_numpy(a).cuda() for a in (ids, vals, g.astype(np.float32)))
    loss, saved = torch.full((d.rows,), 55.0, device="cuda"), torch.full((d.rows, 4), 55.0, device="cuda")
    for s in d.gstore:
        s.fill_(77.0)
    if fused:
        ar.ar_distill_grad(d.bufs, d.grads, d.shape, i, v, loss, tail=True, grad_loss=gg, saved=saved,
                           workspace=d.workspace())
    else:
        ar.ar_distill(d.bufs, d.shape, i, v, loss, tail=True, saved=saved, workspace=d.workspace())
        ar.ar_distill_backward(d.bufs, d.grads, d.shape, i, v, saved, tail=True, grad_loss=gg)
    torch.cuda.synchronize()
    return loss.double().cpu().numpy(), d.gather_grads(), saved.double().cpu().numpy()


@pytest.mark.parametrize("rows, widths", [(4, [700, 701]), (4, [60000]), (258, [1100, 1101])])
@pytest.mark.parametrize("temperature", [1.0, 2.0])
@pytest.mark.parametrize("fill", ["lowest", -6e4, -1e4, -1e3])
@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
def test_every_unlisted_entry_masked(dtype, fill, temperature, rows, widths):
    rng = np.random.default_rng(41)
    vocab, k = sum(widths), 7
    ids = np.stack([rng.permutation(vocab)[:k] for _ in range(rows)]).astype(np.int64)
    vals = np.log(rng.dirichlet(np.ones(k), rows) * rng.uniform(0.5, 0.95, (rows, 1))).astype(np.float32)
    low = torch.finfo(base.DT[dtype]).min if fill == "lowest" else fill
    x = torch.full((rows, vocab), low)
    x[1, ::3] = low * 0.5                                                 # two levels, far apart
    x[2] += base.logits(rng, 1, vocab)[0]                                 # spread out where the type has room for it
    x[2].clamp_(min=torch.finfo(base.DT[dtype]).min)
    x[torch.arange(rows)[:, None], torch.from_numpy(ids)] = base.logits(rng, rows, k)
    d = Far(x, widths, dtype, temperature, 1, 0)
    g = rng.standard_normal(rows)
    want = vo.distill(d.x, temperature, ids, vals, True)[0]
    wg = vo.distill_grad(d.x, temperature, ids, vals, True, g.astype(np.float32).astype(np.float64))
    q, lq, _, qt, _ = vo.teacher(ids, vals, vocab, True, temperature)
    unlisted = vo._unlisted(ids, ids >= 0, vocab)
    _, lpk, lt = vo.distill(d.x, temperature, ids, vals, True)
    zt = np.where(unlisted, d.x / temperature, -np.inf)
    dist = np.max(zt, 1, keepdims=True) - zt
    eq = (4 * np.abs(lq) + k + 16) * U                                    # relative error of a q
    dqt = (q * eq).sum(1) + (k + 8) * U
    with np.errstate(all="ignore"):
        cond = np.where(unlisted, np.exp(zt - np.max(zt, 1, keepdims=True)), 0.0)
        cond = cond / cond.sum(1, keepdims=True)
        p = np.exp(np.where(unlisted, -np.inf, d.logp))
        gtol = cond * (qt[:, None] * 2 * np.where(cond > 0, d.lp_tol(dist), 0.0) + dqt[:, None])
        gtol += p * 2 * (d.lp_tol(np.where(unlisted, 0.0, d.dist)) + (q * eq).sum(1)[:, None] + dqt[:, None])
    np.add.at(gtol, (np.arange(rows)[:, None], ids), q * eq * 2 + 4 * U * q)
    gtol = np.abs(g)[:, None] / temperature * (gtol + 2.0 ** -120) + base.half_step(wg, dtype)
    dk = np.take_along_axis(d.dist, ids, 1)
    ltol = (q * (eq * (1 + np.abs(lq) + np.abs(lpk)) + d.lp_tol(dk) + (k + 8) * U * (np.abs(lq) + np.abs(lpk)))).sum(1)
    ltol += qt * (d.lp_tol(np.abs(lt)) * 2 + 8 * U) + dqt * (1 + np.abs(lt) - np.log(qt))
    for fused in (True, False):
        loss, grads, saved = distill(d, ids, vals, g, fused)
        base.close(loss, want, ltol, "loss")
        base.close(grads, wg, gtol, "gradient")
        # as the header states them: the unlisted entries' reference and sum
        z = np.where(unlisted, (d.x - saved[:, 2:3]) / temperature, -np.inf)
        assert (z.max(1) >= 0).all() and (z.max(1) <= 11.1).all(), "m_t is not near the largest unlisted logit"
        sums = np.exp(z).sum(1)
        base.close(saved[:, 3], sums, sums * d.lp_tol(z.max(1)), "the unlisted sum")

"""Vocabulary reductions of fp32 logits that share an offset: sums, gradients
and saved statistics have to stand against one reference, so that errors do
not grow with the offset.

Tolerances as in test_gpu_vocab.py, with two constants written out.  The
reference is moved only when a tile's sum passes 2^16, so it is at most 16
units of log2 (11.1 nats) from the largest logit: 4 * 11.1 < 48.  A log
probability far from it is a product of rounded factors: at most 6 roundings
(scale, product, ln 2, its product, the subtraction of ln S, the difference of
the logits), so 6 |z - m| u."""
from __future__ import annotations

import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)
ar = pytest.importorskip("reduce_scatter_amd")

import test_gpu_vocab as base  # noqa: E402


class Far(base.Data):
    def lp_tol(self, dist):
        return (self.seq + 48 + 6 * dist) * base.U


def check_all_calls(d, targets, k, gl, gh, ids, vals, keep=None):
    """ar_logprobs (with alternatives and without), its gradient in two calls and in one; distillation of the rows
    `keep` in two calls and in one, renormalised and with a tail."""
    saved = base.check_logprobs(d, targets, k)
    base.check_logprobs(d, targets, 0, entropy=False)
    for fused in (False, True):
        base.check_logprobs_grad(d, targets, gl, gh, saved, fused)
        base.check_logprobs_grad(d, targets, gl, None, saved, fused)
    keep = np.arange(d.rows) if keep is None else keep
    part = type(d)(d.xt[torch.from_numpy(keep)], d.widths, d.dtype, d.T, 1, 0)
    for tail in (False, True):
        for mode in ("fused", "split"):
            base.check_distill(part, ids[keep], vals[keep], tail, gl[keep], mode)


@pytest.mark.parametrize("rows, widths", [(5, [3000, 1001]), (5, [60000]), (258, [1100, 1101])])
@pytest.mark.parametrize("offset, temperature", [
    (0.0, 1.0), (0.0, 0.01), (10.0, 1.0), (10.0, 0.01), (100.0, 1.0), (100.0, 0.01), (1000.0, 1.0), (-1000.0, 0.01),
    (1e6, 1.0), (1e6, 0.01), (-1e8, 1.0), (-1e8, 0.01), (7e8, 1.0), (7e8, 0.01),
])
def test_gradients(offset, temperature, rows, widths):
    rng = np.random.default_rng(33)
    x = base.logits(rng, rows, sum(widths)) * temperature + offset
    x[1, 7] += 27.0 * temperature                                         # a target that is all but certain
    d = Far(x, widths, "f32", temperature)
    t = rng.integers(0, d.vocab, rows)
    t[1] = 7
    gl, gh = rng.standard_normal(rows), rng.standard_normal(rows) * 0.3
    ids = np.stack([rng.permutation(d.vocab)[:20] for _ in range(rows)]).astype(np.int64)
    ids[:, 0] = np.argmax(d.x, 1)
    for r in range(rows):                                                 # distinct
        ids[r, 1:][ids[r, 1:] == ids[r, 0]] = -1
    vals = np.log(rng.dirichlet(np.ones(20), rows) * 0.8).astype(np.float32)
    check_all_calls(d, t, 5, gl, gh, ids, vals)


@pytest.mark.parametrize("dtype, rows, widths, offset", [
    ("f32", 3, [3000, 1001], 0.0), ("f32", 3, [3000, 1001], 1000.0), ("f32", 3, [60000], -1e6),
    ("f32", 258, [2100], 5e8), ("f32", 3, [2048], -1e9), ("bf16", 3, [3000, 1001], 30.0), ("f16", 3, [60000], -900.0),
])
def test_saved_is_a_logit_and_its_sum(dtype, rows, widths, offset):
    """saved[:, 0] and saved[:, 1] as the header states them: m and sum_v exp((x_v - m) / T)."""
    rng = np.random.default_rng(34)
    x = base.logits(rng, rows, sum(widths)) + offset
    x[2] = offset                                                         # uniform: the sum is the vocabulary's size
    d = Far(x, widths, dtype)
    f = lambda *s: torch.full(s, 55.0, device="cuda")
    lp, loss = f(rows), f(rows)
    t = torch.zeros(rows, dtype=torch.int64, device="cuda")
    ids, vals = t[:, None].contiguous(), torch.full((rows, 1), -0.7, device="cuda")
    calls = [
        lambda s: ar.ar_logprobs(d.bufs, d.shape, t, lp, saved=s, workspace=d.workspace()),
        lambda s: ar.ar_logprobs_grad(d.bufs, d.grads, d.shape, t, lp, grad_logprobs=lp, saved=s,
                                      workspace=d.workspace()),
        lambda s: ar.ar_distill(d.bufs, d.shape, ids, vals, loss, saved=s, workspace=d.workspace()),
        lambda s: ar.ar_distill(d.bufs, d.shape, ids, vals, loss, tail=True, saved=s, workspace=d.workspace()),
        lambda s: ar.ar_distill_grad(d.bufs, d.grads, d.shape, ids, vals, loss, tail=True, saved=s,
                                     workspace=d.workspace()),
    ]
    for call in calls:
        saved = f(rows, 4)
        lp.fill_(1.0)
        call(saved)
        torch.cuda.synchronize()
        got = saved.double().cpu().numpy()
        z = d.x - got[:, :1]
        assert (z.max(1) >= 0).all() and (z.max(1) <= 11.1).all(), "m is not near the largest logit"
        want = np.exp(z).sum(1)
        base.close(got[:, 1], want, want * d.lp_tol(z.max(1)), "the sum")

"""Every gradient call writes every element of its buffers and nothing else:
buffers that held NaN before each call, and calls in place whose rows lie in
one workgroup or several."""
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


# a row in one workgroup and in several, in registers and read twice, ends off 16 bytes, the large pointer table
SHAPES = [(5, [700, 701]), (258, [2101, 7000]), (3, [60000]), (130, [131500]), (2, [33000, 20, 0, 9001]), (4, [37] * 17)]


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("i", range(len(SHAPES)))
def test_fresh_and_in_place(i, dtype):
    rows, widths = SHAPES[i]
    rng = np.random.default_rng([61, i])
    d = base.Data(base.logits(rng, rows, sum(widths)), widths, dtype, 1.3, pad=[0, 3][i % 2], offset=i % 3, gpad=2, goffset=1)
    targets = rng.integers(0, d.vocab, rows)
    targets[1] = -100                                     # a row of zeros, unless the entropy counts
    ids, tv = base.teacher_lists(rng, rows, d.vocab, 30, True)
    ids[-1] = -1                                          # another
    gl, gh = (rng.standard_normal(rows).astype(np.float32) for _ in range(2))
    t, a, h, li, lv = (torch.from_numpy(v).cuda() for v in (targets, gl, gh, ids, tv))
    f = lambda *s: torch.full(s, 55.0, device="cuda")
    ws, lp, saved, loss = d.workspace(), f(rows), f(rows, 4), f(rows)
    ar.ar_logprobs(d.bufs, d.shape, t, lp, saved=saved, workspace=ws)
    want = {"logprobs": vo.logprobs_grad(d.x, d.T, targets, gl.astype(np.float64), gh.astype(np.float64)),
            "plain": vo.logprobs_grad(d.x, d.T, targets, gl.astype(np.float64), 0.0)}
    tols = {"logprobs": base.logprob_grad_tol(d, want["logprobs"], gl, gh),
            "plain": base.logprob_grad_tol(d, want["plain"], gl, np.zeros(rows))}
    calls = [
        ("logprobs", lambda x, g, sh: ar.ar_logprobs_backward(x, g, sh, t, saved, grad_logprobs=a, grad_entropy=h)),
        ("logprobs", lambda x, g, sh: ar.ar_logprobs_grad(x, g, sh, t, grad_logprobs=a, grad_entropy=h, workspace=ws)),
        ("plain", lambda x, g, sh: ar.ar_logprobs_backward(x, g, sh, t, saved, grad_logprobs=a)),
        ("plain", lambda x, g, sh: ar.ar_logprobs_grad(x, g, sh, t, grad_logprobs=a, workspace=ws)),
    ]
    for tail in (False, True):
        key, keep = "distill%d" % tail, f(rows, 4)
        ar.ar_distill(d.bufs, d.shape, li, lv, loss, tail=tail, saved=keep, workspace=ws)
        want[key] = vo.distill_grad(d.x, d.T, ids, tv, tail, gl.astype(np.float64))
        tols[key] = np.nan_to_num(base.distill_tols(d, ids, tv, tail, gl)[1]) + base.half_step(want[key], dtype)
        calls.append((key, lambda x, g, sh, tail=tail, keep=keep: ar.ar_distill_backward(x, g, sh, li, lv, keep, tail=tail,
                                                                                       grad_loss=a)))
        calls.append((key, lambda x, g, sh, tail=tail: ar.ar_distill_grad(x, g, sh, li, lv, tail=tail, grad_loss=a,
                                                                          workspace=ws)))
    for key, call in calls:
        for g, store in zip(d.grads, d.gstore):
            store.fill_(77.0)
            g.fill_(float("nan"))
        call(d.bufs, d.grads, d.shape)
        torch.cuda.synchronize()
        base.close(d.gather_grads(), want[key], tols[key], key)
        # in place, in a copy of the logits' whole storage
        stores = [s.clone() for s in d.store]
        work = [s.as_strided(b.shape, b.stride(), b.storage_offset()) for s, b in zip(stores, d.bufs)]
        call(work, work, ar.VocabShape(rows, widths, dtype, pitches=d.shape.pitches, temperature=d.T))
        torch.cuda.synchronize()
        for w, g, s, b, old in zip(work, d.grads, stores, d.bufs, d.store):
            assert torch.equal(w, g), "%s in place differs" % key
            w.copy_(b)
            ints = {"f32": torch.int32}.get(dtype, torch.int16)
            assert torch.equal(s.view(ints), old.view(ints)), "%s in place wrote between the rows" % key

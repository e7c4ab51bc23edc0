"""The output-layer example end to end: its hidden gradient against the chain
rule in 64 bits on the same logits, equal on every rank."""
from __future__ import annotations

import importlib.util
import os

import numpy as np
import pytest

from oracle import vocab as vo

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)
pytest.importorskip("reduce_scatter_amd")

PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "vocab_parallel_step.py")


@pytest.mark.parametrize("ranks, rows, vocab", [(1, 3, 997), (4, 64, 10007), (8, 300, 5000)])
def test_step(ranks, rows, vocab):
    spec = importlib.util.spec_from_file_location("vocab_parallel_step", PATH)
    ex = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(ex)
    student, teacher, hidden, tokens, sampled, advantage, dhidden = ex.main(
        ["--ranks", str(ranks), "--rows", str(rows), "--vocab", str(vocab), "--hidden", "128"])
    for d in dhidden[1:]:
        assert torch.equal(d, dhidden[0])
    f64 = lambda t: t.detach().double().cpu().numpy()
    x = np.concatenate([f64(t) for t in student.logits], 1)
    w = np.concatenate([f64(t) for t in student.weight], 0)
    logp, _ = vo.log_softmax(x)
    t = tokens.cpu().numpy()
    np.testing.assert_allclose(f64(student.logprobs), vo.logprobs(logp, t), atol=1e-5)
    np.testing.assert_allclose(f64(student.entropy), vo.entropy(logp), atol=1e-4)
    ids, vals = teacher.top_ids.cpu().numpy(), teacher.top.cpu().numpy()
    tx = np.concatenate([f64(v) for v in teacher.logits], 1)
    assert (ids == vo.top(tx, vo.log_softmax(tx)[0], ids.shape[1])[0]).all()
    np.testing.assert_allclose(f64(student.loss), vo.distill(x, 1.0, ids, vals, True)[0], atol=1e-4)
    ratio = np.exp(vo.logprobs(logp, t) - f64(sampled))
    a = vo.logprobs_grad(x, 1.0, t, -f64(advantage) * ratio / rows, -0.01 / rows)
    b = vo.distill_grad(x, 1.0, ids, vals, True, np.full(rows, 0.1 / rows))
    # three roundings to bf16 (each gradient, their sum), half a step of 2^-8 of the value each, and a product
    # of `vocab` terms rounded to bf16 once more
    tol = 2.0 ** -8 * ((2 * np.abs(a) + 2 * np.abs(b)) @ np.abs(w)) * 1.1
    got = f64(dhidden[0])
    want = (a + b) @ w
    tol += 2.0 ** -8 * ranks * np.abs(got).max() + 1e-6
    assert (np.abs(got - want) <= tol).all()

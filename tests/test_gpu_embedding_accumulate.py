"""Gradients of the table added to what its buffers hold, as where input and
output layer share it: token numbers that are sorted by counting passes, pieces
of more than 16 positions, runs of equal tokens over many pieces, rows of several
slices, and a workspace that a call writing zeros has used before.

Tolerance, u = 2^-24: c rows of a token in any order, (c + 1) u of the sum of
their sizes, the product with the scale and the sum with the old value, and half
a step of the type; entries without a token keep their bits."""
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
DT = {"f32": torch.float32, "bf16": torch.bfloat16}
HALF = {"f32": (2.0 ** -24, 2.0 ** -150), "bf16": (2.0 ** -8, 2.0 ** -134)}


def f64(t):
    return t.double().cpu().numpy()


def ids_of(kind, count, vocab):
    rng = np.random.default_rng(count)
    if kind == "one":
        return np.full(count, vocab // 2)
    if kind == "none":
        return np.where(rng.random(count) < 0.5, -1, vocab)
    t = np.minimum(np.exp(rng.random(count) * np.log(vocab + 1)).astype(np.int64) - 1, vocab - 1)
    t[rng.random(count) < 0.2] = -100
    return t


def check(kind, count, vocab, n, width, dtype, act, pad=0, scale=0.5):
    g = torch.Generator(device="cuda").manual_seed(count + width)
    ids = ids_of(kind, count, vocab).astype(np.int64)
    entries = ar.vocab_widths(vocab, n)
    go = torch.randn(count, width, generator=g, device="cuda").to(DT[act])
    flats = [torch.randn(e, width + pad, generator=g, device="cuda").to(DT[dtype]) for e in entries]
    grads, kept = [f[:, :width] for f in flats], [f.clone() for f in flats]
    sh = ar.EmbedShape(count, entries, width, dtype, out_dtype=act, grad_pitches=[width + pad] * n, scale=scale)
    ws = torch.full((ar.ar_embedding_workspace(sh) + 16,), 255, dtype=torch.uint8, device="cuda")
    t = torch.from_numpy(ids).cuda()
    scratch = [torch.empty(e, width + pad, dtype=DT[dtype], device="cuda")[:, :width] for e in entries]
    ar.ar_embedding_backward(go, sh, t, scratch, workspace=ws[:-16])
    ar.ar_embedding_backward(go, sh, t, grads, accumulate=True, workspace=ws[:-16])
    torch.cuda.synchronize()
    assert (ws[-16:] == 255).all()
    sums = lo.embedding_backward(f64(go), ids, vocab, scale)
    sizes = lo.embedding_backward(np.abs(f64(go)), ids, vocab, abs(scale))
    c = np.bincount(ids[(ids >= 0) & (ids < vocab)], minlength=vocab)[:, None]
    old = np.concatenate([f64(k[:, :width]) for k in kept])
    rel, tiny = HALF[dtype]
    # the buffer's sum, then the same sum written without accumulation, by the same call's order of adding
    for got, base in ((np.concatenate([f64(x) for x in grads]), old), (np.concatenate([f64(x) for x in scratch]), np.zeros_like(old))):
        want = base + sums
        tol = np.where(c == 0, 0.0, (c + 2) * U * sizes + 2 * U * (np.abs(base) + sizes) + 1.01 * (rel * np.abs(want) + tiny))
        err = np.abs(got - want)
        assert (err <= tol).all(), "%d off, worst %g of %g" % ((err > tol).sum(), err.max(), tol.flat[err.argmax()])
    untouched = torch.from_numpy(c[:, 0] == 0).cuda()
    for f, k, part in zip(flats, kept, untouched.split(entries)):
        assert torch.equal(f[part].view(torch.uint8), k[part].view(torch.uint8))
        assert torch.equal(f[:, width:], k[:, width:])


@pytest.mark.parametrize("kind", ["one", "none", "text"])
@pytest.mark.parametrize("count", [10240, 10241, 17000, 70001])
def test_counts(count, kind):
    check(kind, count, 3001, 8, 40, "f32", "bf16")
    check(kind, count, 1000, 3, 24, "bf16", "bf16", pad=3)


@pytest.mark.parametrize("kind", ["one", "text"])
@pytest.mark.parametrize("width", [513, 1500, 2100])
def test_rows_of_several_slices(width, kind):
    check(kind, 12000, 700, 4, width, "bf16", "bf16")
    check(kind, 12000, 700, 2, width, "f32", "bf16", pad=1, scale=1.0)

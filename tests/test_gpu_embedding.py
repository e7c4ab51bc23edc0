"""Embedding over a split vocabulary and its gradient on the GPU against the
64-bit definitions (oracle/layer.py).

Tolerances, u = 2^-24: a looked-up value is one fp32 product, rounded once more
to its type (no rounding at all where the scale is 1 and the type holds it);
a gradient adds the c rows of its token in any order, (c + 1) u of the sum of
their sizes, times the scale, plus what the buffer held, and is rounded to its type.
"""
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
DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
HALF = {"f32": (2.0 ** -24, 2.0 ** -150), "bf16": (2.0 ** -8, 2.0 ** -134), "f16": (2.0 ** -11, 2.0 ** -25)}


def f64(t):
    return t.detach().double().cpu().numpy()


def half(v, dtype):
    rel, tiny = HALF[dtype]
    return rel * np.abs(v) + tiny


class Table:
    """n rank buffers of rows `pad` elements apart from one another, `at` elements into their storage."""

    def __init__(self, entries, width, dtype, pad=0, at=0, fill=None, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed + 3)
        self.bufs, self.flats, self.width, self.pad, self.at = [], [], width, pad, at
        for e in entries:
            flat = torch.full((at + e * (width + pad) + 2,), 77.0, device="cuda").to(DT[dtype])
            view = flat[at:at + e * (width + pad)].view(e, width + pad)[:, :width]
            view.copy_(torch.randn(e, width, generator=g, device="cuda") if fill is None else torch.full((e, width), fill))
            self.bufs.append(view if e else None)
            self.flats.append(flat)

    def whole(self):
        return np.concatenate([f64(b) for b in self.bufs if b is not None], 0)

    def check(self):
        for b, flat in zip(self.bufs, self.flats):
            if b is not None:
                full = flat.clone()
                full.as_strided(b.shape, b.stride(), b.storage_offset()).fill_(77.0)
                assert (full == 77.0).all(), "wrote outside the rows"


def tokens_of(kind, count, vocab, seed=0):
    rng = np.random.default_rng(seed)
    if kind == "one":
        t = np.full(count, vocab // 2)
    elif kind == "none":
        t = np.where(rng.random(count) < 0.5, -1, vocab)
    elif kind == "text":                                      # few ids make up most of it, some are no token
        t = np.minimum(np.exp(rng.random(count) * np.log(vocab + 1)).astype(np.int64) - 1, vocab - 1)
        t[rng.random(count) < 0.2] = -100
    elif kind == "far":
        t = rng.integers(0, vocab, count)
        t[::3] = np.array([-(1 << 62), 1 << 40, (1 << 32) + 1])[rng.integers(0, 3, len(t[::3]))]
    else:
        t = rng.integers(0, vocab, count)
    return t.astype(np.int64)


def split(vocab, n):
    return [(r + 1) * vocab // n - r * vocab // n for r in range(n)]


def lookup(tokens, entries, width, dtype, out_dtype, pad=0, at=0, scale=1.0, stream=None):
    d = Table(entries, width, dtype, pad, at)
    sh = ar.EmbedShape(len(tokens), entries, width, dtype, out_dtype=out_dtype, pitches=[width + pad] * len(entries), scale=scale)
    flat = torch.full((len(tokens) * width + 6,), 5.0, device="cuda").to(DT[out_dtype])
    out = flat[3:3 + len(tokens) * width].view(len(tokens), width)
    t = torch.from_numpy(tokens).cuda()
    torch.cuda.synchronize()
    ar.ar_embedding(d.bufs, sh, t, out, stream=stream)
    torch.cuda.synchronize()
    assert (flat[:3] == 5).all() and (flat[3 + out.numel():] == 5).all()
    want = lo.embedding(d.whole(), tokens, float(np.float32(scale)))
    exact = scale == 1.0 and (dtype == out_dtype or out_dtype == "f32")
    assert (np.abs(f64(out) - want) <= (0 if exact else 1.01 * half(want, out_dtype) + U * np.abs(want))).all()


@pytest.mark.parametrize("out_dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("width", [1, 7, 8, 9, 100, 512, 513, 1024, 1500, 5003])
def test_lookup(width, dtype, out_dtype):
    lookup(tokens_of("text", 57, 101), split(101, 4), width, dtype, out_dtype)
    lookup(tokens_of("far", 40, 101), [0, 50, 0, 1, 50, 0], width, dtype, out_dtype, pad=3, at=1, scale=45.25)


@pytest.mark.parametrize("count", [1, 2, 5000])
@pytest.mark.parametrize("n", [1, 16, 17, 128])
def test_lookup_ranks(n, count):
    lookup(tokens_of("any", count, 1000), split(1000, n), 72, "bf16", "bf16")
    lookup(tokens_of("none", count, 60), split(60, n), 72, "bf16", "f32")


def test_lookup_copies_bits():
    table = torch.arange(1 << 16, device="cuda", dtype=torch.int32).to(torch.int16).view(torch.bfloat16).view(256, 256)
    out = torch.empty(256, 256, dtype=torch.bfloat16, device="cuda")
    ar.ar_embedding([table], ar.EmbedShape(256, [256], 256, "bf16"), torch.arange(256, device="cuda"), out)
    a, b = table.view(torch.int16), out.view(torch.int16)
    nan = table.isnan()
    assert torch.equal(a[~nan], b[~nan]) and out[nan].isnan().all()


def gradient(tokens, entries, width, dtype, out_dtype, pad=0, at=0, scale=1.0, accumulate=False, stream=None, seed=0):
    vocab, count = sum(entries), len(tokens)
    gen = torch.Generator(device="cuda").manual_seed(seed + 4)
    go = torch.randn(count, width, generator=gen, device="cuda").to(DT[out_dtype])
    d = Table(entries, width, dtype, pad, at, fill=None if accumulate else 9.0, seed=seed)
    old = d.whole() if accumulate else np.zeros((vocab, width))
    sh = ar.EmbedShape(count, entries, width, dtype, out_dtype=out_dtype, grad_pitches=[width + pad] * len(entries), scale=scale)
    ws = torch.full((ar.ar_embedding_workspace(sh) + 16,), 255, dtype=torch.uint8, device="cuda")
    t = torch.from_numpy(tokens).cuda()
    torch.cuda.synchronize()
    ar.ar_embedding_backward(go, sh, t, d.bufs, accumulate=accumulate, workspace=ws[:-16], stream=stream)
    torch.cuda.synchronize()
    assert (ws[-16:] == 255).all(), "wrote behind the workspace"
    d.check()
    s = float(np.float32(scale))
    sums = lo.embedding_backward(f64(go), tokens, vocab, s)
    sizes = lo.embedding_backward(np.abs(f64(go)), tokens, vocab, abs(s))
    ok = tokens[(tokens >= 0) & (tokens < vocab)]
    c = np.bincount(ok, minlength=vocab)[:, None]
    want = old + sums
    tol = (c + 2) * U * sizes + (2 * U * (np.abs(old) + sizes) if accumulate else 0) + 1.01 * half(want, dtype)
    tol = np.where(c == 0, 0.0, tol)
    err = np.abs(d.whole() - want)
    assert (err <= tol).all(), "%d off, worst %g of %g" % ((err > tol).sum(), err.max(), tol.flat[err.argmax()])
    return [b.clone() for b in d.bufs if b is not None]


@pytest.mark.parametrize("out_dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("width", [1, 7, 8, 9, 100, 512, 513, 1500])
def test_gradient(width, dtype, out_dtype):
    gradient(tokens_of("text", 77, 101), split(101, 4), width, dtype, out_dtype)
    gradient(tokens_of("far", 300, 101), [0, 50, 0, 1, 50, 0], width, dtype, out_dtype, pad=3, at=1, scale=45.25)
    gradient(tokens_of("text", 300, 101), split(101, 3), width, dtype, out_dtype, pad=1, accumulate=True, scale=0.5)


@pytest.mark.parametrize("kind", ["one", "none", "text", "any"])
@pytest.mark.parametrize("count", [1, 15, 16, 17, 63, 64, 65, 1000, 8191, 8192, 8193, 10240, 10241, 20000, 70001])
def test_gradient_counts(kind, count):
    gradient(tokens_of(kind, count, 3001, seed=count), split(3001, 8), 40, "f32", "bf16")


@pytest.mark.parametrize("vocab", [1, 2, 255, 2047, 2048, 2049, 131072, 1 << 20])
@pytest.mark.parametrize("count", [500, 9000])
def test_gradient_vocabularies(vocab, count):
    gradient(tokens_of("text", count, vocab, seed=1), split(vocab, 3), 8, "f32", "f32")


@pytest.mark.parametrize("n", [1, 16, 17, 128])
def test_gradient_ranks(n):
    gradient(tokens_of("text", 900, 500), split(500, n), 136, "bf16", "bf16")
    gradient(tokens_of("text", 900, 100), split(100, n), 136, "bf16", "bf16", accumulate=True)


def test_gradient_of_long_runs_and_wide_rows():
    gradient(tokens_of("one", 3000, 10), split(10, 2), 2100, "bf16", "bf16")
    gradient(tokens_of("text", 2000, 50), split(50, 2), 5003, "f32", "f16")
    gradient(tokens_of("text", 300_000, 30_000), split(30_000, 2), 24, "f32", "bf16")


def test_gradient_without_tokens():
    bufs = [torch.full((4, 16), 3.0, device="cuda"), torch.full((5, 16), 3.0, device="cuda")]
    sh = ar.EmbedShape(0, [4, 5], 16, "f32")
    ar.ar_embedding_backward(None, sh, None, bufs, accumulate=True)
    assert all((b == 3).all() for b in bufs)
    ar.ar_embedding_backward(None, sh, None, bufs)
    assert all((b == 0).all() for b in bufs)


def test_gradient_keeps_infinities_in_their_rows():
    go = torch.randn(40, 24, device="cuda")
    tokens = torch.arange(40, device="cuda") % 10
    go[3, 5], go[14, 6] = float("nan"), float("inf")
    out = torch.empty(10, 24, device="cuda")
    sh = ar.EmbedShape(40, [10], 24, "f32")
    ar.ar_embedding_backward(go, sh, tokens, [out], workspace=torch.empty(ar.ar_embedding_workspace(sh), dtype=torch.uint8, device="cuda"))
    assert out[3, 5].isnan() and out[4, 6] == float("inf")
    out[3, 5] = out[4, 6] = 0
    assert out.isfinite().all()


@pytest.mark.parametrize("count", [3000, 12000])
def test_gradient_bits_and_streams(count):
    t = tokens_of("text", count, 400)
    a = gradient(t, split(400, 4), 600, "bf16", "bf16", seed=2)
    b = gradient(t, split(400, 4), 600, "bf16", "bf16", seed=2, stream=torch.cuda.Stream())
    assert all(torch.equal(x, y) for x, y in zip(a, b))


def test_offsets_past_32_bits():
    """Table rows and tokens' rows that start past 2^32 bytes."""
    pitch, width = (1 << 29) + 8, 64
    flat = torch.zeros(5 * pitch + width, dtype=torch.bfloat16, device="cuda")
    table = torch.as_strided(flat, (6, width), (pitch, 1))
    table.copy_(torch.randn(6, width, device="cuda"))
    tokens = torch.tensor([5, 0, 5, 4], device="cuda")
    out = torch.empty(4, width, dtype=torch.bfloat16, device="cuda")
    ar.ar_embedding([table], ar.EmbedShape(4, [6], width, "bf16", pitches=[pitch]), tokens, out)
    assert torch.equal(out, table[tokens])
    sh = ar.EmbedShape(4, [6], width, "bf16", pitches=[pitch])
    ar.ar_embedding_backward(out, sh, tokens, [table],
                             workspace=torch.empty(ar.ar_embedding_workspace(sh), dtype=torch.uint8, device="cuda"))
    want = torch.zeros(6, width, device="cuda").index_add_(0, tokens, out.float()).bfloat16()
    assert torch.equal(table, want)
    del flat, table
    count = (1 << 32) // (4096 * 2) + 100
    big = torch.empty(count, 4096, dtype=torch.bfloat16, device="cuda").normal_()
    ids = torch.full((count,), -1, device="cuda")
    ids[-50:] = torch.arange(50, device="cuda") % 7
    sh = ar.EmbedShape(count, [10], 4096, "f32", out_dtype="bf16")
    grad = torch.empty(10, 4096, device="cuda")
    ar.ar_embedding_backward(big, sh, ids, [grad], workspace=torch.empty(ar.ar_embedding_workspace(sh), dtype=torch.uint8, device="cuda"))
    want = torch.zeros(10, 4096, dtype=torch.float64, device="cuda").index_add_(0, ids[-50:], big[-50:].double())
    assert (grad.double() - want).abs().max() < 20 * U * 60

"""The vocabulary reductions on the GPU against their 64-bit definitions
(oracle/vocab.py) on the same logits.

Tolerances, u = 2^-24 (half a step of fp32).  A lane adds its logits one after
the other, at most `seq` of them, then log2-many partial sums: the sum is off
by at most (seq + 32) u of itself.  A term 2^t carries the rounding of t (|t|
u, up to the two roundings of the scale and the product) and of 2^t (2 u).  So
  ln p_v       (seq + 32 + 4 |z_v - m|) u  (m: the largest z; the kernel's
               reference is within 6 of it, hence a constant of 32, and the
               mean of |z - m| under p, which rounds the sum, is below ln V < 14),
  H            the same for its two sums, whose size is at most 1 + ln V,
  p            that of ln p, relative; p below 2^-126 may be flushed to 0,
  gradients    the parts' errors added up, plus half a step of the type.
"""
from __future__ import annotations

import math

import numpy as np
import pytest

from oracle import vocab as vo

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)
ar = pytest.importorskip("reduce_scatter_amd")

U = 2.0 ** -24
DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
NEG = float("-inf")


class Data:
    """Logits x [rows, V] split into rank buffers with padded rows (NaN
    between them) that start ``offset`` elements into their storage."""

    def __init__(self, x, widths, dtype, temperature=1.0, pad=0, offset=0, gpad=0, goffset=0):
        self.rows, self.vocab = x.shape
        assert sum(widths) == self.vocab
        self.dtype, self.T = dtype, temperature
        self.xt = x.to(DT[dtype])
        self.x = self.xt.double().numpy()
        self.bufs, self.grads, self.store, self.gstore = [], [], [], []
        pitches, gpitches, c = [], [], 0
        for w in widths:
            for view, store, pp, oo, fill in ((self.bufs, self.store, pad, offset, float("nan")),
                                              (self.grads, self.gstore, gpad, goffset, 77.0)):
                flat = torch.full((oo + self.rows * (w + pp) + 1,), fill, dtype=DT[dtype], device="cuda")
                view.append(flat[oo:oo + self.rows * (w + pp)].view(self.rows, w + pp)[:, :w])
                store.append(flat)
            self.bufs[-1].copy_(self.xt[:, c:c + w])
            pitches.append(w + pad)
            gpitches.append(w + gpad)
            c += w
        self.widths = widths
        self.shape = ar.VocabShape(self.rows, widths, dtype, pitches=pitches, grad_pitches=gpitches,
                                   temperature=temperature)
        tile = 64 * 4 * (4 if dtype == "f32" else 8)
        waves = 1
        tiles = sum(-(-w // tile) for w in widths)
        while waves < 16 and waves * 2 <= tiles:
            waves *= 2
        self.seq = -(-tiles // waves) * (tile // 64)
        self.logp, self.empty = vo.log_softmax(self.x, temperature)
        with np.errstate(all="ignore"):
            m = np.where(self.empty, 0.0, np.max(np.where(np.isnan(self.x), NEG, self.x), 1))[:, None]
            self.dist = np.abs((self.x - m) / temperature)               # |z - m|

    def workspace(self, k=0):
        return torch.empty(ar.ar_vocab_workspace(self.shape, k), dtype=torch.uint8, device="cuda")

    def lp_tol(self, dist):
        return (self.seq + 32 + 4 * dist) * U

    def h_tol(self):
        return 2 * (self.seq + 64) * U * (1 + math.log(self.vocab + 1))

    def gather_grads(self):
        c = 0
        for g, store, w in zip(self.grads, self.gstore, self.widths):
            full = store.clone()
            full.as_strided(g.shape, g.stride(), g.storage_offset()).fill_(77.0)
            assert (full == 77.0).all(), "wrote outside the rows"
            c += w
        return torch.cat([g.double().cpu() for g in self.grads], 1).numpy()


def close(got, want, tol, what):
    got, want = np.asarray(got, dtype=np.float64), np.asarray(want)
    tol = np.broadcast_to(np.asarray(tol, dtype=np.float64), want.shape)
    fin = np.isfinite(want)
    assert (np.isnan(got) == np.isnan(want)).all(), "%s: NaN in other places" % what
    inf = np.isinf(want)
    assert (got[inf] == want[inf]).all(), "%s: infinities differ" % what
    err = np.abs(got[fin] - want[fin])
    bad = ~(err <= tol[fin])
    if bad.any():
        i = np.argmax(err - tol[fin])
        raise AssertionError("%s: %d of %d off; worst got %r want %r, tolerance %g"
                             % (what, bad.sum(), bad.size, got[fin][i], want[fin][i], tol[fin][i]))


def half_step(g, dtype):
    eps, tiny = {"f32": (2.0 ** -24, 2.0 ** -149), "bf16": (2.0 ** -9, 2.0 ** -133),
                 "f16": (2.0 ** -12, 2.0 ** -24)}[dtype]
    return 2 * eps * np.abs(g) + tiny


def check_logprobs(d, targets, k=0, entropy=True, stream=None):
    f = lambda *s: torch.full(s, 55.0, device="cuda")
    t = torch.from_numpy(targets).cuda()
    lp, h, saved = f(d.rows), f(d.rows), f(d.rows, 4)
    top, ids = f(d.rows, max(k, 1)), torch.full((d.rows, max(k, 1)), 55, dtype=torch.int64, device="cuda")
    torch.cuda.synchronize()                              # the fills are on torch's stream
    ar.ar_logprobs(d.bufs, d.shape, t, lp, entropy=h if entropy else None, top_k=k, top_logprobs=top if k else None,
                   top_ids=ids if k else None, saved=saved, workspace=d.workspace(k), stream=stream)
    torch.cuda.synchronize()
    has = (targets >= 0) & (targets < d.vocab)
    at = np.where(has, targets, 0)
    dist = np.where(np.isfinite(d.dist), d.dist, 0.0)
    close(lp.cpu(), vo.logprobs(d.logp, targets), np.where(has, d.lp_tol(dist[np.arange(d.rows), at]), 0), "logprobs")
    if entropy:
        close(h.cpu(), vo.entropy(d.logp), d.h_tol(), "entropy")
    if k:
        want_ids, want = vo.top(d.x, d.logp, k)
        assert (ids.cpu().numpy() == want_ids).all(), "top ids"
        near = np.take_along_axis(dist, np.maximum(want_ids, 0), 1)
        close(top.cpu(), want, d.lp_tol(near), "top logprobs")
    return saved


def logprob_grad_tol(d, want, gl, gh):
    with np.errstate(all="ignore"):
        p = np.exp(d.logp)
        eps = d.lp_tol(np.where(np.isfinite(d.dist), d.dist, 0.0))
        lph = np.where(p == 0, 0.0, np.abs(d.logp) + d.h_tol())
        H = vo.entropy(d.logp)[:, None]
        gl, gh = np.abs(gl)[:, None], np.abs(gh)[:, None]
        t = p * (gl + gh * (lph + H + 1)) * 2 * eps + p * gh * (eps + d.h_tol()) + 8 * U * gl * (np.abs(want) > 0)
        t = t + (gl + gh) * 2.0 ** -120
    return np.nan_to_num(t / d.T, nan=0.0) + half_step(want, d.dtype)


def check_logprobs_grad(d, targets, gl, gh, saved, fused):
    t = torch.from_numpy(targets).cuda()
    a = torch.from_numpy(gl.astype(np.float32)).cuda()
    e = torch.from_numpy(gh.astype(np.float32)).cuda() if gh is not None else None
    hh = gh if gh is not None else np.zeros(d.rows)
    if fused:
        lp = torch.full((d.rows,), 55.0, device="cuda")
        ar.ar_logprobs_grad(d.bufs, d.grads, d.shape, t, lp, grad_logprobs=a, grad_entropy=e, workspace=d.workspace())
        has = (targets >= 0) & (targets < d.vocab)
        dist = np.where(np.isfinite(d.dist), d.dist, 0.0)[np.arange(d.rows), np.where(has, targets, 0)]
        close(lp.cpu(), vo.logprobs(d.logp, targets), np.where(has, d.lp_tol(dist), 0), "logprobs of the fused call")
    else:
        ar.ar_logprobs_backward(d.bufs, d.grads, d.shape, t, saved, grad_logprobs=a, grad_entropy=e)
    torch.cuda.synchronize()
    gl32, gh32 = gl.astype(np.float32).astype(np.float64), hh.astype(np.float32).astype(np.float64)
    want = vo.logprobs_grad(d.x, d.T, targets, gl32, gh32)
    close(d.gather_grads(), want, logprob_grad_tol(d, want, gl32, gh32), "gradient")


def teacher_lists(rng, rows, vocab, k, tail):
    ids = np.stack([rng.permutation(max(vocab, k))[:k] for _ in range(rows)]).astype(np.int64)   # past V: padding
    vals = rng.standard_normal((rows, k)) * 2
    if tail:
        mass = rng.uniform(0.3, 0.999, (rows, 1))
        vals = vals - np.log(np.exp(vals).sum(1, keepdims=True)) + np.log(mass)
    return ids, vals.astype(np.float32)


def distill_tols(d, ids, vals, tail, g=None):
    q, lq, valid, qt, live = vo.teacher(ids, vals, d.vocab, tail, d.T)
    loss, lpk, lt = vo.distill(d.x, d.T, ids, vals, tail)
    k = ids.shape[1]
    dist = np.where(np.isfinite(d.dist), d.dist, 0.0)
    with np.errstate(all="ignore"):
        dk = np.take_along_axis(dist, np.where(valid, ids, 0), 1)
        alq, alp = np.nan_to_num(np.abs(lq), posinf=0.0), np.nan_to_num(np.abs(lpk), posinf=0.0)
        eq = (4 * alq + k + 16) * U                                     # relative error of q
        t = (q * (eq * (1 + alq + alp) + d.lp_tol(dk) + (k + 8) * U * (alq + alp))).sum(1)
        dqt = ((q * eq).sum(1) + (k + 8) * U) * (qt > 0)
        alt = np.nan_to_num(np.abs(lt), posinf=0.0)
        lqt = np.nan_to_num(np.abs(np.log(qt)), posinf=0.0)
        # the unlisted mass stands |ln p_t| from the row's sum
        t = t + qt * (d.lp_tol(alt) * 2 + 8 * U * (alt + lqt)) + dqt * (1 + alt + lqt)
        if g is None:
            return t
        p = np.exp(d.logp)
        eps = d.lp_tol(dist)
        dense_q, dense_e = np.zeros_like(p), np.zeros_like(p)
        r, kk = np.nonzero(valid)
        np.add.at(dense_q, (r, ids[r, kk]), q[r, kk])
        np.add.at(dense_e, (r, ids[r, kk]), (q * eq)[r, kk])
        rest = np.where(vo._unlisted(ids, valid, d.vocab) & np.isfinite(lt)[:, None], d.logp - lt[:, None], NEG)
        cond = np.exp(rest)
        big = 2 * p * (eps + (q * eq).sum(1)[:, None] + dqt[:, None]) + dense_e * 2 + 4 * U * dense_q
        big += cond * (qt * 2 * (d.lp_tol(alt) + 8 * U) + dqt)[:, None] + 2 * cond * qt[:, None] * eps
        return t, np.abs(g)[:, None] / d.T * (big + 2.0 ** -120)


def check_distill(d, ids, vals, tail, g, mode):
    f = lambda *s: torch.full(s, 55.0, device="cuda")
    i, v, gg = torch.from_numpy(ids).cuda(), torch.from_numpy(vals).cuda(), torch.from_numpy(g.astype(np.float32)).cuda()
    loss, saved = f(d.rows), f(d.rows, 4)
    g = g.astype(np.float32).astype(np.float64)
    want = vo.distill(d.x, d.T, ids, vals, tail)[0]
    tol, gtol = distill_tols(d, ids, vals, tail, g)
    if mode == "fused":
        ar.ar_distill_grad(d.bufs, d.grads, d.shape, i, v, loss, tail=tail, grad_loss=gg, workspace=d.workspace())
    else:
        ar.ar_distill(d.bufs, d.shape, i, v, loss, tail=tail, saved=saved, workspace=d.workspace())
        ar.ar_distill_backward(d.bufs, d.grads, d.shape, i, v, saved, tail=tail, grad_loss=gg)
    torch.cuda.synchronize()
    close(loss.cpu(), want, tol, "loss")
    wg = vo.distill_grad(d.x, d.T, ids, vals, tail, g)
    close(d.gather_grads(), wg, np.nan_to_num(gtol) + half_step(wg, d.dtype), "gradient")


def logits(rng, rows, vocab, scale=2.5):
    return torch.from_numpy(rng.standard_normal((rows, vocab)).astype(np.float32) * np.float32(scale))


# the smallest vocabularies, one vector and one tile more or less, several tiles, ranks of unequal and no width,
# the large pointer table, rows split over workgroups (few rows, many tiles) and not
SHAPES = [
    (1, [1]), (3, [2]), (2, [7, 0, 2]), (5, [8]), (4, [9, 8]), (2, [0, 0, 65]), (3, [511, 513]), (2, [2048]),
    (3, [2049, 2047]), (2, [4101]), (300, [1000, 1001]), (260, [5000, 5003, 4999]), (1, [50021]),
    (2, [33000, 20, 0, 9001]), (3, [40000] * 5), (2, [37] * 17), (2, [3001] * 40 + [0] * 88), (1, [1]* 128),
    (7, [70001]),
    # the largest vocabulary; a row in all of a workgroup's registers, with few rows and with many
    (2, [1 << 20]), (20, [131072]), (257, [33000]),
]


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("i", range(len(SHAPES)))
def test_logprobs(i, dtype):
    rows, widths = SHAPES[i]
    rng = np.random.default_rng([11, i])
    pad, off = [(0, 0), (3, 1), (8, 0), (1, 3)][i % 4]
    d = Data(logits(rng, rows, sum(widths)), widths, dtype, [1.0, 0.7, 1.9][i % 3], pad, off, gpad=[0, 2, 8][i % 3],
             goffset=i % 2)
    t = rng.integers(0, d.vocab, rows)
    if rows > 2:
        t[1], t[2] = -100, d.vocab                        # no token, twice
    k = [0, 1, 5, 20, 64][i % 5]
    saved = check_logprobs(d, t, k)
    check_logprobs(d, t, [7, 64, 0][i % 3], entropy=False)
    gl, gh = rng.standard_normal(rows), rng.standard_normal(rows) * 0.3
    check_logprobs_grad(d, t, gl, gh, saved, False)
    check_logprobs_grad(d, t, gl, None, saved, False)
    check_logprobs_grad(d, t, gl, gh, None, True)
    check_logprobs_grad(d, t, gl, None, None, True)


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("tail", [False, True])
@pytest.mark.parametrize("i", range(len(SHAPES)))
def test_distill(i, tail, dtype):
    rows, widths = SHAPES[i]
    rng = np.random.default_rng([12, i])
    pad, off = [(0, 0), (3, 1), (8, 0), (1, 3)][i % 4]
    d = Data(logits(rng, rows, sum(widths)), widths, dtype, [1.0, 0.7, 1.9][i % 3], pad, off, gpad=[0, 2, 8][i % 3],
             goffset=i % 2)
    k = [1, 3, 64, 65, 256][i % 5]
    ids, vals = teacher_lists(rng, rows, d.vocab, k, tail)
    if rows > 2:
        ids[1, :] = -1                                    # no teacher
        ids[2, 0] = d.vocab + 5                           # padding
    g = rng.standard_normal(rows)
    if rows > 3:
        g[3] = 0.0
    check_distill(d, ids, vals, tail, g, "fused")
    check_distill(d, ids, vals, tail, g, "split")


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("rows, widths", [(6, [700, 701]), (6, [60000])])
def test_masks(rows, widths, dtype):
    rng = np.random.default_rng(13)
    x = logits(rng, rows, sum(widths))
    v = x.shape[1]
    low = torch.finfo(DT[dtype]).min
    x[0, torch.rand(v) < 0.5] = NEG                       # half the row masked
    x[1] = NEG                                            # nothing left
    x[2] = low                                            # the lowest value everywhere: uniform
    x[3, :] = low
    x[3, v // 2] = 3.0                                    # one entry left
    x[4, :] = NEG
    x[4, v - 1] = -5.0
    x[5, : v // 3] = low
    d = Data(x, widths, dtype, 1.0, 1, 0)
    t = np.array([int(np.argmax(d.x[0])), 3, 5, v // 2, 2, v - 1])
    saved = check_logprobs(d, t, 9)
    gl, gh = rng.standard_normal(rows), rng.standard_normal(rows)
    check_logprobs_grad(d, t, gl, gh, saved, False)
    check_logprobs_grad(d, t, gl, gh, None, True)
    ids = np.stack([np.argsort(-np.where(np.isfinite(r), r, -1e30), kind="stable")[:5] for r in d.x]).astype(np.int64)
    vals = np.log(np.array([0.4, 0.2, 0.1, 0.1, 0.05], dtype=np.float32))[None].repeat(rows, 0)
    # rows whose listed entries are all possible
    keep = [0, 2, 5]
    d2 = Data(x[keep], widths, dtype, 1.0, 1, 0)
    for tail in (False, True):
        for mode in ("fused", "split"):
            check_distill(d2, ids[keep], vals[keep], tail, gl[keep], mode)


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
def test_not_a_number_and_infinity(dtype):
    rng = np.random.default_rng(14)
    x = logits(rng, 5, 3000)
    x[0, 17] = float("nan")
    x[1, 2999] = float("inf")
    x[2, :] = float("nan")
    x[3, 40] = float("nan")
    d = Data(x, [1500, 1500], dtype)
    t = np.array([5, 6, 7, -100, 9])
    saved = check_logprobs(d, t, 4)
    gl, gh = np.ones(5), np.zeros(5)                      # row 3: upstream zero, so is its gradient
    check_logprobs_grad(d, t, gl, gh, saved, False)
    check_logprobs_grad(d, t, gl, None, None, True)
    ids = np.array([[1, 2], [3, 4], [5, 6], [-1, -1], [8, 9]])
    vals = np.log(np.full((5, 2), 0.3, dtype=np.float32))
    for tail in (False, True):
        check_distill(d, ids, vals, tail, np.ones(5), "fused")
        check_distill(d, ids, vals, tail, np.ones(5), "split")


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("rows", [2, 300])
def test_top_order(dtype, rows):
    """Ties, ascending and descending rows, all equal, both zeros."""
    v = 20000
    base = torch.arange(v, dtype=torch.float32)
    kinds = [base / 64, -base / 64, torch.zeros(v), torch.where(base % 2 == 0, -0.0, 0.0),
             torch.where(base % 3 == 0, 1.0, 0.0), -(base % 7), (base * 7919 % 20011) / 1000]
    x = torch.stack([kinds[(r + rows) % len(kinds)] for r in range(rows)])
    d = Data(x, [v // 2, v - v // 2], dtype)
    for k in (1, 2, 63, 64):
        check_logprobs(d, np.zeros(rows, dtype=np.int64), k)


@pytest.mark.parametrize("tail", [False, True])
@pytest.mark.parametrize("rows", [4, 300])
def test_sharp_student_and_odd_lists(rows, tail):
    """Listed entries far above the rest (the unlisted mass is e^-95 and
    less), repeated ids, entries of probability zero, every entry listed."""
    rng = np.random.default_rng(15)
    x = logits(rng, rows, 9000)
    ids = np.stack([rng.permutation(9000)[:6] for _ in range(rows)]).astype(np.int64)
    x[torch.arange(rows)[:, None], torch.from_numpy(ids)] = 110.0
    vals = np.log(np.array([0.3, 0.2, 0.1, 0.1, 0.05, 0.05], dtype=np.float32))[None].repeat(rows, 0)
    ids[1, 3] = ids[1, 0]
    vals[2, 1] = NEG
    d = Data(x, [9000], "f32")
    g = rng.standard_normal(rows)
    check_distill(d, ids, vals, tail, g, "fused")
    check_distill(d, ids, vals, tail, g, "split")
    small = Data(logits(rng, 3, 6), [4, 2], "f32")
    every = np.stack([rng.permutation(6) for _ in range(3)]).astype(np.int64)
    full = np.log(np.full((3, 6), 1 / 6, dtype=np.float32))
    check_distill(small, every, full, tail, np.ones(3), "fused")


def test_in_place_equals_apart():
    rng = np.random.default_rng(16)
    for rows, widths in ((300, [5000, 5001]), (2, [60000])):
        for dtype in ("bf16", "f32"):
            d = Data(logits(rng, rows, sum(widths)), widths, dtype)
            t = torch.from_numpy(rng.integers(0, d.vocab, rows)).cuda()
            gl = torch.randn(rows, device="cuda")
            ids = torch.from_numpy(np.stack([rng.permutation(d.vocab)[:40] for _ in range(rows)])).cuda()
            vals = torch.log(torch.full((rows, 40), 0.02, device="cuda"))
            for f in (lambda x, g: ar.ar_logprobs_grad(x, g, d.shape, t, grad_logprobs=gl, workspace=d.workspace()),
                      lambda x, g: ar.ar_distill_grad(x, g, d.shape, ids, vals, tail=True, grad_loss=gl,
                                                      workspace=d.workspace())):
                f(d.bufs, d.grads)
                work = [b.clone() for b in d.bufs]
                f(work, work)
                torch.cuda.synchronize()
                for a, b in zip(work, d.grads):
                    assert torch.equal(a, b)


def test_columns_of_one_buffer():
    """Rank buffers and gradients as column blocks of one [rows, V] tensor."""
    rng = np.random.default_rng(17)
    x = logits(rng, 9, 4500).cuda()
    g = torch.full_like(x, 55.0)
    cut = [0, 1100, 1101, 4500]
    bufs = [x[:, cut[i]:cut[i + 1]] for i in range(3)]
    grads = [g[:, cut[i]:cut[i + 1]] for i in range(3)]
    sh = ar.VocabShape(9, [1100, 1, 3399], "f32", pitches=[4500] * 3)
    t = torch.from_numpy(rng.integers(0, 4500, 9)).cuda()
    gl = torch.randn(9, device="cuda")
    ar.ar_logprobs_grad(bufs, grads, sh, t, grad_logprobs=gl)
    one = torch.empty_like(x)
    ar.ar_logprobs_grad([x], [one], ar.VocabShape(9, [4500], "f32"), t, grad_logprobs=gl)
    want = vo.logprobs_grad(x.cpu().double().numpy(), 1.0, t.cpu().numpy(), gl.cpu().double().numpy(), 0.0)
    for got in (g, one):
        np.testing.assert_allclose(got.cpu().numpy(), want, rtol=1e-4, atol=1e-6)


def test_equal_calls_equal_bits_on_another_stream():
    rng = np.random.default_rng(18)
    for rows, widths in ((513, [9000, 8999]), (2, [120001])):
        d = Data(logits(rng, rows, sum(widths)), widths, "bf16")
        t = rng.integers(0, d.vocab, rows)
        outs = []
        for stream in (None, torch.cuda.Stream(), torch.cuda.Stream()):
            torch.cuda.synchronize()
            saved = check_logprobs(d, t, 10, stream=stream)
            outs.append(saved.clone())
        assert torch.equal(outs[0], outs[1]) and torch.equal(outs[0], outs[2])


@pytest.mark.parametrize("rows, widths", [(300, [4000, 4001]), (2, [60000])])
def test_graph_replay(rows, widths):
    """Captured once, replayed over changed inputs, with eager work between."""
    rng = np.random.default_rng(19)
    d = Data(logits(rng, rows, sum(widths)), widths, "bf16")
    t = torch.from_numpy(rng.integers(0, d.vocab, rows)).cuda()
    ids, vals = teacher_lists(rng, rows, d.vocab, 20, True)
    ids, vals = torch.from_numpy(ids).cuda(), torch.from_numpy(vals).cuda()
    gl = torch.randn(rows, device="cuda")
    x, g = ar.pointers(d.bufs), ar.pointers(d.grads)
    g2 = [torch.empty_like(b) for b in d.grads]
    sh2 = ar.VocabShape(rows, widths, "bf16")
    ws, ws2 = d.workspace(5), d.workspace()
    f = lambda *s: torch.zeros(s, device="cuda")
    lp, top, tid, loss, saved = f(rows), f(rows, 5), torch.zeros(rows, 5, dtype=torch.int64, device="cuda"), f(rows), f(rows, 4)

    def step():
        ar.ar_logprobs(x, d.shape, t, lp, top_k=5, top_logprobs=top, top_ids=tid, saved=saved, workspace=ws)
        ar.ar_logprobs_backward(x, g, d.shape, t, saved, grad_logprobs=gl)
        ar.ar_distill_grad(x, g2, sh2, ids, vals, loss, tail=True, grad_loss=gl, workspace=ws2)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for i in range(4):
        for b in d.bufs:
            b.copy_(torch.randn(b.shape, device="cuda") * 2)
        step()
        torch.cuda.synchronize()
        want = [v.clone() for v in (lp, top, tid, loss, *d.grads, *g2)]
        for v in (lp, top, tid, loss, *d.grads, *g2):
            v.fill_(7)
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(want, (lp, top, tid, loss, *d.grads, *g2)):
            assert torch.equal(a, b)


def test_offsets_past_32_bits():
    """Row starts more than 2^32 bytes into a buffer: a few rows far apart."""
    pitch, rows = (1 << 29) + 5, 6
    flat = torch.empty(pitch * (rows - 1) + 900, dtype=torch.bfloat16, device="cuda")
    x = torch.as_strided(flat, (rows, 900), (pitch, 1))
    rng = np.random.default_rng(20)
    x.copy_(logits(rng, rows, 900).to(torch.bfloat16))
    sh = ar.VocabShape(rows, [900], "bf16", pitches=[pitch])
    t, lp = torch.from_numpy(rng.integers(0, 900, rows)).cuda(), torch.empty(rows, device="cuda")
    gl = torch.randn(rows, device="cuda")
    want = vo.logprobs_grad(x.double().cpu().numpy(), 1.0, t.cpu().numpy(), gl.double().cpu().numpy(), 0.0)
    logp, _ = vo.log_softmax(x.double().cpu().numpy())
    ar.ar_logprobs_grad([x], [x], sh, t, lp, grad_logprobs=gl)           # in place
    torch.cuda.synchronize()
    np.testing.assert_allclose(lp.cpu().numpy(), vo.logprobs(logp, t.cpu().numpy()), rtol=0, atol=(64 + 32 + 80) * U)
    np.testing.assert_allclose(x.double().cpu().numpy(), want, rtol=2.0 ** -8, atol=1e-7)

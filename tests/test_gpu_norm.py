"""Reduction with residual and RMS norm on the GPU against the 64-bit
definitions (oracle/layer.py) on the same inputs.

Tolerances, u = 2^-24 (half a step of fp32), A = sum of |terms| of an element:
  s      n roundings of partial sums of at most A each: n u A; `summed` half a
         step of its type more
  sq     a lane adds at most 16 squares in turn, then at most 10 lane and wave
         steps: 32 u relative with the squares' own roundings, and 2 sum |s| ds
  rstd   half of sq's, one step of the reciprocal root, the division, eps: 4 u
  y      |rstd w| ds, and |y| times rstd's and 4 roundings (offset + w counted
         by its parts' size)
  out8   half a step of e4m3: 2^-4 of the value, or 2^-10 of the scale
  h, u   products of rounded factors: 3 u of |h|, |u| (|offset| + |w|)
  dx     rstd (|u| 4 u + |h| dc + 3 u |h c|), dc = (32 + 6) u mean |u h|
  dw     any order of adding `rows` terms: (rows + 8) u sum |g h|
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
GUARD = 77.0


def f64(t):
    return t.detach().double().cpu().numpy()


class Out:
    """[rows, width] in a larger buffer; what lies around it has to stay."""

    def __init__(self, *shape, dtype=torch.float32, offset=3):
        n = int(np.prod(shape))
        self.flat = torch.full((n + 2 * offset,), GUARD, device="cuda").to(dtype)
        self.offset, self.t = offset, self.flat[offset:offset + n].view(*shape)

    def check(self):
        around = torch.cat([self.flat[:self.offset], self.flat[self.offset + self.t.numel():]]).float()
        assert (around == float(torch.tensor(GUARD).to(self.flat.dtype))).all(), "wrote around the output"


def spaced(x, pad, offset=0):
    """The same rows with NaN between them, `offset` elements into a buffer."""
    rows, width = x.shape
    flat = torch.full((offset + rows * (width + pad),), float("nan"), device="cuda").to(x.dtype)
    view = flat[offset:].view(rows, width + pad)[:, :width]
    view.copy_(x)
    return view


def close(got, want, tol, what):
    got, want = np.asarray(got, dtype=np.float64), np.asarray(want, dtype=np.float64)
    tol = np.broadcast_to(np.asarray(tol, dtype=np.float64), want.shape)
    assert (np.isnan(got) == np.isnan(want)).all(), "%s: NaN in other places" % what
    inf = np.isinf(want)
    assert (got[inf] == want[inf]).all(), "%s: infinities differ" % what
    fin = np.isfinite(want)
    err = np.abs(got[fin] - want[fin])
    bad = ~(err <= tol[fin])
    if bad.any():
        i = np.argmax(err / np.maximum(tol[fin], 1e-300))
        raise AssertionError("%s: %d of %d off; worst got %r want %r, tolerance %g"
                             % (what, bad.sum(), bad.size, got[fin][i], want[fin][i], tol[fin][i]))


def half(v, dtype):
    rel, tiny = HALF[dtype]
    return rel * np.abs(v) + tiny


def rounded(v, dtype):
    """64-bit values past the type's range as the type holds them (infinities)."""
    top = {"f32": 3.4028235677973366e38, "bf16": 3.3961775292304601e38, "f16": 65520.0}[dtype]
    with np.errstate(all="ignore"):
        return np.where(np.abs(v) >= top, np.sign(v) * np.inf, v)


class Norm:
    def __init__(self, rows, width, n, dtype, weight="same", residual=True, pad=0, offset=0.0, eps=1e-6, group=0, at=0, seed=0,
                 scale=1.0):
        g = torch.Generator(device="cuda").manual_seed(seed + 1)
        randn = lambda *s: torch.randn(s, generator=g, device="cuda")
        self.rows, self.width, self.n, self.dtype, self.group = rows, width, n, dtype, group
        self.wtype = dtype if weight == "same" else weight
        self.x = [spaced((randn(rows, width) * 0.5 * scale).to(DT[dtype]), pad, at) for _ in range(n)]
        self.residual = (randn(rows, width) * scale).to(DT[dtype]) if residual else None
        self.w = (randn(width) * 0.3 + 1 - offset).to(DT[self.wtype])
        self.offset, self.eps = offset, eps
        self.shape = ar.NormShape(rows, width, n, dtype, pitches=[width + pad] * n, weight_dtype=self.wtype, eps=eps,
                                  offset=offset, group=group)

    def expect(self):
        xs = [f64(x) for x in self.x] + ([f64(self.residual)] if self.residual is not None else [])
        with np.errstate(all="ignore"):
            ds = len(xs) * U * sum(np.abs(x) for x in xs)
            s, rstd, y = lo.reduce_norm([f64(x) for x in self.x], f64(self.w), None if self.residual is None else f64(self.residual),
                                        self.eps, self.offset)
            total = np.maximum((s * s).sum(1), 1e-300)
            dr = np.nan_to_num(0.5 * (32 * U + 2 * (np.abs(s) * ds).sum(1) / total) + 5 * U)
            wabs = np.abs(f64(self.w)) + abs(self.offset)
            dy = np.nan_to_num(np.abs(rstd)[:, None] * wabs * ds + (dr[:, None] + 5 * U) * np.abs(rstd[:, None] * s) * wabs)
        return s, ds, rstd, dr, y, dy

    def run(self, out=True, eight=False, rstd=True, stream=None):
        r, w = self.rows, self.width
        o = {"summed": Out(r, w, dtype=DT[self.dtype]) if self.residual is not None else None,
             "out": Out(r, w, dtype=DT[self.dtype], offset=5) if out else None, "rstd": Out(r) if rstd else None,
             "out8": Out(r, w, dtype=torch.uint8) if eight else None,
             "scales": Out(r, self.shape.groups) if eight else None}
        torch.cuda.synchronize()
        ar.ar_reduce_norm(self.x, self.shape, self.w, residual=self.residual, stream=stream,
                          **{k: v.t if v else None for k, v in o.items()})
        torch.cuda.synchronize()
        for v in o.values():
            if v:
                v.check()
        return {k: v.t for k, v in o.items() if v}

    def check(self, **kw):
        o = self.run(**kw)
        s, ds, rstd, dr, y, dy = self.expect()
        with np.errstate(all="ignore"):
            if "rstd" in o:
                close(f64(o["rstd"]), rstd, (dr + U) * np.abs(rstd) + 2.0 ** -149, "rstd")
            if "summed" in o:
                close(f64(o["summed"]), rounded(s, self.dtype), ds + half(s, self.dtype) * 1.01, "summed")
            if "out" in o:
                close(f64(o["out"]), rounded(y, self.dtype), dy + half(y, self.dtype) * 1.01, "out")
            if "out8" in o:
                want = lo.scales(y, self.group)
                size = self.group or self.width
                worst = np.stack([dy[:, c:c + size].max(1) for c in range(0, self.width, size)], 1)
                close(f64(o["scales"]), want, worst / 448 + 4 * U * np.abs(want), "scales")
                each = np.repeat(f64(o["scales"]), size, 1)[:, :self.width]
                q = f64(o["out8"].view(torch.float8_e4m3fn))
                close(q * each, np.where(np.isnan(each), np.nan, y), dy + (2.0 ** -4 + 4 * U) * np.abs(y) + 2.0 ** -10 * each, "out8")
        return o


WIDTHS = [1, 5, 7, 8, 9, 64, 120, 128, 129, 500, 512, 513, 1000, 4096, 5003, 8192, 8193, 16384]


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("width", WIDTHS)
def test_widths(width, dtype):
    Norm(19, width, 3, dtype, seed=width).check()
    Norm(3, width, 2, dtype, group=32, weight="f32", seed=width).check(eight=True)
    Norm(2, width, 2, dtype, pad=3, at=1, offset=1.0, seed=width).check(eight=True)


@pytest.mark.parametrize("n", [1, 2, 3, 4, 5, 7, 8, 9, 15, 16, 17, 31, 128])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_ranks(n, dtype):
    Norm(5, 1030, n, dtype, seed=n, pad=n % 3).check()
    Norm(5, 96, n, dtype, seed=n, residual=False).check()
    Norm(2, 9000, n, dtype, seed=n).check()


@pytest.mark.parametrize("group", [0, 32, 64, 128, 256, 512])
@pytest.mark.parametrize("width", [40, 128, 300, 1000, 4096, 9001])
def test_groups(width, group):
    for dtype in ("bf16", "f32"):
        Norm(33, width, 2, dtype, group=group, seed=group).check(eight=True, out=dtype == "f32", rstd=False)


@pytest.mark.parametrize("rows", [1, 2, 15, 16, 17, 1000, 70001])
@pytest.mark.parametrize("width", [16, 200, 1500])
def test_rows(rows, width):
    if rows * width > 20_000_000:
        rows = 20_000_000 // width
    Norm(rows, width, 1, "bf16", seed=rows, residual=False, weight="f32").check()


def test_outputs_alone():
    d = Norm(7, 700, 2, "bf16")
    ref = d.run(eight=True)
    for name in ("out", "rstd"):
        o = Out(*ref[name].shape, dtype=ref[name].dtype)
        ar.ar_reduce_norm(d.x, d.shape, d.w, residual=d.residual, **{name: o.t})
        torch.cuda.synchronize()
        o.check()
        assert torch.equal(o.t, ref[name])
    o = Out(7, 700, dtype=torch.bfloat16)
    ar.ar_reduce_norm(d.x, d.shape, d.w, residual=d.residual, summed=o.t)
    assert torch.equal(o.t, ref["summed"])
    q, sc = Out(7, 700, dtype=torch.uint8), Out(7, 1)
    ar.ar_reduce_norm(d.x, d.shape, d.w, residual=d.residual, out8=q.t, scales=sc.t)
    assert torch.equal(q.t, ref["out8"]) and torch.equal(sc.t, ref["scales"])


@pytest.mark.parametrize("width", [64, 300, 4096])
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
def test_special_rows(width, dtype):
    d = Norm(12, width, 2, dtype, group=64)
    c = width // 2
    for x in d.x + [d.residual]:
        x[1] = 0.0                                          # a row of padding
    d.x[0][2, c] = float("nan")
    d.x[0][3, c] = float("inf")
    d.x[0][4, c], d.x[1][4, c] = float("inf"), float("-inf")
    top = torch.finfo(DT[dtype]).max
    d.x[0][5], d.x[1][5], d.residual[5] = top * 0.5, top * 0.25, 0.0          # squares past fp32 (but for fp16)
    d.x[0][6, c], d.x[1][6, c] = top, top                                     # `summed` past its type
    tiny = torch.finfo(DT[dtype]).tiny
    d.x[0][7], d.x[1][7], d.residual[7] = tiny, 0.0, 0.0                      # squares below fp32's range
    d.w[1] = 0.0
    d.w[2] = -1.0
    if dtype != "f16":
        # the sum itself is in fp32
        d.x[0][6, c], d.x[1][6, c] = top * 0.5, top * 0.25
    d.check(eight=True)


def test_eps_zero_and_large():
    d = Norm(4, 256, 1, "f32", residual=False, eps=0.0)
    d.x[0][1] = 0.0                                         # 0 * inf: the definition says NaN
    d.x[0][2] = 1e-25
    d.x[0][3] = 1e25
    d.check()
    Norm(4, 256, 1, "f32", eps=1e4).check()


@pytest.mark.parametrize("width", [13, 100, 500, 1001, 8197])
def test_in_place(width):
    for dtype in ("bf16", "f32"):
        d = Norm(40, width, 2, dtype)
        ref = d.run()
        res, x1 = d.residual.clone(), d.x[1].clone()
        ar.ar_reduce_norm([d.x[0], x1], d.shape, d.w, residual=res, summed=res, out=x1)
        torch.cuda.synchronize()
        assert torch.equal(res, ref["summed"]) and torch.equal(x1, ref["out"])


def test_equal_calls_give_equal_bits_on_any_stream():
    d = Norm(300, 4104, 8, "bf16", group=128)
    a = d.run(eight=True)
    for b in (d.run(eight=True), d.run(eight=True, stream=torch.cuda.Stream())):
        for k in a:
            assert torch.equal(a[k], b[k])


# ---- backward -----------------------------------------------------------------

def check_backward(rows, width, dtype, weight="same", pad=0, offset=0.0, summed=True, want_dw=True, seed=0, x=None, in_place=None,
                   rstd=None, stream=None):
    d = Norm(rows, width, 1, dtype, weight=weight, residual=False, pad=pad, at=1 if pad else 0, offset=offset, seed=seed)
    if x is not None:
        d.x[0].copy_(x)
    xs = d.x[0]
    g = torch.Generator(device="cuda").manual_seed(seed + 5)
    go = torch.randn(rows, width, generator=g, device="cuda").to(DT[dtype])
    gs = torch.randn(rows, width, generator=g, device="cuda").to(DT[dtype]) if summed else None
    if rstd is None:
        rstd = torch.rsqrt(xs.double().square().mean(1) + d.eps).float()
    want, want_w = lo.reduce_norm_backward(f64(xs), f64(d.w), f64(rstd), f64(go), None if gs is None else f64(gs), offset)
    h = f64(xs) * f64(rstd)[:, None]
    wabs = np.abs(f64(d.w)) + abs(offset)
    with np.errstate(all="ignore"):
        u = np.abs(f64(go)) * wabs
        c = (f64(go) * (f64(d.w) + offset) * h).mean(1, keepdims=True)
        dc = 38 * U * (u * np.abs(h)).mean(1, keepdims=True)
        tol = f64(rstd)[:, None] * (5 * U * u + np.abs(h) * dc + 5 * U * np.abs(h * c)) + U * (np.abs(want) + (0 if gs is None else np.abs(f64(gs))))
        tol_w = (rows + 8) * U * np.abs(f64(go) * h).sum(0)
    gx = Out(rows, width, dtype=DT[dtype])
    target = {"grad_out": go, "grad_summed": gs, "x": xs}.get(in_place, gx.t)
    dw = Out(width) if want_dw else None
    ws = torch.full((ar.ar_norm_workspace(d.shape),), 255, dtype=torch.uint8, device="cuda") if want_dw else None
    torch.cuda.synchronize()
    ar.ar_reduce_norm_backward(xs, d.shape, d.w, rstd, go, target, grad_summed=gs, grad_weight=dw.t if dw else None, workspace=ws,
                               stream=stream)
    torch.cuda.synchronize()
    gx.check()
    close(f64(target), want, tol + half(want, dtype) * 1.01, "grad_x")
    if dw:
        dw.check()
        close(f64(dw.t), want_w, tol_w, "grad_weight")
    return target.clone(), dw.t.clone() if dw else None


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("width", WIDTHS)
def test_backward_widths(width, dtype):
    check_backward(21, width, dtype, seed=width)
    check_backward(5, width, dtype, weight="f32", pad=5, offset=1.0, summed=False, seed=width)


@pytest.mark.parametrize("rows", [1, 2, 16, 17, 1000, 5000])
@pytest.mark.parametrize("width", [3, 100, 400, 1024])
def test_backward_rows(rows, width):
    check_backward(rows, width, "bf16", seed=rows)
    check_backward(rows, width, "f32", seed=rows, want_dw=False)


def test_backward_without_rows_clears_the_weight_gradient():
    sh = ar.NormShape(0, 300, 1, "bf16")
    dw = torch.full((300,), 9.0, device="cuda")
    ar.ar_reduce_norm_backward(None, sh, None, None, None, None, grad_weight=dw)
    assert (dw == 0).all()


@pytest.mark.parametrize("width", [13, 100, 500, 1001, 4096, 8197, 16383])
@pytest.mark.parametrize("where", ["grad_out", "grad_summed", "x"])
def test_backward_in_place(width, where):
    for dtype in ("bf16", "f32"):
        a = check_backward(150, width, dtype, seed=3)
        b = check_backward(150, width, dtype, seed=3, in_place=where)
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_backward_of_padding_and_infinities():
    x = torch.randn(6, 300, device="cuda")
    x[1] = 0
    check_backward(6, 300, "f32", x=x)
    x[2, 7] = float("nan")
    rstd = torch.rsqrt(x.square().mean(1) + 1e-6)
    check_backward(6, 300, "f32", x=x, rstd=rstd)


def test_backward_bits_and_streams():
    a = check_backward(3000, 4104, "bf16", seed=8)
    b = check_backward(3000, 4104, "bf16", seed=8, stream=torch.cuda.Stream())
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_gradient_by_differences():
    """The backward call against differences of the forward call, in fp32 with steps that leave 12 bits."""
    d = Norm(2, 40, 1, "f32", residual=False, eps=1e-2)
    go = torch.randn(2, 40, device="cuda")
    out, rstd, gx = torch.empty(2, 40, device="cuda"), torch.empty(2, device="cuda"), torch.empty(2, 40, device="cuda")

    def value(x):
        ar.ar_reduce_norm([x], d.shape, d.w, out=out, rstd=rstd)
        return (out.double() * go.double()).sum(1)

    value(d.x[0])
    ar.ar_reduce_norm_backward(d.x[0], d.shape, d.w, rstd, go, gx)
    step = 2.0 ** -9
    for c in range(40):
        up, down = d.x[0].clone(), d.x[0].clone()
        up[:, c] += step
        down[:, c] -= step
        slope = (value(up) - value(down)) / (up[:, c].double() - down[:, c].double())
        # values of up to 40 * 3 * 2 with 16 u each over a step of 2^-8; third derivatives times step^2
        assert (slope - gx[:, c].double()).abs().max() < 240 * 16 * U * 256 + 100 * step ** 2


def test_rows_far_apart():
    """Row starts past 2^32 bytes."""
    pitch, rows, width = (1 << 29) + 5, 6, 700
    flat = torch.empty(pitch * (rows - 1) + width, dtype=torch.bfloat16, device="cuda")
    x = torch.as_strided(flat, (rows, width), (pitch, 1))
    x.copy_(torch.randn(rows, width, device="cuda"))
    d = Norm(rows, width, 1, "bf16", residual=False)
    d.x, d.shape = [x], ar.NormShape(rows, width, 1, "bf16", pitches=[pitch])
    d.check()
    rstd = torch.rsqrt(x.double().square().mean(1) + 1e-6).float()
    go, a, b = torch.randn(rows, width, device="cuda").bfloat16(), *(torch.empty(rows, width, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    sh = ar.NormShape(rows, width, 1, "bf16")
    ar.ar_reduce_norm_backward(x, sh, d.w, rstd, go, a)
    ar.ar_reduce_norm_backward(x.contiguous(), sh, d.w, rstd, go, b)
    assert torch.equal(a, b)

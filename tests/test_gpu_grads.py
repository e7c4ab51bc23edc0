"""The gradient norm and clipping on the GPU against the 64-bit definitions
(oracle/layer.py).  The sum is in 64 bits and rounded once: half a step of fp32
(a little more for the sum's own roundings); a clipped value carries the
factor's rounding and its own, and one of its type."""
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
HALF = {torch.float32: (2.0 ** -24, 2.0 ** -150), torch.bfloat16: (2.0 ** -8, 2.0 ** -134), torch.float16: (2.0 ** -11, 2.0 ** -25)}


def f64(t):
    return t.detach().double().cpu().numpy()


def make(sizes, dtypes, scale=1.0, seed=0, adjoin=False, odd=0):
    """Buffers one behind the other where types agree (adjoin), or apart by `odd` elements."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    out = []
    if adjoin:
        for dt in sorted(set(dtypes)):
            mine = [s for s, d in zip(sizes, dtypes) if d == dt]
            out += (torch.randn(sum(mine) + odd, generator=g, device="cuda") * scale).to(DT[dt])[odd:].split(mine)
        return list(out)
    return [(torch.randn(s + odd, generator=g, device="cuda") * scale).to(DT[d])[odd:] for s, d in zip(sizes, dtypes)]


def check(grads, max_norm=1.0, scale=1.0, eps=1e-6, in_place=False, stream=None):
    f32 = lambda v: float(np.float32(v))
    want_norm, f = lo.clip([f64(g) for g in grads], f32(max_norm), f32(scale), f32(eps))
    before = [g.clone() for g in grads]
    gl = ar.GradList(grads)
    outs = gl if in_place else ar.GradList([torch.empty_like(g) for g in grads])
    ws = torch.full((ar.ar_grad_workspace(gl) + 8,), 255, dtype=torch.uint8, device="cuda")
    norms = torch.full((2, 1), 3.0, device="cuda")
    torch.cuda.synchronize()
    ar.ar_grad_norm(gl, norms[0], scale=scale, workspace=ws[:-8], stream=stream)
    ar.ar_clip_grads(gl, outs, norms[1], max_norm, scale=scale, eps=eps, workspace=ws[:-8], stream=stream)
    torch.cuda.synchronize()
    assert (ws[-8:] == 255).all()
    for n in f64(norms)[:, 0]:
        assert n == want_norm or np.isnan(n) and np.isnan(want_norm) or abs(n - want_norm) <= 1.01 * U * want_norm
    for src, b, o in zip(grads, before, outs._tensors):
        if not in_place:
            assert torch.equal(src.isnan(), b.isnan()) and torch.equal(src.nan_to_num(0.0), b.nan_to_num(0.0))
        with np.errstate(all="ignore"):
            want = f64(b) * f
        got = f64(o)
        assert (np.isnan(want) == np.isnan(got)).all()
        ok = np.isfinite(want)
        rel, tiny = HALF[b.dtype]
        assert (np.abs(got[ok] - want[ok]) <= (1.01 * rel + 3 * U) * np.abs(want[ok]) + tiny).all()
    return outs._tensors, norms[1]


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("size", [0, 1, 7, 8, 9, 2047, 2048, 2049, 16383, 16384, 16385, 100_001, 17_000_003])
def test_one_buffer(size, dtype):
    check(make([size], [dtype], odd=size % 3))
    check(make([size], [dtype]), max_norm=1e9, scale=0.125, in_place=True)


@pytest.mark.parametrize("count", [1, 2, 119, 120, 121, 127, 128, 129, 500])
@pytest.mark.parametrize("adjoin", [False, True])
def test_many_buffers(count, adjoin):
    rng = np.random.default_rng(count)
    sizes = [int(s) for s in np.exp(rng.uniform(0, 9, count))]
    sizes[count // 2] = 0
    dtypes = [["f32", "bf16", "f16"][i] for i in rng.integers(0, 3, count)]
    check(make(sizes, dtypes, adjoin=adjoin, odd=count % 2), max_norm=0.5)
    check(make(sizes, dtypes, adjoin=adjoin), max_norm=2.0, scale=3.0, in_place=True)


def test_an_empty_list():
    norm = torch.full((1,), 4.0, device="cuda")
    e = ar.GradList([])
    ar.ar_grad_norm(e, norm)
    assert norm.item() == 0
    norm.fill_(4)
    ar.ar_clip_grads(e, e, norm, 1.0)
    assert norm.item() == 0


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("size", [1e-30, 1e-6, 3e4, 1e20, 1e30])
def test_ranges(size, dtype):
    """Squares beyond fp32's range either way."""
    if dtype == "f16" and not 1e-7 < size < 65504:
        return
    g = make([5000, 3], [dtype, "f32"], scale=1.0)
    for t in g:
        t.copy_((t.float().clamp(-1, 1).double() * size).to(t.dtype))
    check(g, max_norm=size / 10)


def test_infinities_and_nan():
    for bad in (float("inf"), -float("inf"), float("nan")):
        g = make([300, 200], ["f32", "bf16"])
        g[1][17] = bad
        check(g)
        check(g, max_norm=float("inf"))


def test_zeros_and_limits():
    check([torch.zeros(100, device="cuda")], max_norm=0.0, eps=0.0)
    check(make([100], ["f32"]), max_norm=0.0)
    check(make([100], ["f32"]), max_norm=float("inf"), scale=2.0)


def test_unchanged_in_place_keeps_every_bit():
    g = torch.arange(1 << 16, device="cuda", dtype=torch.int32).to(torch.int16).view(torch.bfloat16)
    g[(~g.isfinite())] = 0
    g = g.clone()
    before = g.clone()
    gl = ar.GradList([g])
    ar.ar_clip_grads(gl, gl, torch.empty(1, device="cuda"), float("inf"),
                     workspace=torch.empty(ar.ar_grad_workspace(gl), dtype=torch.uint8, device="cuda"))
    assert torch.equal(g.view(torch.int16), before.view(torch.int16))


def test_dense_layouts_of_any_order():
    g = [torch.randn(40, 30, device="cuda").t(), torch.randn(3, 4, 5, 6, device="cuda").contiguous(memory_format=torch.channels_last)]
    outs, _ = check(g)
    assert all(o.stride() == t.stride() for o, t in zip(outs, g))


def test_bits_and_streams():
    g = make([100_000, 7, 33_333], ["f32", "bf16", "f16"])
    a, na = check(g)
    b, nb = check(g, stream=torch.cuda.Stream())
    assert torch.equal(na, nb) and all(torch.equal(x, y) for x, y in zip(a, b))


def test_more_than_32_bits_of_elements():
    size = (1 << 32) + 12345
    g = torch.zeros(size, dtype=torch.bfloat16, device="cuda")
    g[-1], g[0], g[1 << 31] = 3.0, 4.0, 12.0
    gl = ar.GradList([g])
    norm = torch.empty(1, device="cuda")
    ar.ar_clip_grads(gl, gl, norm, 6.5, eps=0.0, workspace=torch.empty(ar.ar_grad_workspace(gl), dtype=torch.uint8, device="cuda"))
    assert norm.item() == 13.0
    assert (g[-1].item(), g[0].item(), g[1 << 31].item()) == (1.5, 2.0, 6.0)

"""The C ABI of the operators around a step's collectives without a GPU:
argument validation (before any HIP call), workspace sizes, the binding's
checks of tensors."""
from __future__ import annotations

import ctypes

import pytest

torch = pytest.importorskip("torch")
ar = pytest.importorskip("reduce_scatter_amd", reason="libar.so not built")

from reduce_scatter_amd import _binding as b  # noqa: E402

ADDR = 1 << 24                              # addresses that no refused call may touch
INVALID, UNSUPPORTED, ALIGNMENT = "AR_ERR_INVALID_ARG", "AR_ERR_UNSUPPORTED", "AR_ERR_ALIGNMENT"


def status(f, *a, **k):
    with pytest.raises(ar.ArError) as e:
        f(*a, **k)
    return e.value.name


def norm_shape(rows=4, width=64, n=2, dtype="bf16", **kw):
    return ar.NormShape(rows, width, n, dtype, **kw)


def norm(sh, x=None, weight=ADDR, out=ADDR * 100, **kw):
    x = [ADDR * (i + 2) for i in range(sh.n)] if x is None else x
    ar.ar_reduce_norm(x, sh, weight, out=out, stream=0, **kw)


@pytest.mark.parametrize("kw, want", [
    (dict(rows=-1), INVALID), (dict(rows=1 << 31), UNSUPPORTED), (dict(n=0), INVALID), (dict(n=129), INVALID),
    (dict(width=0), INVALID), (dict(width=16385), UNSUPPORTED), (dict(dtype="i32"), UNSUPPORTED), (dict(dtype=7), INVALID),
    (dict(weight_dtype="f16"), UNSUPPORTED), (dict(weight_dtype="i32"), UNSUPPORTED), (dict(pitches=[64, 63]), INVALID),
    (dict(pitches=[64, 1 << 31]), UNSUPPORTED), (dict(eps=-1e-6), INVALID), (dict(eps=float("nan")), INVALID),
    (dict(eps=float("inf")), INVALID), (dict(offset=float("nan")), INVALID), (dict(group=-32), INVALID),
    (dict(group=48), UNSUPPORTED), (dict(group=16), UNSUPPORTED), (dict(group=1024), UNSUPPORTED),
])
def test_norm_shapes(kw, want):
    sh = norm_shape(**kw)
    assert status(norm, sh) == want
    assert status(ar.ar_norm_workspace, sh) == want
    assert status(ar.ar_reduce_norm_backward, ADDR, sh, ADDR, ADDR, ADDR, ADDR * 9, stream=0) == want


def test_norm_arguments():
    sh = norm_shape()
    assert status(norm, sh, [None, ADDR]) == INVALID
    assert status(norm, sh, [ADDR * 2 + 1, ADDR]) == ALIGNMENT
    assert status(norm, sh, weight=None) == INVALID
    assert status(norm, sh, weight=ADDR + 1) == ALIGNMENT
    assert status(norm, sh, out=None) == INVALID                                          # nothing asked for
    assert status(norm, sh, out8=ADDR * 50) == INVALID                                    # without scales
    assert status(norm, sh, scales=ADDR * 50) == INVALID
    for name in ("residual", "summed", "out"):
        assert status(norm, sh, **{name: ADDR * 60 + 1}) == ALIGNMENT
    for name in ("rstd", "scales"):
        assert status(norm, sh, out8=ADDR * 50 if name == "scales" else None,
                      **({"scales": ADDR * 51 + 2} if name == "scales" else {"rstd": ADDR * 51 + 2})) == \
            (ALIGNMENT)
    size = 4 * 64 * 2
    assert status(norm, sh, summed=ADDR * 100 + size - 2) == INVALID                      # two outputs meet
    assert status(norm, sh, out=ADDR * 2 + 2) == INVALID                                  # a partial, shifted
    assert status(norm, norm_shape(pitches=[65, 65]), out=ADDR * 2) == INVALID            # in place at another pitch
    assert status(norm, sh, residual=ADDR * 70, summed=ADDR * 70 + 128) == INVALID
    assert status(norm, sh, out=ADDR) == INVALID                                          # the weight
    assert status(norm, sh, rstd=ADDR * 100) == INVALID
    assert status(norm, sh, out8=ADDR * 2, scales=ADDR * 90) == INVALID                   # 8 bits over a partial


def test_norm_backward_arguments():
    sh = norm_shape()
    need = ar.ar_norm_workspace(sh)
    assert need == 4 * 64                                                                 # one workgroup holds four rows
    base = dict(x=ADDR, shape=sh, weight=ADDR * 2, rstd=ADDR * 3, grad_out=ADDR * 4, grad_x=ADDR * 5)
    call = lambda **kw: ar.ar_reduce_norm_backward(**{**base, **kw}, stream=0)
    for name in ("x", "weight", "rstd", "grad_out", "grad_x"):
        assert status(call, **{name: None}) == INVALID
    for name in ("x", "weight", "rstd", "grad_out", "grad_x", "grad_summed", "grad_weight"):
        assert status(call, **{name: ADDR * 9 + 1}) == ALIGNMENT
    assert status(call, grad_weight=ADDR * 8) == INVALID                                  # no workspace
    raw = lambda ws, size: b._lib.ar_reduce_norm_backward(ADDR, 0, sh.ref, ADDR * 2, ADDR * 3, ADDR * 4, None, ADDR * 5,
                                                         ADDR * 8, ws, size, 0)
    assert raw(ADDR * 7, need - 1) == 1
    assert raw(ADDR * 7 + 8, need) == 3
    assert raw(ADDR * 8, need) == 1                                                       # the gradient itself
    assert status(call, grad_x=ADDR * 4 + 2) == INVALID
    assert status(call, grad_x=ADDR * 2) == INVALID
    assert b._lib.ar_reduce_norm_backward(ADDR, 63, sh.ref, ADDR * 2, ADDR * 3, ADDR * 4, None, ADDR * 5, None, None, 0, 0) == 1
    # in place over x needs x at the width
    assert b._lib.ar_reduce_norm_backward(ADDR, 65, sh.ref, ADDR * 2, ADDR * 3, ADDR * 4, None, ADDR, None, None, 0, 0) == 1


def embed_shape(tokens=5, entries=(6, 0, 4), width=16, dtype="f32", **kw):
    return ar.EmbedShape(tokens, list(entries), width, dtype, **kw)


@pytest.mark.parametrize("kw, want", [
    (dict(tokens=-1), INVALID), (dict(tokens=(1 << 28) + 1), UNSUPPORTED), (dict(entries=[]), INVALID),
    (dict(entries=[1] * 129), INVALID), (dict(entries=[3, -1]), INVALID), (dict(entries=[0, 0]), INVALID),
    (dict(entries=[1 << 20, 1]), UNSUPPORTED), (dict(entries=[1 << 62, 1 << 62]), UNSUPPORTED), (dict(width=0), INVALID),
    (dict(width=65537), UNSUPPORTED), (dict(dtype="i32"), UNSUPPORTED), (dict(out_dtype="i32"), UNSUPPORTED),
    (dict(dtype=-1), INVALID), (dict(pitches=[16, 15, 16]), INVALID), (dict(grad_pitches=[16, 16, 1 << 31]), UNSUPPORTED),
    (dict(scale=float("inf")), INVALID), (dict(scale=float("nan")), INVALID),
])
def test_embed_shapes(kw, want):
    sh = embed_shape(**kw)
    bufs = [ADDR * (i + 2) for i in range(sh.n)]
    assert status(ar.ar_embedding, bufs, sh, ADDR, ADDR * 200, stream=0) == want
    assert status(ar.ar_embedding_workspace, sh) == want
    assert status(ar.ar_embedding_backward, ADDR, sh, ADDR, bufs, stream=0) == want


def test_embed_arguments():
    sh = embed_shape()
    t = [ADDR * 2, None, ADDR * 4]
    look = lambda tables=t, ids=ADDR, out=ADDR * 9: ar.ar_embedding(tables, sh, ids, out, stream=0)
    assert status(look, [None, None, ADDR]) == INVALID
    assert status(look, [ADDR * 2 + 2, None, ADDR]) == ALIGNMENT
    assert status(look, ids=None) == INVALID
    assert status(look, ids=ADDR + 4) == ALIGNMENT
    assert status(look, out=None) == INVALID
    assert status(look, out=ADDR * 9 + 2) == ALIGNMENT
    assert status(look, out=ADDR * 4 + 64) == INVALID
    assert status(look, out=ADDR) == INVALID
    need = ar.ar_embedding_workspace(sh)
    assert need > 0 and ar.ar_embedding_workspace(embed_shape(0)) == 0
    raw = lambda g=ADDR * 7, ids=ADDR, bufs=t, ws=ADDR * 8, size=need: b._lib.ar_embedding_backward(
        g, sh.ref, ids, (ctypes.c_void_p * 3)(*bufs), 0, ws, size, 0)
    assert raw(g=None) == raw(ids=None) == raw(bufs=[ADDR, None, None]) == raw(size=need - 1) == raw(ws=None) == 1
    assert raw(g=ADDR * 7 + 2) == raw(ids=ADDR + 4) == raw(bufs=[ADDR * 2, None, ADDR * 4 + 1]) == raw(ws=ADDR * 8 + 8) == 3
    assert raw(bufs=[ADDR * 2, None, ADDR * 2 + 128]) == 1                                # one another
    assert raw(bufs=[ADDR * 7, None, ADDR * 2]) == 1                                      # the incoming gradient
    assert raw(ws=ADDR * 2) == 1 and raw(ws=ADDR) == 1


def test_norms_of_lists():
    t = [torch.zeros(3), torch.zeros(0), torch.zeros(2, 2, dtype=torch.bfloat16)]
    gl = ar.GradList(t)
    assert ar.ar_grad_workspace(gl) == 3 * 8                               # the norm, two partial sums
    assert ar.ar_grad_workspace(ar.GradList([])) == 0
    for f in (lambda: ar.ar_grad_norm(gl, ADDR, stream=0), lambda: ar.ar_clip_grads(gl, gl, ADDR, 1.0, stream=0)):
        with pytest.raises(ValueError, match="gradients .*host memory"):
            f()
    with pytest.raises(ValueError, match="fill their memory"):
        ar.GradList([torch.zeros(4, 4)[:, :2]])
    ar.GradList([torch.zeros(4, 6).t(), torch.zeros(2, 3, 5).permute(2, 0, 1)])           # dense in another order
    with pytest.raises(ValueError, match="types, shapes and strides"):
        ar.ar_clip_grads(gl, ar.GradList([torch.zeros(3), torch.zeros(0), torch.zeros(4, dtype=torch.bfloat16)]), ADDR, 1.0)
    with pytest.raises(ValueError, match="types, shapes and strides"):
        ar.ar_clip_grads(ar.GradList([torch.zeros(4, 6)]), ar.GradList([torch.zeros(6, 4).t()]), ADDR, 1.0)


def raw_list(bufs, sizes, dtypes, count=None):
    m = len(bufs)
    keep = ((ctypes.c_void_p * max(1, m))(*bufs), (ctypes.c_longlong * max(1, m))(*sizes), (ctypes.c_int * max(1, m))(*dtypes))
    return b._GradsStruct(m if count is None else count, ctypes.cast(keep[0], ctypes.c_void_p), keep[1], keep[2]), keep


def test_grad_arguments():
    def call(bufs=(ADDR, ADDR * 2), sizes=(4, 5), dtypes=(0, 1), outs=None, scale=1.0, norm=ADDR * 5, ws=ADDR * 6, size=64,
             max_norm=1.0, eps=0.0, count=None, clip=None):
        s, keep = raw_list(bufs, sizes, dtypes, count)
        ref = ctypes.byref(s)
        outs = (ctypes.c_void_p * len(bufs))(*(bufs if outs is None else outs))
        got = [b._lib.ar_grad_norm(ref, scale, norm, ws, size, 0)] if not clip else []
        return got + ([b._lib.ar_clip_grads(ref, outs, max_norm, scale, eps, norm, ws, size, 0)] if clip is not False else [])

    both = dict(clip=None)
    for kw, want in [(dict(count=-1), 1), (dict(count=(1 << 20) + 1), 2), (dict(sizes=(4, -1)), 1), (dict(dtypes=(0, 3)), 2),
                     (dict(dtypes=(0, 9)), 1), (dict(sizes=(1 << 40, 1)), 2), (dict(bufs=(ADDR, None)), 1),
                     (dict(bufs=(ADDR + 2, ADDR)), 3), (dict(scale=0.0), 1), (dict(scale=float("inf")), 1),
                     (dict(scale=float("nan")), 1), (dict(norm=None), 1), (dict(norm=ADDR * 5 + 2), 3), (dict(ws=None), 1),
                     (dict(size=15), 1), (dict(ws=ADDR * 6 + 8), 3), (dict(norm=ADDR * 2 + 4), 1), (dict(ws=ADDR), 1),
                     (dict(norm=ADDR * 6 + 8), 1)]:
        assert call(**kw, **both) == [want, want], kw
    for kw, want in [(dict(max_norm=-1.0), 1), (dict(max_norm=float("nan")), 1), (dict(eps=-1.0), 1), (dict(eps=float("inf")), 1),
                     (dict(outs=(None, ADDR)), 1), (dict(outs=(ADDR * 3, ADDR * 3 + 8)), 1), (dict(outs=(ADDR + 4, ADDR * 4)), 1),
                     (dict(outs=(ADDR * 3, ADDR * 4 + 1)), 3), (dict(outs=(ADDR * 2, ADDR)), 1),
                     (dict(bufs=(ADDR, ADDR), sizes=(4, 4), dtypes=(0, 0)), 1)]:        # the same buffer twice, in place
        assert call(**kw, clip=True) == [want], kw


HOST = dict(f=torch.zeros(512), i=torch.zeros(64, dtype=torch.int64), w=torch.zeros(4096, dtype=torch.uint8),
            q=torch.zeros(512, dtype=torch.uint8))
NS, ES = ar.NormShape(4, 16, 2, "f32"), ar.EmbedShape(4, [8, 8], 16, "f32")
X = [torch.zeros(4, 16) for _ in range(2)]
CALLS = [
    (ar.ar_reduce_norm, dict(partials=[ADDR, ADDR * 2], shape=NS, weight=ADDR, out=ADDR),
     dict(partials=X, weight="f", out="f", residual="f", summed="f", rstd="f", out8="q", scales="f")),
    (ar.ar_reduce_norm_backward, dict(x=ADDR, shape=NS, weight=ADDR, rstd=ADDR, grad_out=ADDR, grad_x=ADDR),
     dict(x=X[0], weight="f", rstd="f", grad_out="f", grad_x="f", grad_summed="f", grad_weight="f", workspace="w")),
    (ar.ar_embedding, dict(tables=[ADDR, ADDR * 2], shape=ES, token_ids=ADDR, out=ADDR),
     dict(tables=[torch.zeros(8, 16)] * 2, token_ids="i", out="f")),
    (ar.ar_embedding_backward, dict(grad_out=ADDR, shape=ES, token_ids=ADDR, grads=[ADDR, ADDR * 2]),
     dict(grad_out="f", token_ids="i", grads=[torch.zeros(8, 16)] * 2, workspace="w")),
    (ar.ar_grad_norm, dict(grads=ar.GradList([]), norm=ADDR), dict(norm="f", workspace="w")),
    (ar.ar_clip_grads, dict(grads=ar.GradList([]), outs=ar.GradList([]), norm=ADDR, max_norm=1.0), dict(norm="f", workspace="w")),
]


@pytest.mark.parametrize("call, base, name, value", [(c, base, n, v) for c, base, host in CALLS for n, v in host.items()])
def test_host_memory_is_refused_by_name(call, base, name, value):
    value = HOST[value] if isinstance(value, str) else value
    with pytest.raises(ValueError, match="%s .*host memory" % name):
        call(**{**base, name: value}, stream=0)


def test_tensors_that_do_not_fit():
    bf = lambda *s: torch.zeros(s, dtype=torch.bfloat16)
    for kw, match in [(dict(partials=[bf(4, 16)] * 2), "dtype"), (dict(partials=[torch.zeros(4, 15)] * 2), "need more"),
                      (dict(partials=[torch.zeros(4, 20)[:, :16]] * 2), "pitch"), (dict(partials=[torch.zeros(4, 16)]), "ranks"),
                      (dict(weight=bf(16)), "float32"), (dict(weight=torch.zeros(15)), "16 elements"),
                      (dict(residual=torch.zeros(4, 20)[:, :16]), "contiguous"), (dict(rstd=bf(4)), "float32"),
                      (dict(out8=torch.zeros(4, 16, dtype=torch.int8)), "float8_e4m3fn"), (dict(scales=torch.zeros(3)), "4 elements")]:
        with pytest.raises(ValueError, match=match):
            ar.ar_reduce_norm(**{**CALLS[0][1], **kw}, stream=0)
    with pytest.raises(ValueError, match="one pitch per rank"):
        ar.NormShape(4, 16, 2, "f32", pitches=[16])
    with pytest.raises(ValueError, match="one pitch per rank"):
        ar.EmbedShape(4, [8, 8], 16, "f32", pitches=[16])
    with pytest.raises(ValueError, match="int64"):
        ar.ar_embedding([ADDR, ADDR], ES, torch.zeros(4, dtype=torch.int32), ADDR, stream=0)
    with pytest.raises(ValueError, match="need more"):
        ar.ar_embedding([torch.zeros(7, 16), torch.zeros(8, 16)], ES, ADDR, ADDR, stream=0)


def test_nothing_to_do_needs_no_memory():
    ar.ar_reduce_norm([None, None], ar.NormShape(0, 16, 2, "f32"), None, out=ADDR, stream=0)
    ar.ar_embedding([None, None], ar.EmbedShape(0, [8, 8], 16, "f32"), None, None, stream=0)
    ar.ar_embedding_backward(None, ar.EmbedShape(0, [8, 8], 16, "f32"), None, [None, None], accumulate=True, stream=0)
    ar.ar_reduce_norm_backward(None, ar.NormShape(0, 16, 1, "f32"), None, None, None, None, stream=0)

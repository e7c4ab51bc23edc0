"""The vocabulary reductions' C ABI without a GPU: argument validation (before
any HIP call), workspace sizes, and the binding's checks of tensors."""
from __future__ import annotations

import ctypes

import pytest

torch = pytest.importorskip("torch")
ar = pytest.importorskip("reduce_scatter_amd", reason="libar.so not built")

from reduce_scatter_amd import _binding as b  # noqa: E402

LL = ctypes.c_longlong


def shape(rows=4, widths=(8, 8), dtype="f32", **kw):
    return ar.VocabShape(rows, list(widths), dtype, **kw)


def cpu(*dims, dtype=torch.float32):
    return torch.zeros(dims, dtype=dtype)


def status(f, *a, **k):
    with pytest.raises(ar.ArError) as e:
        f(*a, **k)
    return e.value.name


ADDR = 1 << 20                              # addresses that no refused call may touch


def call(sh, x=None, targets=ADDR, logprobs=ADDR, **kw):
    x = [ADDR * (i + 2) for i in range(sh.n)] if x is None else x
    ar.ar_logprobs(x, sh, targets, logprobs, stream=0, **kw)


def test_workspace():
    assert ar.ar_vocab_workspace(shape(), 0) == 0                       # one workgroup holds a row
    few = shape(1, [1 << 20], "bf16")
    assert ar.ar_vocab_workspace(few, 0) > 0
    assert ar.ar_vocab_workspace(few, 64) > ar.ar_vocab_workspace(few, 1) > ar.ar_vocab_workspace(few, 0)
    assert ar.ar_vocab_workspace(shape(100000, [1 << 17], "bf16"), 64) == 0
    assert status(ar.ar_vocab_workspace, shape(), -1) == "AR_ERR_INVALID_ARG"
    assert status(ar.ar_vocab_workspace, shape(), 65) == "AR_ERR_UNSUPPORTED"


@pytest.mark.parametrize("kw, want", [
    (dict(rows=-1), "AR_ERR_INVALID_ARG"),
    (dict(rows=1 << 31), "AR_ERR_UNSUPPORTED"),
    (dict(widths=[]), "AR_ERR_INVALID_ARG"),
    (dict(widths=[4] * 129), "AR_ERR_INVALID_ARG"),
    (dict(widths=[4, -1]), "AR_ERR_INVALID_ARG"),
    (dict(widths=[0, 0]), "AR_ERR_INVALID_ARG"),
    (dict(widths=[1 << 20, 1]), "AR_ERR_UNSUPPORTED"),
    (dict(widths=[1 << 40]), "AR_ERR_UNSUPPORTED"),
    (dict(dtype="i32"), "AR_ERR_UNSUPPORTED"),
    (dict(dtype=9), "AR_ERR_INVALID_ARG"),
    (dict(pitches=[8, 7]), "AR_ERR_INVALID_ARG"),
    (dict(pitches=[8, 1 << 31]), "AR_ERR_UNSUPPORTED"),
    (dict(grad_pitches=[7, 8]), "AR_ERR_INVALID_ARG"),
    (dict(rows=(1 << 31) - 1, pitches=[(1 << 31) - 1] * 2), "AR_ERR_UNSUPPORTED"),
    (dict(temperature=0.0), "AR_ERR_INVALID_ARG"),
    (dict(temperature=-1.0), "AR_ERR_INVALID_ARG"),
    (dict(temperature=float("nan")), "AR_ERR_INVALID_ARG"),
    (dict(temperature=float("inf")), "AR_ERR_INVALID_ARG"),
    (dict(temperature=1e-35), "AR_ERR_UNSUPPORTED"),
])
def test_shape_refusals(kw, want):
    sh = shape(**kw)
    assert status(ar.ar_vocab_workspace, sh) == want
    assert status(call, sh) == want


def test_null_and_misaligned_arguments():
    sh = shape()
    assert status(call, sh, [None, ADDR]) == "AR_ERR_INVALID_ARG"
    assert status(call, sh, [ADDR + 2, ADDR]) == "AR_ERR_ALIGNMENT"
    assert status(call, sh, targets=None) == "AR_ERR_INVALID_ARG"
    assert status(call, sh, logprobs=None) == "AR_ERR_INVALID_ARG"
    assert status(call, sh, targets=ADDR + 4) == "AR_ERR_ALIGNMENT"
    assert status(call, sh, logprobs=ADDR + 2) == "AR_ERR_ALIGNMENT"
    assert status(call, sh, entropy=ADDR + 2) == "AR_ERR_ALIGNMENT"
    assert status(call, sh, saved=ADDR + 2) == "AR_ERR_ALIGNMENT"
    assert status(call, sh, top_k=3) == "AR_ERR_INVALID_ARG"                            # lists missing
    assert status(call, sh, top_k=3, top_logprobs=ADDR) == "AR_ERR_INVALID_ARG"
    assert status(call, sh, top_logprobs=ADDR, top_ids=ADDR) == "AR_ERR_INVALID_ARG"    # lists without a length
    assert status(call, sh, top_k=-1, top_logprobs=ADDR, top_ids=ADDR) == "AR_ERR_INVALID_ARG"
    assert status(call, sh, top_k=65, top_logprobs=ADDR, top_ids=ADDR) == "AR_ERR_UNSUPPORTED"
    assert status(call, sh, top_k=2, top_logprobs=ADDR, top_ids=ADDR + 4) == "AR_ERR_ALIGNMENT"
    half = shape(dtype="bf16")
    assert status(call, half, [ADDR + 1, ADDR]) == "AR_ERR_ALIGNMENT"


def test_workspace_refusals():
    sh = shape(1, [1 << 20], "bf16")
    assert status(call, sh) == "AR_ERR_INVALID_ARG"                                     # needed and missing
    need = ar.ar_vocab_workspace(sh)
    args = [(ctypes.c_void_p * 1)(ADDR * 8), sh.ref, ADDR, ADDR, None, 0, None, None, None]
    assert b._lib.ar_logprobs(*args, ADDR, need - 1, 0) == 1
    assert b._lib.ar_logprobs(*args, ADDR + 8, need, 0) == 3


def test_gradient_buffers():
    sh = shape()                                            # two ranks, 4 rows of 8 fp32: 128 bytes each
    x = [ADDR, ADDR + 4096]
    back = lambda g, s=sh, xs=x, **k: ar.ar_logprobs_backward(xs, g, s, ADDR * 4, ADDR * 4, stream=0, **k)
    assert status(back, [None, ADDR * 2]) == "AR_ERR_INVALID_ARG"
    assert status(back, [ADDR * 2 + 2, ADDR * 3]) == "AR_ERR_ALIGNMENT"
    assert status(back, [ADDR * 2, ADDR * 2 + 64]) == "AR_ERR_INVALID_ARG"              # one another
    assert status(back, [ADDR + 64, ADDR * 2]) == "AR_ERR_INVALID_ARG"                  # own logits, shifted
    assert status(back, [ADDR + 4096, ADDR]) == "AR_ERR_INVALID_ARG"                    # each other's logits
    other = shape(pitches=[8, 8], grad_pitches=[9, 8])
    assert status(back, x, other) == "AR_ERR_INVALID_ARG"                               # in place at another pitch
    cols = shape(pitches=[16, 16])                                                      # columns of one [4, 16] buffer
    assert status(back, [ADDR * 2, ADDR * 2 + 28], cols, [ADDR, ADDR + 32]) == "AR_ERR_INVALID_ARG"
    assert status(lambda: ar.ar_logprobs_backward(x, [ADDR * 2, ADDR * 3], sh, None, ADDR, stream=0)) == \
        "AR_ERR_INVALID_ARG"
    assert status(lambda: ar.ar_logprobs_backward(x, [ADDR * 2, ADDR * 3], sh, ADDR, None, stream=0)) == \
        "AR_ERR_INVALID_ARG"


def test_teacher_refusals():
    sh = shape()
    x = [ADDR, ADDR * 2]
    f = lambda ids=ADDR * 3, vals=ADDR * 3, loss=ADDR * 4, k=2, **kw: ar.ar_distill(x, sh, ids, vals, loss, k=k,
                                                                                    stream=0, **kw)
    assert status(f, ids=0) == "AR_ERR_INVALID_ARG"
    assert status(f, vals=0) == "AR_ERR_INVALID_ARG"
    assert status(f, loss=None) == "AR_ERR_INVALID_ARG"
    assert status(f, k=0) == "AR_ERR_INVALID_ARG"
    assert status(f, k=257) == "AR_ERR_UNSUPPORTED"
    assert status(f, ids=ADDR + 4) == "AR_ERR_ALIGNMENT"
    assert status(f, vals=ADDR + 2) == "AR_ERR_ALIGNMENT"
    xs = (ctypes.c_void_p * 2)(*x)
    assert b._lib.ar_distill(xs, sh.ref, ADDR, ADDR, 2, 7, ADDR, None, None, 0, 0) == 1  # no such mode
    assert b._lib.ar_distill_backward(xs, xs, sh.ref, ADDR, ADDR, 2, 0, None, None, 0) == 1
    assert b._lib.ar_distill_grad(xs, xs, sh.ref, ADDR, None, 2, 0, None, None, None, None, 0, 0) == 1


def test_no_rows_is_no_work():
    sh = shape(rows=0)
    ar.ar_logprobs([None, None], sh, None, None, stream=0)
    ar.ar_logprobs_backward([None, None], [None, None], sh, None, None, stream=0)
    ar.ar_distill([None, None], sh, None, None, None, k=1, stream=0)


def test_binding_checks_tensors():
    sh = shape(dtype="bf16")
    x = [cpu(4, 8, dtype=torch.bfloat16) for _ in range(2)]
    t, lp = cpu(4, dtype=torch.int64), cpu(4)
    bad = [
        lambda: ar.ar_logprobs(x[:1], sh, t, lp),                                       # ranks
        lambda: ar.ar_logprobs([cpu(4, 8)] * 2, sh, t, lp),                             # dtype of logits
        lambda: ar.ar_logprobs([x[0], cpu(3, 8, dtype=torch.bfloat16)], sh, t, lp),     # rows
        lambda: ar.ar_logprobs([x[0], cpu(8, 4, dtype=torch.bfloat16)], sh, t, lp),     # pitch
        lambda: ar.ar_logprobs([x[0], cpu(8, 4, dtype=torch.bfloat16).t()], sh, t, lp),  # columns apart
        lambda: ar.ar_logprobs(x, sh, t.int(), lp),
        lambda: ar.ar_logprobs(x, sh, t[:3], lp),
        lambda: ar.ar_logprobs(x, sh, t, lp.double()),
        lambda: ar.ar_logprobs(x, sh, t, cpu(8)[::2]),
        lambda: ar.ar_logprobs(x, sh, t, lp, entropy=cpu(3)),
        lambda: ar.ar_logprobs(x, sh, t, lp, saved=cpu(4, 3)),
        lambda: ar.ar_logprobs(x, sh, t, lp, top_k=2, top_logprobs=cpu(4, 2), top_ids=cpu(4, 2, dtype=torch.int32)),
        lambda: ar.ar_distill(x, sh, cpu(4, 2, dtype=torch.int64), cpu(4, 1), lp),
        lambda: ar.ar_distill(x, sh, cpu(8, dtype=torch.int64), cpu(8), lp),            # k unknown
        lambda: ar.VocabShape(4, [8, 8], "bf16", pitches=[8]),
    ]
    for f in bad:
        with pytest.raises(ValueError):
            f()


def test_widths_follow_the_layout():
    for v, n in ((50021, 16), (7, 3), (2, 5)):
        L = ar.Layout((1, v), (n,), (1,))
        assert ar.vocab_widths(v, n) == [ar.local_shape(L, r)[1] for r in range(n)]

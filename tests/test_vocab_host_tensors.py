"""Tensors in pageable host memory are refused by name, not handed to a kernel (CPU)."""
from __future__ import annotations

import pytest

torch = pytest.importorskip("torch")
ar = pytest.importorskip("reduce_scatter_amd", reason="libar.so not built")

ADDR = 1 << 20                              # addresses that no refused call may touch
SHAPE = ar.VocabShape(4, [8, 8], "f32")
X, G = [ADDR * 2, ADDR * 3], [ADDR * 4, ADDR * 5]
HOST = [torch.zeros(4, 8) for _ in range(2)]
F, I, W = torch.zeros(16), torch.zeros(16, dtype=torch.int64), torch.zeros(64, dtype=torch.uint8)

CALLS = [
    (ar.ar_logprobs, dict(logits=X, shape=SHAPE, targets=ADDR, logprobs=ADDR),
     dict(logits=HOST, targets=I, logprobs=F, entropy=F, saved=F, workspace=W)),
    (ar.ar_logprobs, dict(logits=X, shape=SHAPE, targets=ADDR, logprobs=ADDR, top_k=2, top_logprobs=ADDR, top_ids=ADDR),
     dict(top_logprobs=F, top_ids=I)),
    (ar.ar_logprobs_backward, dict(logits=X, grads=G, shape=SHAPE, targets=ADDR, saved=ADDR),
     dict(logits=HOST, grads=HOST, targets=I, saved=F, grad_logprobs=F, grad_entropy=F)),
    (ar.ar_logprobs_grad, dict(logits=X, grads=G, shape=SHAPE, targets=ADDR),
     dict(logits=HOST, grads=HOST, targets=I, logprobs=F, grad_logprobs=F, grad_entropy=F, entropy=F, saved=F,
          workspace=W)),
    (ar.ar_distill, dict(logits=X, shape=SHAPE, teacher_ids=ADDR, teacher_values=ADDR, loss=ADDR, k=4),
     dict(logits=HOST, teacher_ids=I, teacher_values=F, loss=F, saved=F, workspace=W)),
    (ar.ar_distill_backward, dict(logits=X, grads=G, shape=SHAPE, teacher_ids=ADDR, teacher_values=ADDR, saved=ADDR, k=4),
     dict(logits=HOST, grads=HOST, teacher_ids=I, teacher_values=F, saved=F, grad_loss=F)),
    (ar.ar_distill_grad, dict(logits=X, grads=G, shape=SHAPE, teacher_ids=ADDR, teacher_values=ADDR, k=4),
     dict(logits=HOST, grads=HOST, teacher_ids=I, teacher_values=F, loss=F, grad_loss=F, saved=F, workspace=W)),
]


@pytest.mark.parametrize("call, base, name, value", [(c, base, n, v) for c, base, host in CALLS for n, v in host.items()])
def test_refused_by_name(call, base, name, value):
    # a refusal comes before any launch, whatever the other arguments are
    with pytest.raises(ValueError, match="%s .*host memory" % name):
        call(**{**base, name: value}, stream=0)


def test_a_reused_table_is_refused_too():
    table = ar.pointers(HOST)
    for _ in range(2):
        with pytest.raises(ValueError, match="logits .*host memory"):
            ar.ar_logprobs(table, SHAPE, ADDR, ADDR, stream=0)


def test_no_rows_need_no_memory():
    ar.ar_logprobs(HOST, ar.VocabShape(0, [8, 8], "f32"), I, F, stream=0)

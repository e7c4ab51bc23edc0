"""One training step of a small tensor-parallel language model, all ranks on one GPU.

Rank r holds its part of the vocabulary's table (which is the output layer's
weight as well) and its part of one feed-forward block.  The step
  1. looks the tokens up in the split table (`ar_embedding`) and normalises
     them (`ar_reduce_norm` of one buffer),
  2. runs the block, whose ranks leave partial sums; they are added to the
     residual stream and normalised in one call (`ar_reduce_norm`),
  3. takes the loss and its gradient from the split logits (`ar_logprobs_grad`),
  4. goes back: all-reduces of the hidden gradients (`ar_allreduce`), the norms
     (`ar_reduce_norm_backward`), the table (`ar_embedding_backward`, added to
     what the output layer left there),
  5. clips all gradients by their global norm, in place (`ar_clip_grads`).

    python examples/tensor_parallel_step.py [--ranks 4] [--tokens 256] [--hidden 256] [--vocab 10007] [--dtype bf16]
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import reduce_scatter_amd as ar  # noqa: E402

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


class Model:
    """The split weights, and what a program keeps from step to step: shapes,
    pointer tables, activations, gradients, workspaces."""

    def __init__(self, ranks, tokens, hidden, inner, vocab, dtype, max_norm=1.0, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        dt = DTYPES[dtype]
        weight = lambda *s: (torch.randn(s, generator=g, device="cuda") * s[-1] ** -0.5).to(dt)
        new = lambda *s, t=dt: torch.empty(s, dtype=t, device="cuda")
        space = lambda size: torch.empty(size, dtype=torch.uint8, device="cuda")
        self.tokens, self.max_norm = tokens, max_norm
        entries = ar.vocab_widths(vocab, ranks)
        self.table = [weight(e, hidden) for e in entries]
        self.up = [weight(w, hidden) for w in ar.vocab_widths(inner, ranks)]
        self.down = [weight(hidden, w.shape[0]) for w in self.up]
        self.gains = [1 + 0.1 * torch.randn(hidden, generator=g, device="cuda") for _ in range(2)]

        self.embed = ar.EmbedShape(tokens, entries, hidden, dtype)
        self.first = ar.NormShape(tokens, hidden, 1, dtype, weight_dtype="f32")
        self.second = ar.NormShape(tokens, hidden, ranks, dtype, weight_dtype="f32")
        self.logit_shape = ar.VocabShape(tokens, entries, dtype)
        self.x0, self.h0, self.x1, self.h1 = (new(tokens, hidden) for _ in range(4))
        self.rstd = [new(tokens, t=torch.float32) for _ in range(2)]
        self.partials = [new(tokens, hidden) for _ in range(ranks)]
        self.logits = [new(tokens, e) for e in entries]
        self.logprobs = new(tokens, t=torch.float32)
        self.dx0, self.dx1 = new(tokens, hidden), new(tokens, hidden)
        self.tables = [ar.pointers(t) for t in (self.table, self.partials, self.logits)]

        self.grads = {"table": [torch.empty_like(t) for t in self.table], "up": [torch.empty_like(t) for t in self.up],
                      "down": [torch.empty_like(t) for t in self.down], "gains": [torch.empty_like(t) for t in self.gains]}
        self.list = ar.GradList([t for part in self.grads.values() for t in part])
        self.norm = new(1, t=torch.float32)
        self.spaces = [space(n) for n in (ar.ar_norm_workspace(self.first), ar.ar_embedding_workspace(self.embed),
                                          ar.ar_grad_workspace(self.list), ar.ar_vocab_workspace(self.logit_shape))]

    def forward(self, ids):
        table, partials, _ = self.tables
        ar.ar_embedding(table, self.embed, ids, self.x0)
        ar.ar_reduce_norm([self.x0], self.first, self.gains[0], out=self.h0, rstd=self.rstd[0])
        self.inner = [torch.relu(self.h0 @ w.t()) for w in self.up]
        for out, a, w in zip(self.partials, self.inner, self.down):
            torch.matmul(a, w.t(), out=out)
        ar.ar_reduce_norm(partials, self.second, self.gains[1], out=self.h1, residual=self.x0, summed=self.x1, rstd=self.rstd[1])
        for out, w in zip(self.logits, self.table):
            torch.matmul(self.h1, w.t(), out=out)

    def backward(self, ids, targets):
        """The clipped gradients of the mean negative log probability of ``targets``, and their norm before clipping."""
        grads, logits, n = self.grads, self.tables[2], self.tokens
        norm_space, embed_space, clip_space, vocab_space = self.spaces
        ar.ar_logprobs_grad(logits, logits, self.logit_shape, targets, self.logprobs,
                            grad_logprobs=torch.full((n,), -1.0 / n, device="cuda"), workspace=vocab_space)
        dh = []
        for d, w, g in zip(self.logits, self.table, grads["table"]):
            torch.matmul(d.t(), self.h1, out=g)
            dh.append(d @ w)
        ar.ar_allreduce(dh, dh, dh[0].numel(), dh[0].dtype, "sum")
        ar.ar_reduce_norm_backward(self.x1, self.second, self.gains[1], self.rstd[1], dh[0], self.dx1,
                                   grad_weight=grads["gains"][1], workspace=norm_space)
        dh = []
        for a, up, down, gu, gd in zip(self.inner, self.up, self.down, grads["up"], grads["down"]):
            torch.matmul(self.dx1.t(), a, out=gd)
            da = (self.dx1 @ down) * (a > 0)
            torch.matmul(da.t(), self.h0, out=gu)
            dh.append(da @ up)
        ar.ar_allreduce(dh, dh, dh[0].numel(), dh[0].dtype, "sum")
        ar.ar_reduce_norm_backward(self.x0, self.first, self.gains[0], self.rstd[0], dh[0], self.dx0, grad_summed=self.dx1,
                                   grad_weight=grads["gains"][0], workspace=norm_space)
        ar.ar_embedding_backward(self.dx0, self.embed, ids, grads["table"], accumulate=True, workspace=embed_space)
        ar.ar_clip_grads(self.list, self.list, self.norm, self.max_norm, workspace=clip_space)
        return grads


def main(argv=None):
    p = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    p.add_argument("--ranks", type=int, default=4)
    p.add_argument("--tokens", type=int, default=256)
    p.add_argument("--hidden", type=int, default=256)
    p.add_argument("--inner", type=int, default=512)
    p.add_argument("--vocab", type=int, default=10007)
    p.add_argument("--dtype", choices=sorted(DTYPES), default="bf16")
    p.add_argument("--max-norm", type=float, default=0.1)
    a = p.parse_args(argv)
    g = torch.Generator(device="cuda").manual_seed(1)
    ids, targets = (torch.randint(0, a.vocab, (a.tokens,), generator=g, device="cuda") for _ in range(2))
    ids[::7], targets[::5] = ids[0].clone(), -100                     # a frequent token; positions without a target
    ids[3] = -1                                               # a position without a token
    model = Model(a.ranks, a.tokens, a.hidden, a.inner, a.vocab, a.dtype, a.max_norm)
    model.forward(ids)
    model.backward(ids, targets)
    print("loss %.4f, gradient norm %.4f, clipped to %g" % (-model.logprobs.mean(), model.norm, a.max_norm))
    return model, ids, targets


if __name__ == "__main__":
    main()

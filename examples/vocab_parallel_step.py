"""One training step of a tensor-parallel output layer, all ranks on one GPU.

The layer's weight is split by vocabulary over n ranks, so rank r computes the
logits of its own columns only.  The step
  1. scores the sampled tokens (`ar_logprobs`: log probability, entropy, the
     most likely alternatives) and takes a policy gradient through the ratio to
     the probabilities they were sampled with (`ar_logprobs_backward`),
  2. pulls the student towards a teacher's top entries, which `ar_logprobs`
     made from the teacher's logits (`ar_distill_grad`),
  3. turns both into the gradient of the hidden state: every rank's part is a
     product with its own weight, and their sum is an all-reduce
     (`ar_allreduce`).

    python examples/vocab_parallel_step.py [--ranks 4] [--rows 64] [--hidden 256] [--vocab 10007]
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import reduce_scatter_amd as ar  # noqa: E402


class OutputLayer:
    """The split weight, and what a program keeps from step to step: shapes,
    pointer tables, result buffers, the workspace."""

    def __init__(self, ranks, rows, hidden, vocab, alternatives=16, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.widths = ar.vocab_widths(vocab, ranks)
        self.weight = [torch.randn(w, hidden, generator=g, device="cuda").mul_(hidden ** -0.5).bfloat16()
                       for w in self.widths]
        self.shape = ar.VocabShape(rows, self.widths, "bf16")
        new = lambda: [torch.empty(rows, w, dtype=torch.bfloat16, device="cuda") for w in self.widths]
        self.logits, self.policy_grads, self.distill_grads = new(), new(), new()
        self.tables = [ar.pointers(t) for t in (self.logits, self.policy_grads, self.distill_grads)]
        f32 = lambda *s: torch.empty(s, device="cuda")
        self.logprobs, self.entropy, self.saved, self.loss = f32(rows), f32(rows), f32(rows, 4), f32(rows)
        self.top = f32(rows, alternatives)
        self.top_ids = torch.empty(rows, alternatives, dtype=torch.int64, device="cuda")
        self.dhidden = [f32(rows, hidden) for _ in self.widths]
        self.workspace = torch.empty(ar.ar_vocab_workspace(self.shape, alternatives), dtype=torch.uint8, device="cuda")

    def forward(self, hidden):
        for x, w in zip(self.logits, self.weight):
            torch.matmul(hidden, w.t(), out=x)

    def score(self, tokens):
        k = self.top.shape[1]
        ar.ar_logprobs(self.tables[0], self.shape, tokens, self.logprobs, entropy=self.entropy, top_k=k,
                       top_logprobs=self.top, top_ids=self.top_ids, saved=self.saved, workspace=self.workspace)

    def backward(self, tokens, sampled_logprobs, advantage, teacher, bonus=0.01, pull=0.1):
        """Gradient of the hidden state, in every rank's buffer."""
        rows = len(tokens)
        logits, policy, distill = self.tables
        ratio = torch.exp(self.logprobs - sampled_logprobs)
        ar.ar_logprobs_backward(logits, policy, self.shape, tokens, self.saved,
                                grad_logprobs=-advantage * ratio / rows,
                                grad_entropy=torch.full((rows,), -bonus / rows, device="cuda"))
        ar.ar_distill_grad(logits, distill, self.shape, teacher[0], teacher[1], self.loss, tail=True,
                           grad_loss=torch.full((rows,), pull / rows, device="cuda"), workspace=self.workspace)
        for out, a, b, w in zip(self.dhidden, self.policy_grads, self.distill_grads, self.weight):
            out.copy_((a + b) @ w)
        ar.ar_allreduce(self.dhidden, self.dhidden, self.dhidden[0].numel(), "f32", "sum")
        return self.dhidden


def main(argv=None):
    p = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    p.add_argument("--ranks", type=int, default=4)
    p.add_argument("--rows", type=int, default=64)
    p.add_argument("--hidden", type=int, default=256)
    p.add_argument("--vocab", type=int, default=10007)
    a = p.parse_args(argv)
    g = torch.Generator(device="cuda").manual_seed(1)
    hidden = torch.randn(a.rows, a.hidden, generator=g, device="cuda").bfloat16()
    tokens = torch.randint(0, a.vocab, (a.rows,), generator=g, device="cuda")
    advantage = torch.randn(a.rows, generator=g, device="cuda")

    teacher = OutputLayer(a.ranks, a.rows, a.hidden, a.vocab, seed=2)
    teacher.forward(hidden)
    teacher.score(tokens)
    student = OutputLayer(a.ranks, a.rows, a.hidden, a.vocab, seed=3)
    student.forward(hidden)
    student.score(tokens)
    sampled = student.logprobs + 0.05 * torch.randn(a.rows, generator=g, device="cuda")
    dhidden = student.backward(tokens, sampled, advantage, (teacher.top_ids, teacher.top))
    print("mean log probability %.4f, entropy %.4f, distillation loss %.4f, |dhidden| %.3e on every one of %d ranks"
          % (student.logprobs.mean(), student.entropy.mean(), student.loss.mean(), dhidden[0].norm(), a.ranks))
    return student, teacher, hidden, tokens, sampled, advantage, dhidden


if __name__ == "__main__":
    main()

"""The operators around a step's collectives run together: the training-step
example against the chain rule in 64 bits, and the calls captured into HIP graphs."""
from __future__ import annotations

import importlib.util
import os

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)
ar = pytest.importorskip("reduce_scatter_amd")

PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "tensor_parallel_step.py")


def example():
    spec = importlib.util.spec_from_file_location("tensor_parallel_step", PATH)
    ex = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(ex)
    return ex


def gradients64(model, ids, targets):
    """(loss, gradients, their norm) by autograd on the CPU."""
    f = lambda t: t.detach().double().cpu()
    table = torch.cat([f(t) for t in model.table]).requires_grad_()
    up, down = ([f(t).requires_grad_() for t in part] for part in (model.up, model.down))
    gains = [f(t).requires_grad_() for t in model.gains]
    ids, targets = ids.cpu(), targets.cpu()
    norm = lambda x, w: x * torch.rsqrt(x.square().mean(1, keepdim=True) + 1e-6) * w
    x0 = table[ids.clamp(min=0)] * (ids >= 0)[:, None]
    h0 = norm(x0, gains[0])
    x1 = x0 + sum(torch.relu(h0 @ u.t()) @ d.t() for u, d in zip(up, down))
    logp = torch.log_softmax(norm(x1, gains[1]) @ table.t(), 1)
    picked = torch.where(targets >= 0, logp.gather(1, targets.clamp(min=0)[:, None])[:, 0], 0.0)
    loss = -picked.mean()
    loss.backward()
    grads = [table.grad] + [t.grad for t in up + down + gains]
    return loss.item(), grads, torch.cat([g.flatten() for g in grads]).norm().item()


@pytest.mark.parametrize("ranks, tokens, hidden, vocab", [(1, 5, 64, 97), (4, 256, 128, 5003), (8, 100, 100, 1000)])
def test_step(ranks, tokens, hidden, vocab):
    """In fp32: at most eleven products stand between a weight and its gradient, each with an error of at most 512 u
    of the sum of its terms' sizes, which is at most 16 times the result's norm here (32 bits of 2-norm, not per value)."""
    model, ids, targets = example().main(["--ranks", str(ranks), "--tokens", str(tokens), "--hidden", str(hidden), "--vocab", str(vocab),
                                          "--dtype", "f32", "--max-norm", "0.05"])
    loss, want, norm = gradients64(model, ids, targets)
    tol = 11 * 512 * 2.0 ** -24 * 16
    assert abs(-model.logprobs.double().mean().item() - loss) < tol
    assert abs(model.norm.item() - norm) < tol * norm
    factor = 0.05 / (norm + 1e-6)
    assert factor < 1
    got = [torch.cat(model.grads["table"])] + model.grads["up"] + model.grads["down"] + model.grads["gains"]
    for a, b in zip(got, want):
        assert (a.double().cpu() - b * factor).norm() < tol * factor * max(b.norm().item(), 1e-3 * norm)


def test_step_runs_in_16_bits():
    model, _, _ = example().main(["--tokens", "300", "--vocab", "3001"])
    assert torch.isfinite(model.norm) and all(torch.isfinite(t).all() for part in model.grads.values() for t in part)
    total = torch.cat([t.double().flatten() for part in model.grads.values() for t in part]).norm().item()
    # every clipped value is off by at most half a step of bf16
    assert abs(total - min(0.1, model.norm.item())) < 0.1 * 2.0 ** -7


class Chain:
    """Lookup, norm of it with two partials, backward, table gradient, clipping: the buffers of one such program."""

    def __init__(self, tokens, width, vocab, seed):
        g = torch.Generator(device="cuda").manual_seed(seed)
        bf = lambda *s: torch.randn(s, generator=g, device="cuda").bfloat16()
        self.g, self.vocab = g, vocab
        entries = ar.vocab_widths(vocab, 3)
        self.table, self.partials = [bf(e, width) for e in entries], [bf(tokens, width) for _ in range(2)]
        self.weight, self.go = bf(width), bf(tokens, width)
        self.ids = torch.randint(-1, vocab, (tokens,), generator=g, device="cuda")
        self.embed, self.shape = ar.EmbedShape(tokens, entries, width, "bf16"), ar.NormShape(tokens, width, 2, "bf16", group=128)
        new = lambda *s, t=torch.bfloat16: torch.zeros(s, dtype=t, device="cuda")
        self.x, self.s, self.out, self.dx = (new(tokens, width) for _ in range(4))
        self.rstd, self.dw, self.norm = (new(n, t=torch.float32) for n in (tokens, width, 1))
        self.out8, self.scales = new(tokens, width, t=torch.uint8), new(tokens, self.shape.groups, t=torch.float32)
        self.grads = [new(e, width) for e in entries]
        self.list = ar.GradList(self.grads + [self.dw])
        self.clipped = [torch.zeros_like(t) for t in self.grads + [self.dw]]
        self.out_list = ar.GradList(self.clipped)
        space = lambda n: torch.empty(n, dtype=torch.uint8, device="cuda")
        self.spaces = [space(ar.ar_norm_workspace(self.shape)), space(ar.ar_embedding_workspace(self.embed)),
                       space(ar.ar_grad_workspace(self.list))]
        self.results = [self.x, self.s, self.out, self.dx, self.rstd, self.dw, self.norm, self.out8, self.scales, *self.grads, *self.clipped]

    def refill(self):
        for t in self.table + self.partials + [self.weight, self.go]:
            t.copy_(torch.randn(t.shape, generator=self.g, device="cuda"))
        self.ids.copy_(torch.randint(-1, self.vocab, self.ids.shape, generator=self.g, device="cuda"))

    def run(self):
        ar.ar_embedding(self.table, self.embed, self.ids, self.x)
        ar.ar_reduce_norm(self.partials, self.shape, self.weight, out=self.out, residual=self.x, summed=self.s, rstd=self.rstd,
                          out8=self.out8, scales=self.scales)
        ar.ar_reduce_norm_backward(self.s, self.shape, self.weight, self.rstd, self.go, self.dx, grad_weight=self.dw,
                                   workspace=self.spaces[0])
        ar.ar_embedding_backward(self.dx, self.embed, self.ids, self.grads, workspace=self.spaces[1])
        ar.ar_clip_grads(self.list, self.out_list, self.norm, 1.0, workspace=self.spaces[2])


@pytest.mark.parametrize("tokens, width, vocab", [(1, 64, 10), (700, 1000, 500), (12000, 136, 3000)])
def test_graphs(tokens, width, vocab):
    """Two captured programs, replayed in turn with eager runs, new inputs and synchronisations between them."""
    chains = [Chain(tokens, width, vocab, seed) for seed in (1, 2)]
    graphs = []
    for c in chains:
        c.run()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            c.run()
        graphs.append(graph)
    for _ in range(4):
        want = []
        for c in chains:
            c.refill()
            c.run()
            torch.cuda.synchronize()
            want.append([t.clone() for t in c.results])
            for t in c.results:
                t.fill_(7)
        for graph in graphs:
            graph.replay()
        torch.cuda.synchronize()
        for c, w in zip(chains, want):
            for a, b in zip(c.results, w):
                assert torch.equal(a, b)


def test_two_streams_at_once():
    """Programs of their own workspaces on two streams give what they give one after the other."""
    chains = [Chain(2000, 520, 900, seed) for seed in (3, 4)]
    want = []
    for c in chains:
        c.run()
        torch.cuda.synchronize()
        want.append([t.clone() for t in c.results])
        for t in c.results:
            t.fill_(7)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in chains]
    for _ in range(5):
        for c, s in zip(chains, streams):
            with torch.cuda.stream(s):
                c.run()
    torch.cuda.synchronize()
    for c, w in zip(chains, want):
        for a, b in zip(c.results, w):
            assert torch.equal(a, b)

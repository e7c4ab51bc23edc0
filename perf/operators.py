"""The vocabulary-split operators as measured cases: log probabilities of given
tokens (with entropy and top alternatives) and distillation from a teacher's
top logits, forward and with their gradients, on logits whose vocabulary axis
is split over n rank buffers of one GPU.

``run`` computes a case in plain torch operations, or, where ``own`` is set,
through the library's entry points; ``exact`` computes the same results from
the definitions in 64 bits.
"""
from __future__ import annotations

import math

import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
ELEM = {"f32": 4, "bf16": 2, "f16": 2}
QTAIL_MIN = 2.0 ** -20                 # a remaining teacher mass below this is rounding of its log probabilities
NEG = float("-inf")


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

def _case(name, kind, rows, vocab, n, dtype, **kw):
    c = dict(name=name, kind=kind, rows=rows, vocab=vocab, n=n, dtype=dtype, k=0, tail=False, temperature=1.0,
             pad=0, mask="none", ignore=0.0, entropy=False)
    c.update(kw)
    return c


def listed():
    return [
        # one token of one request, its five best alternatives: the latency of a serving step
        _case("score_one", "score", 1, 32768, 1, "bf16", k=5, entropy=True),
        # a decoding batch over eight vocabulary shards, twenty alternatives and the entropy
        _case("score_decode", "score", 64, 131072, 8, "bf16", k=20, entropy=True),
        # a prompt's log probabilities, odd vocabulary in a padded buffer, grammar-masked logits, a temperature
        _case("score_prompt", "score", 1021, 50021, 4, "f16", k=8, entropy=True, pad=3, mask="inf", temperature=0.8),
        # scoring a batch of sampled sequences for a policy update
        _case("score_batch", "score", 8192, 131072, 8, "bf16", entropy=True),
        # a policy step: log probabilities, ratio to the old ones, then the gradient with an entropy bonus
        _case("policy_step", "policy", 4096, 131072, 8, "bf16", entropy=True, ignore=0.1),
        # the same in 32 bits, small vocabulary, masks of the type's lowest value
        _case("policy_f32", "policy", 2000, 32000, 2, "f32", entropy=True, mask="lowest"),
        # cross-entropy of a fine-tuning batch with its gradient, odd vocabulary, padding rows
        _case("cross_entropy", "cross", 4096, 100003, 4, "bf16", ignore=0.2),
        # a teacher's lists made while it generates: sixty-four alternatives of a batch
        _case("teacher_lists", "score", 512, 131072, 8, "bf16", k=64),
        # evaluation of a student against renormalised teacher lists
        _case("distill_eval", "distill", 1000, 65536, 4, "f16", k=32, temperature=2.0),
        # a small student step: few rows, short lists
        _case("distill_small", "distill_grad", 16, 32768, 2, "f32", k=8, tail=True),
        # distillation that weighs easy tokens up: the upstream gradient depends on the loss; odd sizes, sixteen shards
        _case("distill_weighed", "distill_weighed", 777, 50021, 16, "bf16", k=100, tail=True, ignore=0.1),
        # the student's training batch
        _case("distill_train", "distill_grad", 8192, 131072, 8, "bf16", k=64, tail=True, ignore=0.05),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["score", "score", "policy", "cross", "distill", "distill_grad", "distill_weighed"])
    dtype = rng.choice(["bf16", "bf16", "f16", "f32"])
    n = rng.choice([1, 2, 3, 4, 6, 8, 16, 32])
    vocab = _log_int(rng, 1000, 260000)
    rows = min(_log_int(rng, 1, 8192), (8192 * 131072 * 2) // (2 * vocab * ELEM[dtype]))
    c = _case(None, kind, rows, vocab, n, dtype, temperature=rng.choice([1.0, 1.0, 1.3, 2.0]),
              pad=rng.choice([0, 0, 0, 1, 5, 8]), ignore=rng.choice([0.0, 0.1, 0.3]))
    del c["name"]
    if kind.startswith("distill"):
        c["k"] = _log_int(rng, 1, 200)
        c["tail"] = rng.random() < 0.5
    else:
        c["mask"] = rng.choice(["none", "none", "inf", "lowest"])
        c["entropy"] = kind == "policy" or (kind == "score" and rng.random() < 0.6)
        if kind == "score":
            c["k"] = rng.choice([0, 1, 5, 20, 33, 64])
    return c


def work(case):
    r, v, e, k = case["rows"], case["vocab"], ELEM[case["dtype"]], case["k"]
    x = r * v
    grad = case["kind"] in ("policy", "cross", "distill_grad", "distill_weighed")
    if case["kind"].startswith("distill"):
        small = r * (12 * k + 4 + (4 if grad else 0))
        flops = x * (8 if grad else 4)
    else:
        small = r * (8 + 4 + (4 if case["entropy"] else 0) + 12 * k + (12 if grad else 0))
        flops = x * ((9 if grad else 4) + (2 if case["entropy"] else 0))
    return {"bytes": x * e * (2 if grad else 1) + small, "flops": flops}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _bounds(vocab, n):
    return [r * vocab // n for r in range(n + 1)]


def _inputs(case, seed):
    """The case's data from the seed alone: rank buffers (views of padded
    rows), token ids, per-row weights, the teacher's lists."""
    g = torch.Generator(device="cuda")
    g.manual_seed(seed * 1_000_003 + 17)
    rows, vocab, k, T = case["rows"], case["vocab"], case["k"], case["temperature"]
    dt = DTYPES[case["dtype"]]
    d = {}
    randint = lambda hi, *shape: torch.randint(0, hi, shape, generator=g, device="cuda")
    rand = lambda *shape: torch.rand(shape, generator=g, device="cuda")
    randn = lambda *shape: torch.randn(shape, generator=g, device="cuda")
    targets = randint(vocab, rows)
    distill = case["kind"].startswith("distill")
    if distill:
        # distinct ids, one in each of k equal strata of the vocabulary, in a shuffled order
        step = vocab // k
        ids = (torch.arange(k, device="cuda") * step + randint(step, rows, k)).gather(
            1, torch.argsort(rand(rows, k), dim=1))
        vals = 12.0 - 1.5 * torch.log(torch.arange(1, k + 1, device="cuda").float()) + randn(rows, k)
        boost = vals + 0.7 * randn(rows, k)
        if case["tail"]:                                     # log probabilities of the full distribution
            mass = 0.6 + 0.399 * rand(rows, 1)
            vals = vals / T
            vals = vals - torch.logsumexp(vals, 1, keepdim=True) + torch.log(mass)
        drop = rand(rows, k) < 0.02                          # lists shorter than k are padded with -1
        if k > 1:
            drop[:, 0] = False
            ids = torch.where(drop, torch.full_like(ids, -1), ids)
        if case["ignore"] > 0:
            skip = rand(rows) < case["ignore"]
            ids = torch.where(skip[:, None], torch.full_like(ids, -1), ids)
        d["ids"], d["vals"] = ids.contiguous(), vals.float().contiguous()
    b = _bounds(vocab, case["n"])
    shards = []
    for r in range(case["n"]):
        w = b[r + 1] - b[r]
        buf = torch.empty(rows, w + case["pad"], dtype=dt, device="cuda")
        x = buf[:, :w]
        for lo in range(0, rows, 1024):                      # a model's logits: near zero, a heavy upper side
            hi = min(rows, lo + 1024)
            t = torch.randn(hi - lo, w, generator=g, device="cuda")
            t.mul_(2.0).add_(0.25 * t * t.abs())
            x[lo:hi] = t.to(dt)
        buf[:, w:] = 0
        shards.append(x)
    if distill:
        for r in range(case["n"]):
            inside = (d["ids"] >= b[r]) & (d["ids"] < b[r + 1])
            rr, kk = inside.nonzero(as_tuple=True)
            shards[r][rr, d["ids"][rr, kk] - b[r]] = boost[rr, kk].to(dt)
    if case["mask"] != "none":
        low = NEG if case["mask"] == "inf" else torch.finfo(dt).min
        for r in range(case["n"]):
            w = b[r + 1] - b[r]
            for lo in range(0, rows, 1024):
                hi = min(rows, lo + 1024)
                shards[r][lo:hi].masked_fill_(rand(hi - lo, w) < 0.3, low)
    if not distill:
        for r in range(case["n"]):                           # the given token is likely in most rows, never masked
            inside = (targets >= b[r]) & (targets < b[r + 1])
            rr = inside.nonzero(as_tuple=True)[0]
            shards[r][rr, targets[rr] - b[r]] = torch.where(rr % 4 != 0, 9.0, 1.0).to(dt)
    if case["mask"] != "none" and rows > 2:
        for r in range(case["n"]):
            shards[r][rows // 2] = low                       # a row whose mask leaves nothing
    if case["ignore"] > 0:
        targets = torch.where(rand(rows) < case["ignore"], torch.full_like(targets, -100), targets)
    d["targets"] = targets
    scale = 4096.0 if dt == torch.float16 else 1.0 / rows    # 16-bit halves keep small gradients by a loss scale
    d["weights"] = randn(rows) * scale
    d["bonus"] = torch.full((rows,), 0.01 * scale, device="cuda")
    if case["kind"] == "policy":                             # the policy that sampled the tokens: close to this one
        old = torch.zeros(rows, device="cuda")
        lse = torch.full((rows,), NEG, device="cuda")
        for r in range(case["n"]):
            for lo in range(0, rows, 1024):
                part = shards[r][lo:lo + 1024].float() / T
                lse[lo:lo + 1024] = torch.logaddexp(lse[lo:lo + 1024], torch.logsumexp(part, 1))
            inside = (targets >= b[r]) & (targets < b[r + 1])
            rr = inside.nonzero(as_tuple=True)[0]
            old[rr] = shards[r][rr, targets[rr] - b[r]].float() / T
        d["old"] = torch.nan_to_num(old - lse, 0.0, 0.0, 0.0) + 0.1 * randn(rows)
    d["shards"], d["bounds"] = shards, b
    return d


def prepare(case, seed):
    s = {"case": dict(case), **_inputs(case, seed)}
    if not own:
        return s
    import reduce_scatter_amd as ar
    rows, k, kind = case["rows"], case["k"], case["kind"]
    widths = [x.shape[1] for x in s["shards"]]
    pitches = [x.stride(0) for x in s["shards"]]
    s["ar"] = ar
    s["shape"] = ar.VocabShape(rows, widths, case["dtype"], pitches=pitches, grad_pitches=widths,
                               temperature=case["temperature"])
    s["logits"] = ar.pointers(s["shards"])
    f32 = lambda *shape: torch.empty(shape, dtype=torch.float32, device="cuda")
    if kind in ("policy", "cross", "distill_grad", "distill_weighed"):
        s["grads"] = [torch.empty(rows, w, dtype=DTYPES[case["dtype"]], device="cuda") for w in widths]
        s["gtable"] = ar.pointers(s["grads"])
    s["saved"] = f32(rows, 4)
    s["workspace"] = torch.empty(ar.ar_vocab_workspace(s["shape"], k if kind == "score" else 0), dtype=torch.uint8,
                                 device="cuda")
    if kind.startswith("distill"):
        s["loss"] = f32(rows)
    else:
        s["logprobs"] = f32(rows)
        s["H"] = f32(rows) if case["entropy"] else None
        if k:
            s["top"] = f32(rows, k)
            s["top_ids"] = torch.empty(rows, k, dtype=torch.int64, device="cuda")
    return s


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------

def run(s):
    return _run_own(s) if own else _run_plain(s)


def _run_own(s):
    ar, c = s["ar"], s["case"]
    kind, x, sh, ws = c["kind"], s["logits"], s["shape"], s["workspace"]
    if kind == "score":
        out = {"logprobs": s["logprobs"]}
        if c["k"]:
            ar.ar_logprobs(x, sh, s["targets"], s["logprobs"], entropy=s["H"], top_k=c["k"], top_logprobs=s["top"],
                           top_ids=s["top_ids"], workspace=ws)
            out["top_logprobs"], out["top_ids"] = s["top"], s["top_ids"]
        else:
            ar.ar_logprobs(x, sh, s["targets"], s["logprobs"], entropy=s["H"], workspace=ws)
        if c["entropy"]:
            out["entropy"] = s["H"]
        return out
    if kind == "policy":
        ar.ar_logprobs(x, sh, s["targets"], s["logprobs"], entropy=s["H"], saved=s["saved"], workspace=ws)
        g = torch.exp(s["logprobs"] - s["old"]) * s["weights"]
        ar.ar_logprobs_backward(x, s["gtable"], sh, s["targets"], s["saved"], grad_logprobs=g,
                                grad_entropy=s["bonus"])
        return {"logprobs": s["logprobs"], "entropy": s["H"], "grads": s["grads"]}
    if kind == "cross":
        ar.ar_logprobs_grad(x, s["gtable"], sh, s["targets"], s["logprobs"], grad_logprobs=s["weights"],
                            saved=s["saved"], workspace=ws)
        return {"logprobs": s["logprobs"], "grads": s["grads"]}
    if kind == "distill":
        ar.ar_distill(x, sh, s["ids"], s["vals"], s["loss"], tail=c["tail"], workspace=ws)
        return {"loss": s["loss"]}
    if kind == "distill_grad":
        ar.ar_distill_grad(x, s["gtable"], sh, s["ids"], s["vals"], s["loss"], tail=c["tail"],
                           grad_loss=s["weights"], saved=s["saved"], workspace=ws)
        return {"loss": s["loss"], "grads": s["grads"]}
    ar.ar_distill(x, sh, s["ids"], s["vals"], s["loss"], tail=c["tail"], saved=s["saved"], workspace=ws)
    g = s["weights"] / (1.0 + s["loss"])
    ar.ar_distill_backward(x, s["gtable"], sh, s["ids"], s["vals"], s["saved"], tail=c["tail"], grad_loss=g)
    return {"loss": s["loss"], "grads": s["grads"]}


def _split(s, g):
    b = s["bounds"]
    return [g[:, b[r]:b[r + 1]].to(x.dtype) for r, x in enumerate(s["shards"])]


def _stats(z):
    """Row maximum (0 for a row of -inf only), ln of the sum relative to it, exponentials, which rows are empty."""
    m = z.amax(1, keepdim=True)
    empty = m == NEG
    m = torch.where(empty, torch.zeros_like(m), m)
    d = z - m
    e = torch.exp(d)
    s = e.sum(1, keepdim=True)
    return d, e, s, torch.log(s), empty


def _run_plain(s):
    c = s["case"]
    x = torch.cat([t.float() for t in s["shards"]], 1)
    z = x if c["temperature"] == 1.0 else x / c["temperature"]
    if c["kind"].startswith("distill"):
        return _plain_distill(s, z)
    d, e, tot, ls, empty = _stats(z)
    t = s["targets"]
    valid = (t >= 0) & (t < c["vocab"])
    lp = d.gather(1, t.clamp(0, c["vocab"] - 1)[:, None]) - ls
    lp = torch.where(empty, torch.full_like(lp, NEG), lp)[:, 0]
    lp = torch.where(valid, lp, torch.zeros_like(lp))
    out = {"logprobs": lp}
    if c["entropy"]:
        H = ls - torch.where(e > 0, e * d, torch.zeros_like(d)).sum(1, keepdim=True) / tot
        H = torch.where(empty, torch.zeros_like(H), H)
    if c["k"]:
        # order by value, then by lowest id: one 64-bit key per logit
        bits = torch.where(x == 0, torch.zeros_like(x), x).view(torch.int32).to(torch.int64)
        order = torch.where(bits >= 0, bits, -(bits & 0x7FFFFFFF)) * (1 << 31)
        order = order + (2 ** 31 - 1 - torch.arange(c["vocab"], device=x.device))
        kk = min(c["k"], c["vocab"])
        ids = torch.topk(order, kk, 1).indices
        top = d.gather(1, ids) - ls
        out["top_logprobs"] = torch.where(empty, torch.full_like(top, NEG), top)
        out["top_ids"] = ids
    if c["kind"] in ("policy", "cross"):
        if c["kind"] == "policy":
            g = torch.exp(lp - s["old"]) * s["weights"]
            gh = s["bonus"][:, None]
        else:
            g, gh = s["weights"], None
        g = torch.where(valid, g, torch.zeros_like(g))[:, None]
        p = e / tot
        grad = -g * p
        if gh is not None:
            grad = grad - gh * torch.where(p > 0, p * (d - ls + H), torch.zeros_like(p))
        grad.scatter_add_(1, t.clamp(0, c["vocab"] - 1)[:, None], g)
        grad = torch.where(empty, torch.zeros_like(grad), grad / c["temperature"])
        out["grads"] = _split(s, grad)
    if c["entropy"]:
        out["entropy"] = H[:, 0]
    return out


def _plain_distill(s, z):
    c = s["case"]
    ids, vals, T = s["ids"], s["vals"], c["temperature"]
    valid = (ids >= 0) & (ids < c["vocab"])
    safe = ids.clamp(0, c["vocab"] - 1)
    neg = torch.full_like(vals, NEG)
    if c["tail"]:
        logq = torch.where(valid, vals, neg)
        q = torch.exp(logq)
        live = valid.any(1, keepdim=True)
        qt = 1.0 - q.sum(1, keepdim=True)
        qt = torch.where((qt < QTAIL_MIN) | ~live, torch.zeros_like(qt), qt)
    else:
        t = torch.where(valid, vals / T, neg)
        tm = t.amax(1, keepdim=True)
        live = tm > NEG
        t = t - torch.where(live, tm, torch.zeros_like(tm))
        te = torch.exp(t)
        ts = te.sum(1, keepdim=True).clamp(min=1e-30)
        q = te / ts
        logq = t - torch.log(ts)
        qt = torch.zeros_like(tm)
    m = z.amax(1, keepdim=True)
    d = z - m
    e = torch.exp(d)
    ls = torch.log(e.sum(1, keepdim=True))
    terms = q * (logq - (d.gather(1, safe) - ls))
    loss = torch.where(q > 0, terms, torch.zeros_like(q)).sum(1, keepdim=True)
    grad_wanted = c["kind"] != "distill"
    rest = None
    if c["tail"]:
        # the same sums without the listed ids
        keep = torch.ones_like(z, dtype=torch.bool)
        rr, kk = valid.nonzero(as_tuple=True)
        keep[rr, ids[rr, kk]] = False
        rest = torch.where(keep, e, torch.zeros_like(e))
        rsum = rest.sum(1, keepdim=True)
        # a remaining mass that the common maximum would flush to zero is summed relative to its own
        lt = torch.log(rsum)
        far = rsum < 1e-20
        if bool(far.any()):
            dm = torch.where(keep, d, torch.full_like(d, NEG))
            mm = dm.amax(1, keepdim=True)
            mm = torch.where(mm == NEG, torch.zeros_like(mm), mm)
            lt = torch.where(far, mm + torch.log(torch.exp(dm - mm).sum(1, keepdim=True)), lt)
        loss = loss + torch.where(qt > 0, qt * (torch.log(qt) - (lt - ls)), torch.zeros_like(qt))
    out = {"loss": loss[:, 0]}
    if grad_wanted:
        g = s["weights"]
        if c["kind"] == "distill_weighed":
            g = g / (1.0 + loss[:, 0])
        Q = q.sum(1, keepdim=True) + qt
        grad = Q * torch.exp(d - ls)
        if c["tail"]:
            grad = grad - torch.where(qt > 0, qt * torch.where(keep, torch.exp(d - lt), torch.zeros_like(d)),
                                      torch.zeros_like(d))
        grad.scatter_add_(1, safe, torch.where(valid, -q, torch.zeros_like(q)))
        grad = torch.where(live, grad * (g[:, None] / T), torch.zeros_like(grad))
        out["grads"] = _split(s, grad)
    return out


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------

def exact(case, seed):
    s = _inputs(case, seed)
    b, vocab, T, kind, k = s["bounds"], case["vocab"], case["temperature"], case["kind"], case["k"]
    names = {"score": ["logprobs"] + (["top_logprobs", "top_ids"] if k else []), "policy": ["logprobs"],
             "cross": ["logprobs"]}.get(kind, ["loss"])
    if case["entropy"]:
        names = names + ["entropy"]
    has_grads = kind in ("policy", "cross", "distill_grad", "distill_weighed")
    parts = {n: [] for n in names}
    grads = [torch.empty(x.shape, dtype=torch.float64, device=x.device) for x in s["shards"]] if has_grads else None
    step = max(1, (1 << 26) // vocab)
    for lo in range(0, case["rows"], step):
        hi = min(case["rows"], lo + step)
        x = torch.cat([t[lo:hi].double() for t in s["shards"]], 1)
        res, grad = (_exact_distill if kind.startswith("distill") else _exact_logprobs)(case, s, x, slice(lo, hi))
        for n in names:
            parts[n].append(res[n])
        if has_grads:
            for r in range(case["n"]):
                grads[r][lo:hi] = grad[:, b[r]:b[r + 1]]
    out = {n: torch.cat(p) for n, p in parts.items()}
    if has_grads:
        out["grads"] = grads
    # the order in which run gives them
    order = ["logprobs", "top_logprobs", "top_ids", "loss"] + (["grads", "entropy"] if kind == "policy" else
                                                              ["entropy", "grads"])
    return {n: out[n] for n in order if n in out}


def _exact_logprobs(case, s, x, rows):
    logp = torch.log_softmax(x / case["temperature"], 1)
    empty = (x == NEG).all(1)
    logp[empty] = NEG
    p = torch.exp(logp)
    plogp = torch.where(p > 0, p * logp, torch.zeros_like(p))
    H = -plogp.sum(1)
    t = s["targets"][rows]
    has = ((t >= 0) & (t < case["vocab"])).double()
    at = t.clamp(0, case["vocab"] - 1)
    lp = torch.where(has > 0, logp.gather(1, at[:, None])[:, 0], torch.zeros_like(H))
    res = {"logprobs": lp, "entropy": H}
    if case["k"]:
        ids = torch.sort(x, dim=1, descending=True, stable=True).indices[:, :case["k"]]
        res["top_ids"], res["top_logprobs"] = ids, logp.gather(1, ids)
    grad = None
    if case["kind"] in ("policy", "cross"):
        w = s["weights"][rows].double()
        g = (w * torch.exp(lp - s["old"][rows].double()) if case["kind"] == "policy" else w) * has
        grad = p * -g[:, None]
        if case["kind"] == "policy":
            grad -= s["bonus"][rows].double()[:, None] * (plogp + p * H[:, None])
        grad[torch.arange(len(t), device=x.device), at] += g
        grad[empty] = 0
        grad /= case["temperature"]
    return res, grad


def _exact_distill(case, s, x, rows):
    T, vocab = case["temperature"], case["vocab"]
    ids, vals = s["ids"][rows], s["vals"][rows].double()
    valid = (ids >= 0) & (ids < vocab)
    r = torch.arange(len(ids), device=x.device)[:, None].expand_as(ids)
    # the teacher spread over the vocabulary
    t = vals if case["tail"] else torch.log_softmax(torch.where(valid, vals / T, torch.full_like(vals, NEG)), 1)
    q = torch.where(valid, torch.exp(t), torch.zeros_like(t))
    live = valid.any(1)
    q[~live] = 0
    full = torch.zeros_like(x).index_put_((r[valid], ids[valid]), q[valid], accumulate=True)
    logp = torch.log_softmax(x / T, 1)
    lpk = logp.gather(1, ids.clamp(0, vocab - 1))
    loss = torch.where(q > 0, torch.xlogy(q, q) - q * lpk, torch.zeros_like(q)).sum(1)
    grad = torch.exp(logp)
    if case["tail"]:
        qt = 1 - q.sum(1)
        qt = torch.where((qt < QTAIL_MIN) | ~live, torch.zeros_like(qt), qt)
        out = torch.ones_like(x, dtype=torch.bool).index_put_((r[valid], ids[valid]),
                                                              torch.tensor(False, device=x.device))
        rest = torch.where(out, logp, torch.full_like(logp, NEG))
        lt = torch.logsumexp(rest, 1)
        loss = loss + torch.where(qt > 0, torch.xlogy(qt, qt) - qt * lt, torch.zeros_like(qt))
        grad *= (q.sum(1) + qt)[:, None]
        cond = torch.softmax(rest, 1)
        grad -= torch.where(qt[:, None] > 0, qt[:, None] * cond, torch.zeros_like(cond))
    else:
        grad *= q.sum(1)[:, None]
    grad -= full
    g = s["weights"][rows].double()
    if case["kind"] == "distill_weighed":
        g = g / (1 + loss)
    grad *= (g / T)[:, None]
    grad[~live] = 0
    return {"loss": loss}, grad

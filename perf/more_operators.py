"""The operators around the collectives of a tensor-parallel step as measured
cases: the sum of the ranks' partial results with the residual, RMS norm and an
8-bit output, and its backward pass; the embedding lookup from a table split by
vocabulary entries over the ranks, and its gradient; the global gradient norm
with clipping.

``run`` computes a case in plain torch operations, or, where ``own`` is set,
through the library's entry points; ``exact`` computes the same results from
the definitions in 64 bits.
"""
from __future__ import annotations

import math
import random

import numpy as np
import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16, "e4m3": torch.float8_e4m3fn}
ELEM = {"f32": 4, "bf16": 2, "f16": 2}
E4M3_MAX = 448.0
LEAST_SCALE = 2.0 ** -100               # a group of zeros has this scale
CLIP_EPS = 1e-6


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

def _norm(name, rows, width, n, dtype, **kw):
    c = dict(name=name, kind="norm", rows=rows, width=width, n=n, dtype=dtype, weight=dtype, pad=0, residual=True,
             out=True, eight=False, group=0, rstd=False, offset=0.0, eps=1e-6, empty=0.0)
    c.update(kw)
    return c


def _norm_back(name, rows, width, dtype, **kw):
    c = dict(name=name, kind="norm_back", rows=rows, width=width, n=1, dtype=dtype, weight=dtype, pad=0, residual=True,
             offset=0.0, eps=1e-6, empty=0.0)
    c.update(kw)
    return c


def _embed(name, kind, tokens, vocab, n, width, table, act, **kw):
    c = dict(name=name, kind=kind, tokens=tokens, vocab=vocab, n=n, width=width, table=table, act=act, pad=0,
             scale=1.0, ignore=0.0)
    c.update(kw)
    return c


def _clip(name, tensors, least, most, dtype, **kw):
    c = dict(name=name, kind="clip", tensors=tensors, least=least, most=most, dtype=dtype, spread=1, max_norm=1.0,
             scale=1.0)
    c.update(kw)
    return c


def listed():
    return [
        # one token of one request: eight ranks' partial sums into the residual stream, the next layer's input
        _norm("norm_one", 1, 4096, 8, "bf16"),
        # a decoding batch whose next product takes 8 bits with a scale to every 128 columns
        _norm("norm_decode", 64, 8192, 8, "bf16", out=False, eight=True, group=128),
        # a prompt: odd width in padded buffers, weights in 32 bits around one, 8 bits with a scale to each row
        _norm("norm_prompt", 3001, 5003, 4, "f16", weight="f32", pad=5, eight=True, offset=1.0, empty=0.1),
        # a training batch: what the backward pass needs is stored as well
        _norm("norm_train", 16384, 8192, 8, "bf16", rstd=True),
        # the same layer's backward pass, the residual stream's gradient coming in as well
        _norm_back("norm_back", 16384, 8192, "bf16"),
        # a small batch in 32 bits, odd sizes, a last norm without a residual behind it
        _norm_back("norm_back_odd", 777, 5003, "f32", residual=False, empty=0.1),
        # the input of a decoding step from a table over eight ranks
        _embed("embed_decode", "embed", 32, 131072, 8, 8192, "bf16", "bf16"),
        # a prompt's input from a table in 32 bits, scaled, odd vocabulary
        _embed("embed_prompt", "embed", 16384, 50021, 4, 5120, "f32", "bf16", scale=71.55, pad=4, ignore=0.1),
        # a fine-tuning batch's gradient of the table, in 32 bits
        _embed("embed_back_small", "embed_back", 1021, 32000, 2, 4096, "f32", "bf16", ignore=0.2),
        # a pre-training batch's gradient
        _embed("embed_back", "embed_back", 65536, 131072, 8, 4096, "bf16", "bf16"),
        # adapters: many small gradients
        _clip("clip_adapters", 448, 1000, 200_000, "f32", max_norm=0.5),
        # a model's gradients: matrices in 16 bits, norm weights in 32, unscaled from a loss scale
        _clip("clip_model", 300, 4096, 40_000_000, "mixed", scale=2.0 ** -10),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["norm", "norm", "norm_back", "norm_back", "embed", "embed_back", "embed_back", "clip"])
    dtype = rng.choice(["bf16", "bf16", "f16", "f32"])
    if kind in ("norm", "norm_back"):
        width = rng.choice([_log_int(rng, 64, 16384), 128 * _log_int(rng, 1, 128)])
        n = rng.choice([1, 2, 3, 4, 8, 16]) if kind == "norm" else 1
        most = (16384 * 8192 * 2 * 8) // (width * ELEM[dtype] * (n + 3))
        rows = _log_int(rng, 1, min(most, 1 << 18))
        common = dict(weight=rng.choice([dtype, "f32"]), pad=rng.choice([0, 0, 0, 1, 8]), residual=rng.random() < 0.7,
                      offset=rng.choice([0.0, 1.0]), eps=rng.choice([1e-5, 1e-6]), empty=rng.choice([0.0, 0.2]))
        if kind == "norm_back":
            c = _norm_back(None, rows, width, dtype, **common)
        else:
            eight = rng.random() < 0.5
            c = _norm(None, rows, width, n, dtype, eight=eight, group=rng.choice([0, 32, 64, 128, 256, 512]) if eight else 0,
                      out=not eight or rng.random() < 0.3, rstd=rng.random() < 0.5, **common)
    elif kind in ("embed", "embed_back"):
        width = rng.choice([_log_int(rng, 64, 8192), 128 * _log_int(rng, 1, 64)])
        vocab = min(_log_int(rng, 500, 260000), (131072 * 8192) // width)
        table = rng.choice([dtype, "f32"])
        if kind == "embed_back":
            vocab = max(1, min(vocab, (131072 * 4096 * 2) // (width * ELEM[table])))
        tokens = _log_int(rng, 1, min(1 << 18, (65536 * 4096 * 2) // (width * ELEM[dtype])))
        c = _embed(None, kind, tokens, vocab, rng.choice([1, 2, 3, 4, 8, 16]), width, table, dtype,
                   pad=rng.choice([0, 0, 0, 1, 8]), scale=rng.choice([1.0, 1.0, 45.25]), ignore=rng.choice([0.0, 0.1, 0.4]))
    else:
        least = _log_int(rng, 1, 10000)
        most = _log_int(rng, least + 1, 20_000_000)
        tensors = _log_int(rng, 1, min(1500, max(2, 600_000_000 // most)))
        c = _clip(None, tensors, least, most, rng.choice(["bf16", "f16", "f32", "mixed"]), spread=rng.randrange(1 << 20),
                  max_norm=rng.choice([0.1, 1.0, 1e6]), scale=rng.choice([1.0, 2.0 ** -10]))
    del c["name"]
    return c


def _distinct(tokens, vocab):
    """Expected number of distinct ids among `tokens` draws of _tokens()."""
    v = np.arange(vocab, dtype=np.float64)
    p = np.log((v + 2) / (v + 1)) / math.log(vocab + 1)
    return float(-np.expm1(tokens * np.log1p(-np.minimum(p, 1 - 1e-12))).sum())


def _sizes(case):
    """Elements of every gradient, sizes spread evenly over their logarithm; the smaller ones of a mixed list are in 32 bits."""
    rng = random.Random(case["spread"])
    sizes = [_log_int(rng, case["least"], case["most"]) for _ in range(case["tensors"])]
    border = math.sqrt(case["least"] * case["most"])
    types = [("f32" if s < border else "bf16") if case["dtype"] == "mixed" else case["dtype"] for s in sizes]
    return sizes, types


def work(case):
    kind = case["kind"]
    if kind == "norm":
        r, w, e = case["rows"], case["width"], ELEM[case["dtype"]]
        x = r * w
        tensors = case["n"] + (2 if case["residual"] else 0) + (1 if case["out"] else 0)
        small = w * ELEM[case["weight"]] + (4 * r if case["rstd"] else 0)
        if case["eight"]:
            small += x + 4 * r * (-(-w // case["group"]) if case["group"] else 1)
        return {"bytes": x * e * tensors + small, "flops": x * (case["n"] + 5 + (3 if case["eight"] else 0))}
    if kind == "norm_back":
        r, w, e = case["rows"], case["width"], ELEM[case["dtype"]]
        return {"bytes": r * w * e * (4 if case["residual"] else 3) + 4 * r + w * (ELEM[case["weight"]] + 4),
                "flops": r * w * 11}
    if kind == "embed":
        t, w = case["tokens"] * (1 - case["ignore"]), case["width"]
        return {"bytes": _distinct(t, case["vocab"]) * w * ELEM[case["table"]] + case["tokens"] * (w * ELEM[case["act"]] + 8),
                "flops": t * w}
    if kind == "embed_back":
        t, w = case["tokens"] * (1 - case["ignore"]), case["width"]
        return {"bytes": t * w * ELEM[case["act"]] + case["tokens"] * 8 + case["vocab"] * w * ELEM[case["table"]],
                "flops": t * w}
    sizes, types = _sizes(case)
    return {"bytes": 2 * sum(s * ELEM[t] for s, t in zip(sizes, types)), "flops": 3 * sum(sizes)}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed * 1_000_003 + 29)
    return g


def _rows_of(g, rows, width, dtype, pad, sigma):
    """[rows, width] normal values, rows `pad` elements further apart than their width."""
    buf = torch.zeros(rows, width + pad, dtype=DTYPES[dtype], device="cuda")
    step = max(1, (1 << 26) // width)
    for lo in range(0, rows, step):
        hi = min(rows, lo + step)
        buf[lo:hi, :width] = (torch.randn(hi - lo, width, generator=g, device="cuda") * sigma).to(buf.dtype)
    return buf[:, :width]


def _bounds(vocab, n):
    return [r * vocab // n for r in range(n + 1)]


def _tokens(g, case):
    """Token ids as a text has them: the id's logarithm is even, so few ids make up most of it; -1 where there is none."""
    t, vocab = case["tokens"], case["vocab"]
    u = torch.rand(t, generator=g, device="cuda", dtype=torch.float64)
    ids = (torch.exp(u * math.log(vocab + 1)) - 1).long().clamp(0, vocab - 1)
    skip = torch.rand(t, generator=g, device="cuda") < case["ignore"]
    return torch.where(skip, torch.full_like(ids, -1), ids)


def _norm_inputs(case, seed):
    g, rows, width, dtype = _generator(seed), case["rows"], case["width"], case["dtype"]
    d = {}
    gone = torch.rand(rows, generator=g, device="cuda") < case["empty"]      # rows of padding: nothing but zeros
    columns = 0.5 + torch.rand(width, generator=g, device="cuda")            # a residual stream's columns differ in size,
    columns[torch.randint(0, width, (3,), generator=g, device="cuda")] = 30.0   # a few by far
    w = 1.0 + 0.2 * torch.randn(width, generator=g, device="cuda") - case["offset"]
    d["weight"] = w.to(DTYPES[case["weight"]])
    if case["kind"] == "norm":
        d["partials"] = [_rows_of(g, rows, width, dtype, case["pad"], 0.3) for _ in range(case["n"])]
        d["residual"] = None
        if case["residual"]:
            d["residual"] = _rows_of(g, rows, width, dtype, 0, 1.0).mul_(columns.to(DTYPES[dtype]))
        for x in d["partials"] + ([d["residual"]] if case["residual"] else []):
            x.masked_fill_(gone[:, None], 0.0)
        return d
    d["x"] = _rows_of(g, rows, width, dtype, case["pad"], 1.0).mul_(columns.to(DTYPES[dtype]))
    d["x"].masked_fill_(gone[:, None], 0.0)
    sigma = 1.0 if dtype == "f16" else 1e-3                                   # 16-bit halves carry a loss scale
    d["grad_out"] = _rows_of(g, rows, width, dtype, 0, sigma)
    d["grad_summed"] = _rows_of(g, rows, width, dtype, 0, sigma) if case["residual"] else None
    d["grad_out"].masked_fill_(gone[:, None], 0.0)
    d["rstd"] = torch.cat([torch.rsqrt(x.float().square().mean(1) + case["eps"]) for x in d["x"].split(4096)])
    return d


def _embed_inputs(case, seed):
    g, width = _generator(seed), case["width"]
    b = _bounds(case["vocab"], case["n"])
    d = {"tokens": _tokens(g, case), "bounds": b}
    if case["kind"] == "embed":
        d["tables"] = [_rows_of(g, b[r + 1] - b[r], width, case["table"], case["pad"], 0.02) for r in range(case["n"])]
    else:
        d["grad_out"] = _rows_of(g, case["tokens"], width, case["act"], 0, 1.0 if case["act"] == "f16" else 1e-3)
    return d


def _clip_inputs(case, seed):
    """Gradients as views of one flat buffer to a type, one behind the other."""
    g = _generator(seed)
    sizes, types = _sizes(case)
    d = {"flat": {}, "grads": [], "sizes": {}}
    for t in sorted(set(types)):
        mine = [s for s, u in zip(sizes, types) if u == t]
        flat = torch.empty(sum(mine), dtype=DTYPES[t], device="cuda")
        for lo in range(0, flat.numel(), 1 << 27):
            hi = min(flat.numel(), lo + (1 << 27))
            flat[lo:hi] = (torch.randn(hi - lo, generator=g, device="cuda") * (1e-3 / case["scale"])).to(flat.dtype)
        d["flat"][t], d["sizes"][t] = flat, mine
        d["grads"] += list(flat.split(mine))
    return d


def prepare(case, seed):
    kind = case["kind"]
    inputs = {"norm": _norm_inputs, "norm_back": _norm_inputs, "embed": _embed_inputs, "embed_back": _embed_inputs,
              "clip": _clip_inputs}[kind]
    s = {"case": dict(case), **inputs(case, seed)}
    if not own:
        return s
    import reduce_scatter_amd as ar
    s["ar"] = ar
    new = lambda *shape, dtype="f32": torch.empty(shape, dtype=DTYPES[dtype], device="cuda")
    space = lambda size: torch.empty(size, dtype=torch.uint8, device="cuda")
    if kind in ("norm", "norm_back"):
        rows, width, dtype = case["rows"], case["width"], case["dtype"]
        first = s["partials"][0] if kind == "norm" else s["x"]
        s["shape"] = ar.NormShape(rows, width, case["n"], dtype, pitches=[first.stride(0)] * case["n"],
                                  weight_dtype=case["weight"], eps=case["eps"], offset=case["offset"],
                                  group=case.get("group", 0))
        if kind == "norm":
            s["table"] = ar.pointers(s["partials"])
            s["out"] = new(rows, width, dtype=dtype) if case["out"] else None
            s["summed"] = new(rows, width, dtype=dtype) if case["residual"] else None
            s["rstd"] = new(rows) if case["rstd"] else None
            s["out8"] = new(rows, width, dtype="e4m3") if case["eight"] else None
            s["scales"] = new(rows, -(-width // case["group"]) if case["group"] else 1) if case["eight"] else None
        else:
            s["grad_x"], s["grad_weight"] = new(rows, width, dtype=dtype), new(width)
            s["workspace"] = space(ar.ar_norm_workspace(s["shape"]))
    elif kind in ("embed", "embed_back"):
        entries = [hi - lo for lo, hi in zip(s["bounds"], s["bounds"][1:])]
        pitches = [case["width"] + case["pad"]] * case["n"]
        s["shape"] = ar.EmbedShape(case["tokens"], entries, case["width"], case["table"], out_dtype=case["act"],
                                   pitches=pitches, grad_pitches=[case["width"]] * case["n"], scale=case["scale"])
        if kind == "embed":
            s["table"] = ar.pointers(s["tables"])
            s["out"] = new(case["tokens"], case["width"], dtype=case["act"])
        else:
            s["grads"] = [new(e, case["width"], dtype=case["table"]) for e in entries]
            s["table"] = ar.pointers(s["grads"])
            s["workspace"] = space(ar.ar_embedding_workspace(s["shape"]))
    else:
        s["outs"] = {t: torch.empty_like(f) for t, f in s["flat"].items()}
        s["list"] = ar.GradList(s["grads"])
        s["out_list"] = ar.GradList([o for t in sorted(s["outs"]) for o in s["outs"][t].split(s["sizes"][t])])
        s["norm"] = new(1)
        s["workspace"] = space(ar.ar_grad_workspace(s["list"]))
    return s


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------

def run(s):
    return _run_own(s) if own else _run_plain(s)


def _run_own(s):
    ar, c = s["ar"], s["case"]
    kind = c["kind"]
    if kind == "norm":
        ar.ar_reduce_norm(s["table"], s["shape"], s["weight"], out=s["out"], residual=s["residual"], summed=s["summed"],
                          rstd=s["rstd"], out8=s["out8"], scales=s["scales"])
        return {k: s[k] for k in ("out", "summed", "rstd", "out8", "scales") if s[k] is not None}
    if kind == "norm_back":
        ar.ar_reduce_norm_backward(s["x"], s["shape"], s["weight"], s["rstd"], s["grad_out"], s["grad_x"],
                                   grad_summed=s["grad_summed"], grad_weight=s["grad_weight"], workspace=s["workspace"])
        return {"grad_x": s["grad_x"], "grad_weight": s["grad_weight"]}
    if kind == "embed":
        ar.ar_embedding(s["table"], s["shape"], s["tokens"], s["out"])
        return {"out": s["out"]}
    if kind == "embed_back":
        ar.ar_embedding_backward(s["grad_out"], s["shape"], s["tokens"], s["table"], workspace=s["workspace"])
        return {"grads": s["grads"]}
    ar.ar_clip_grads(s["list"], s["out_list"], s["norm"], c["max_norm"], scale=c["scale"], eps=CLIP_EPS,
                     workspace=s["workspace"])
    return {"norm": s["norm"], "grads": s["outs"]}


def _scale8(y, group):
    """y / scale and the scales: the largest of a row, or of a group of columns, stands for E4M3_MAX."""
    rows, width = y.shape
    g = group or width
    short = -width % g
    z = torch.nn.functional.pad(y, (0, short)) if short else y
    z = z.view(rows, -1, g)
    scale = (z.abs().amax(2, keepdim=True) / E4M3_MAX).clamp_min(LEAST_SCALE)
    return (z / scale).reshape(rows, -1)[:, :width], scale[:, :, 0]


def _run_plain(s):
    c = s["case"]
    kind = c["kind"]
    if kind == "norm":
        parts = [p.float() for p in ([s["residual"]] if c["residual"] else []) + s["partials"]]
        x = sum(parts[1:], parts[0])
        rstd = torch.rsqrt(x.square().mean(1, keepdim=True) + c["eps"])
        y = x * rstd * (s["weight"].float() + c["offset"])
        out = {}
        if c["out"]:
            out["out"] = y.to(DTYPES[c["dtype"]])
        if c["residual"]:
            out["summed"] = x.to(DTYPES[c["dtype"]])
        if c["rstd"]:
            out["rstd"] = rstd[:, 0]
        if c["eight"]:
            q, out["scales"] = _scale8(y, c["group"])
            out["out8"] = q.to(DTYPES["e4m3"])
        return out
    if kind == "norm_back":
        rstd, g = s["rstd"][:, None], s["grad_out"].float()
        h = s["x"].float() * rstd
        u = g * (s["weight"].float() + c["offset"])
        dx = rstd * (u - h * (u * h).mean(1, keepdim=True))
        if c["residual"]:
            dx = dx + s["grad_summed"].float()
        return {"grad_x": dx.to(DTYPES[c["dtype"]]), "grad_weight": (g * h).sum(0)}
    if kind == "embed":
        t, b = s["tokens"], s["bounds"]
        inside = [((t >= lo) & (t < hi))[:, None] for lo, hi in zip(b, b[1:])]
        # every rank's part of the rows, zeros where another holds the entry
        parts = [torch.where(i, x[(t - lo).clamp(0, x.shape[0] - 1)].float(), 0.0) for i, x, lo in zip(inside, s["tables"], b)]
        return {"out": (sum(parts[1:], parts[0]) * c["scale"]).to(DTYPES[c["act"]])}
    if kind == "embed_back":
        t = s["tokens"]
        at = torch.where((t >= 0) & (t < c["vocab"]), t, c["vocab"])
        grad = torch.zeros(c["vocab"] + 1, c["width"], device="cuda").index_add_(0, at, s["grad_out"].float())
        grad = (grad * c["scale"]).to(DTYPES[c["table"]])
        return {"grads": [grad[lo:hi] for lo, hi in zip(s["bounds"], s["bounds"][1:])]}
    flat = s["flat"]
    total = sum([f.float().square().sum(dtype=torch.float64) for f in flat.values()])
    norm = (total.sqrt() * c["scale"]).float()
    factor = (c["max_norm"] / (norm + CLIP_EPS)).clamp(max=1.0) * c["scale"]
    return {"norm": norm.reshape(1), "grads": {t: (f.float() * factor).to(f.dtype) for t, f in flat.items()}}


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------

def exact(case, seed):
    kind = case["kind"]
    f64 = lambda t: t.to(torch.float64)
    if kind in ("norm", "norm_back"):
        d, rows, width = _norm_inputs(case, seed), case["rows"], case["width"]
        w = f64(d["weight"]) + case["offset"]
        step = max(1, (1 << 25) // width)
        kept, dw = {}, torch.zeros(width, dtype=torch.float64, device="cuda")
        keep = lambda k, v: kept.setdefault(k, []).append(v)
        for lo in range(0, rows, step):
            at = slice(lo, min(rows, lo + step))
            if kind == "norm_back":
                r = f64(d["rstd"][at])[:, None]
                g, h = f64(d["grad_out"][at]), f64(d["x"][at]) * r
                dot = torch.linalg.vecdot(g * w, h)[:, None] / width
                dx = r * (g * w - dot * h)
                keep("grad_x", dx + f64(d["grad_summed"][at]) if case["residual"] else dx)
                dw += (g * h).sum(0)
                continue
            x = torch.zeros(at.stop - at.start, width, dtype=torch.float64, device="cuda")
            for p in d["partials"] + ([d["residual"]] if case["residual"] else []):
                x += p[at]
            r = 1.0 / torch.sqrt(torch.linalg.vecdot(x, x) / width + case["eps"])
            y = x * w * r[:, None]
            if case["out"]:
                keep("out", y)
            if case["residual"]:
                keep("summed", x)
            if case["rstd"]:
                keep("rstd", r)
            if case["eight"]:
                size = case["group"] or width
                scales = torch.stack([p.abs().amax(1) for p in y.split(size, 1)], 1) / E4M3_MAX
                scales = torch.where(scales < LEAST_SCALE, torch.full_like(scales, LEAST_SCALE), scales)
                keep("scales", scales)
                # before the rounding to 8 bits
                keep("out8", y / scales.repeat_interleave(size, 1)[:, :width])
        out = {k: torch.cat(v) for k, v in kept.items()}
        if kind == "norm_back":
            out["grad_weight"] = dw
        return out
    if kind == "embed":
        d = _embed_inputs(case, seed)
        out = torch.zeros(case["tokens"], case["width"], dtype=torch.float64, device="cuda")
        for r, x in enumerate(d["tables"]):
            rows = ((d["tokens"] >= d["bounds"][r]) & (d["tokens"] < d["bounds"][r + 1])).nonzero()[:, 0]
            out[rows] = f64(x[d["tokens"][rows] - d["bounds"][r]]) * case["scale"]
        return {"out": out}
    if kind == "embed_back":
        d = _embed_inputs(case, seed)
        grads = []
        for lo, hi in zip(d["bounds"], d["bounds"][1:]):
            rows = ((d["tokens"] >= lo) & (d["tokens"] < hi)).nonzero()[:, 0]
            part = torch.zeros(hi - lo, case["width"], dtype=torch.float64, device="cuda")
            for some in rows.split(8192):
                part.index_put_((d["tokens"][some] - lo,), f64(d["grad_out"][some]) * case["scale"], accumulate=True)
            grads.append(part)
        return {"grads": grads}
    d = _clip_inputs(case, seed)
    norm = case["scale"] * math.sqrt(sum(float(f64(p).square().sum()) for f in d["flat"].values() for p in f.split(1 << 26)))
    factor = case["scale"] * min(1.0, case["max_norm"] / (norm + CLIP_EPS))
    return {"norm": torch.tensor([norm], dtype=torch.float64),
            "grads": {t: torch.cat([f64(p) * factor for p in f.split(1 << 26)]) for t, f in d["flat"].items()}}

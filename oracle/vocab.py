"""Reductions over a vocabulary axis in 64 bits (numpy), from the definitions
in ``include/ar_vocab.h``: log probabilities with entropy and top
alternatives, distillation from a teacher's top entries, and their gradients.
``x`` is the whole [rows, V] array of logits."""
from __future__ import annotations

import numpy as np

TAIL_LEAST = 2.0 ** -20


def log_softmax(x, temperature=1.0):
    """(ln p, rows without a distribution); a NaN or +inf makes its row NaN."""
    x = np.asarray(x, dtype=np.float64)
    with np.errstate(all="ignore"):
        m = np.where(np.isnan(x).any(1), np.nan, np.max(np.where(np.isnan(x), -np.inf, x), axis=1))[:, None]
        empty = (m == -np.inf)[:, 0]
        d = (x - np.where(empty[:, None], 0.0, m)) / temperature
        d[np.isposinf(m[:, 0])] = np.nan
        logp = d - np.log(np.exp(d).sum(1, keepdims=True))
    logp[empty] = -np.inf
    return logp, empty


def entropy(logp):
    with np.errstate(all="ignore"):
        p = np.exp(logp)
        return -np.where(p == 0, 0.0, p * logp).sum(1)


def logprobs(logp, targets):
    has = (targets >= 0) & (targets < logp.shape[1])
    lp = logp[np.arange(len(targets)), np.where(has, targets, 0)]
    return np.where(has, lp, 0.0)


def top(x, logp, k):
    """(ids, ln p) of the k largest logits: equal ones by lowest id, NaN as -inf, -1 / -inf past V."""
    key = np.where(np.isnan(x), -np.inf, np.asarray(x, dtype=np.float64))
    order = np.argsort(-key, axis=1, kind="stable")[:, :k]
    ids = np.full((len(x), k), -1, dtype=np.int64)
    lps = np.full((len(x), k), -np.inf)
    ids[:, :order.shape[1]] = order
    lps[:, :order.shape[1]] = np.take_along_axis(logp, order, 1)
    return ids, lps


def logprobs_grad(x, temperature, targets, gl, gh):
    logp, empty = log_softmax(x, temperature)
    rows, vocab = logp.shape
    has = (targets >= 0) & (targets < vocab)
    gl = np.where(has, gl, 0.0)[:, None]
    gh = np.broadcast_to(np.asarray(gh, dtype=np.float64), rows)[:, None]
    with np.errstate(all="ignore"):
        p = np.exp(logp)
        inner = np.where(p == 0, 0.0, p * (logp + entropy(logp)[:, None]))
        onehot = np.zeros_like(p)
        onehot[np.arange(rows)[has], targets[has]] = 1.0
        g = (gl * (onehot - p) - gh * inner) / temperature
    g[empty | ((gl == 0) & (gh == 0))[:, 0]] = 0.0
    return g


def teacher(ids, values, vocab, tail, temperature):
    """(q, ln q, valid, q_t, rows with a teacher) of [rows, K] entries."""
    valid = (ids >= 0) & (ids < vocab)
    v = np.where(valid, np.asarray(values, dtype=np.float64), -np.inf)
    with np.errstate(all="ignore"):
        if tail:
            lq, live = v, valid.any(1)
            qt = 1.0 - np.exp(lq).sum(1)
            qt = np.where(qt < TAIL_LEAST, 0.0, qt)
        else:
            m = v.max(1)
            live = m > -np.inf
            d = (v - np.where(live, m, 0.0)[:, None]) / temperature
            lq = d - np.log(np.exp(d).sum(1, keepdims=True))
            qt = np.zeros(len(ids))
    lq = np.where(live[:, None], lq, -np.inf)
    return np.exp(lq), lq, valid, np.where(live, qt, 0.0), live


def _unlisted(ids, valid, vocab):
    out = np.ones((len(ids), vocab), dtype=bool)
    r, k = np.nonzero(valid)
    out[r, ids[r, k]] = False
    return out


def _by_id(ids, valid, q, vocab):
    """[rows, V] probabilities of the teacher: a repeated id adds its entries'."""
    dense = np.zeros((len(ids), vocab))
    r, k = np.nonzero(valid)
    np.add.at(dense, (r, ids[r, k]), q[r, k])
    return dense


def distill(x, temperature, ids, values, tail):
    """(loss, ln p at the listed ids, ln of the unlisted mass)."""
    logp, _ = log_softmax(x, temperature)
    vocab = logp.shape[1]
    q, lq, valid, qt, live = teacher(ids, values, vocab, tail, temperature)
    at = np.where(valid, ids, 0)
    lpk = np.take_along_axis(logp, at, 1)
    with np.errstate(all="ignore"):
        # an id that stands once keeps the logarithm it was given
        dense = _by_id(ids, valid, q, vocab)
        total = np.take_along_axis(dense, at, 1)
        loss = np.where(q == 0, 0.0, q * (np.where(total == q, lq, np.log(total)) - lpk)).sum(1)
        rest = np.where(_unlisted(ids, valid, vocab), logp, -np.inf)
        m = rest.max(1)
        lt = np.where(m == -np.inf, -np.inf, m + np.log(np.exp(rest - np.where(m == -np.inf, 0, m)[:, None]).sum(1)))
        loss = loss + np.where(qt == 0, 0.0, qt * (np.log(qt) - lt))
    return np.where(live, loss, 0.0), lpk, lt


def distill_grad(x, temperature, ids, values, tail, g):
    logp, empty = log_softmax(x, temperature)
    rows, vocab = logp.shape
    q, _, valid, qt, live = teacher(ids, values, vocab, tail, temperature)
    dense = _by_id(ids, valid, q, vocab)
    with np.errstate(all="ignore"):
        out = (q.sum(1) + qt)[:, None] * np.exp(logp) - dense
        # shares of the unlisted mass against its own largest entry: at -1e38 a logarithm has lost their number
        rest = np.where(_unlisted(ids, valid, vocab), np.asarray(x, dtype=np.float64), -np.inf)
        most = rest.max(1, keepdims=True)
        share = np.exp((rest - np.where(most == -np.inf, 0.0, most)) / temperature)
        cond = np.where(rest == -np.inf, 0.0, share / share.sum(1, keepdims=True))
        out = (out - qt[:, None] * cond) * (np.asarray(g, dtype=np.float64) / temperature)[:, None]
    out[empty | ~live | (np.asarray(g) == 0)] = 0.0
    return out

"""The operators around a step's collectives in 64 bits (numpy), from the
definitions in ``include/ar_layer.h``: reduction with residual and RMS norm,
embedding over a split vocabulary, the gradient norm, and their gradients.
Inputs are whole arrays of any float type."""
from __future__ import annotations

import numpy as np

E4M3_MAX = 448.0
LEAST_SCALE = 2.0 ** -100


def _f64(a):
    return np.asarray(a, dtype=np.float64)


def reduce_norm(partials, weight, residual=None, eps=1e-6, offset=0.0):
    """(s, rstd, y)."""
    s = sum(_f64(p) for p in partials) + (0.0 if residual is None else _f64(residual))
    with np.errstate(all="ignore"):
        rstd = 1.0 / np.sqrt((s * s).mean(1) + eps)
        return s, rstd, s * rstd[:, None] * (offset + _f64(weight))


def scales(y, group=0):
    """[rows, groups]: what stands for 448, NaN where some value is not finite."""
    rows, width = y.shape
    g = group or width
    out = []
    for c in range(0, width, g):
        m = np.abs(y[:, c:c + g]).max(1)
        out.append(np.where(np.isfinite(m), np.maximum(m / E4M3_MAX, LEAST_SCALE), np.nan))
    return np.stack(out, 1)


def reduce_norm_backward(x, weight, rstd, grad_out, grad_summed=None, offset=0.0):
    """(grad_x, grad_weight)."""
    with np.errstate(all="ignore"):
        h = _f64(x) * _f64(rstd)[:, None]
        g = _f64(grad_out)
        u = g * (offset + _f64(weight))
        dx = _f64(rstd)[:, None] * (u - h * (u * h).mean(1, keepdims=True))
        if grad_summed is not None:
            dx = dx + _f64(grad_summed)
        return dx, (g * h).sum(0)


def embedding(table, tokens, scale=1.0):
    ok = (tokens >= 0) & (tokens < len(table))
    return np.where(ok[:, None], _f64(table)[np.where(ok, tokens, 0)] * scale, 0.0)


def embedding_backward(grad_out, tokens, vocab, scale=1.0):
    out = np.zeros((vocab, grad_out.shape[1]))
    ok = (tokens >= 0) & (tokens < vocab)
    np.add.at(out, tokens[ok], _f64(grad_out)[ok] * scale)
    return out


def grad_norm(grads, scale=1.0):
    return scale * np.sqrt(sum(float((_f64(g) ** 2).sum()) for g in grads))


def clip(grads, max_norm, scale=1.0, eps=1e-6):
    """(norm, the factor of every element)."""
    norm = grad_norm(grads, scale)
    with np.errstate(all="ignore"):
        f = np.float64(max_norm) / (norm + eps)            # 0 / 0 is not below 1 either
    return norm, scale * (norm if np.isnan(norm) else f if f < 1.0 else 1.0)

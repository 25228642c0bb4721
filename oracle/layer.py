"""Float64 oracle of the norm, embedding, attention and clipping operators (CPU, numpy).

Each function is the operator's definition, written out directly; gradients are the
formulas that differentiating it gives. Test infrastructure only.
"""
import numpy as np


def rms_norm(s, weight=None, eps=1e-6):
    """(y, rstd) of rows s."""
    s = np.asarray(s, np.float64)
    rstd = 1.0 / np.sqrt(np.mean(s * s, axis=1) + eps)
    y = s * rstd[:, None]
    return (y if weight is None else y * np.asarray(weight, np.float64)), rstd


def rms_norm_backward(dy, s, weight, rstd, dsum=None):
    """(dx, dweight) for the given rstd."""
    dy, s = np.asarray(dy, np.float64), np.asarray(s, np.float64)
    n = s * np.asarray(rstd, np.float64)[:, None]
    g = dy if weight is None else dy * np.asarray(weight, np.float64)
    dx = np.asarray(rstd, np.float64)[:, None] * (g - n * np.mean(g * n, axis=1, keepdims=True))
    if dsum is not None:
        dx = dx + np.asarray(dsum, np.float64)
    return dx, np.sum(dy * n, axis=0)


def embedding(ids, table, scale=1.0):
    ids, table = np.asarray(ids, np.int64), np.asarray(table, np.float64)
    has = (ids >= 0) & (ids < len(table))
    return np.where(has[..., None], scale * table[np.where(has, ids, 0)], 0.0)


def embedding_backward(dy, ids, vocab, scale=1.0):
    """(gradient, sum of magnitudes, tokens) of each row of the table."""
    ids = np.asarray(ids, np.int64).reshape(-1)
    dy = np.asarray(dy, np.float64).reshape(len(ids), -1)
    has = (ids >= 0) & (ids < vocab)
    out, mag = np.zeros((vocab, dy.shape[1])), np.zeros((vocab, dy.shape[1]))
    np.add.at(out, ids[has], scale * dy[has])
    np.add.at(mag, ids[has], np.abs(scale * dy[has]))
    return out, mag, np.bincount(ids[has], minlength=vocab)


def clip(grads, max_norm, sumsq=None):
    """(norm, clipped gradients)."""
    grads = [np.asarray(g, np.float64) for g in grads]
    total = sum(float(np.sum(g * g)) for g in grads) if sumsq is None else sumsq
    norm = np.sqrt(total)
    factor = min(1.0, max_norm / (norm + 1e-6))
    return norm, [g * factor for g in grads]

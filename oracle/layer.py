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


def _sequences(offsets, tokens):
    """(first, end) of each sequence: clamped, an offset that falls counts as the largest before it."""
    if offsets is None:
        return [(0, tokens)]
    at = np.maximum.accumulate(np.clip(np.asarray(offsets, np.int64), 0, tokens))
    return list(zip(at[:-1], at[1:]))


def _hidden(n, causal, window):
    far = np.arange(n)[:, None] - np.arange(n)
    hidden = np.zeros((n, n), bool)
    if causal:
        hidden |= far < 0
        if window:
            hidden |= far >= window
    return hidden


def attention_heads(q, k, v, offsets=None, causal=True, window=0, scale=None):
    """Per sequence and query head: (rows, head, key head, scores, probabilities, lse)."""
    q, k, v = (np.asarray(t, np.float64) for t in (q, k, v))
    scale = q.shape[2] ** -0.5 if scale is None else scale
    group = q.shape[1] // k.shape[1]
    for b, e in _sequences(offsets, q.shape[0]):
        if e <= b:
            continue
        hidden = _hidden(e - b, causal, window)
        for h in range(q.shape[1]):
            s = np.where(hidden, -np.inf, scale * (q[b:e, h] @ k[b:e, h // group].T))
            top = s.max(axis=1, keepdims=True)
            p = np.exp(s - top)
            total = p.sum(axis=1, keepdims=True)
            yield slice(b, e), h, h // group, s, p / total, (top + np.log(total))[:, 0]


def attention(q, k, v, **how):
    """(out, lse); zeros outside the sequences."""
    q, v = np.asarray(q, np.float64), np.asarray(v, np.float64)
    out, lse = np.zeros(q.shape), np.zeros((q.shape[1], q.shape[0]))
    for rows, h, kv, _, p, l in attention_heads(q, k, v, **how):
        out[rows, h] = p @ v[rows, kv]
        lse[h, rows] = l
    return out, lse


def attention_backward(do, q, k, v, scale=None, **how):
    """(dq, dk, dv); zeros outside the sequences."""
    do, q, k, v = (np.asarray(t, np.float64) for t in (do, q, k, v))
    scale = q.shape[2] ** -0.5 if scale is None else scale
    dq, dk, dv = np.zeros(q.shape), np.zeros(k.shape), np.zeros(k.shape)
    for rows, h, kv, _, p, _ in attention_heads(q, k, v, scale=scale, **how):
        g = do[rows, h]
        dv[rows, kv] += p.T @ g
        dp = g @ v[rows, kv].T
        ds = p * (dp - np.sum(p * dp, axis=1, keepdims=True))
        dq[rows, h] = scale * (ds @ k[rows, kv])
        dk[rows, kv] += scale * (ds.T @ q[rows, h])
    return dq, dk, dv

"""Float64 oracle of routing, expert order and combination (numpy, test infrastructure).

Written token by token from the definitions."""
from __future__ import annotations

import numpy as np

LOWEST = np.finfo(np.float64).min


def scores(logits: np.ndarray, score: str) -> np.ndarray:
    l = logits.astype(np.float64)
    with np.errstate(all="ignore"):
        if score == "sigmoid":
            return 1.0 / (1.0 + np.exp(-l))
        m = np.fmax.reduce(l, axis=1, keepdims=True)
        s = np.where(l == -np.inf, 0.0, np.exp(l - m))
        return np.where(l == -np.inf, 0.0, s / s.sum(axis=1, keepdims=True))


def route(logits, top_k, score="softmax", bias=None, n_groups=1, top_groups=1, group_top=2, renormalize=True,
          scale=1.0):
    """(ids, weights): slots without an expert have id -1 and weight 0."""
    T, E = logits.shape
    s = scores(logits, score)
    ids = np.full((T, top_k), -1, np.int64)
    w = np.zeros((T, top_k))
    per = E // n_groups
    for t in range(T):
        key = s[t] + (0.0 if bias is None else bias.astype(np.float64))
        key = np.where(np.isnan(key), LOWEST, key)
        key = np.where(logits[t] == -np.inf, -np.inf, key)
        if n_groups > 1:
            best = []
            for g in range(n_groups):
                k = sorted((k for k in key[g * per:(g + 1) * per] if k > -np.inf), reverse=True)[:group_top]
                # two NaN keys together stay the lowest number (their sum would be -inf, no key)
                best.append((-max(LOWEST, k[0] if k[0] == LOWEST else sum(k)) if k else np.inf, g))
            kept = [g for v, g in sorted(best)[:top_groups] if v < np.inf]
            key = np.where(np.isin(np.arange(E) // per, kept), key, -np.inf)
        order = sorted((-k, e) for e, k in enumerate(key) if k > -np.inf)[:top_k]
        for j, (_, e) in enumerate(order):
            ids[t, j], w[t, j] = e, s[t, e]
        if renormalize:
            w[t] /= w[t].sum() + 1e-20
    w = w * scale
    w[ids < 0] = 0.0
    return ids, w


def route_backward(dweights, logits, ids, score="softmax", renormalize=True, scale=1.0):
    T, E = logits.shape
    s = scores(logits, score)
    out = np.zeros((T, E))
    for t in range(T):
        slots = [j for j, e in enumerate(ids[t]) if 0 <= e < E]
        total = sum(s[t, ids[t, j]] for j in slots) + 1e-20
        dot = sum(dweights[t, j] * s[t, ids[t, j]] for j in slots)
        ds = np.zeros(E)
        for j in slots:
            d = dweights[t, j]
            ds[ids[t, j]] = scale * ((d - dot / total) / total if renormalize else d)
        if score == "sigmoid":
            out[t] = ds * s[t] * (1.0 - s[t])
        else:
            out[t] = s[t] * (ds - (ds * s[t]).sum())
        out[t][logits[t] == -np.inf] = 0.0
    return out


def expert_order(ids, n_experts, align, capacity):
    flat = np.asarray(ids).reshape(-1)
    slots = [[] for _ in range(n_experts)]
    for i, e in enumerate(flat):
        if 0 <= e < n_experts:
            slots[e].append(i)
    offsets, rows, pos = [0], np.full(capacity, -1), np.full(len(flat), -1)
    for s in slots:
        for r, i in enumerate(s):
            rows[offsets[-1] + r] = i
            pos[i] = offsets[-1] + r
        offsets.append(offsets[-1] + -(-len(s) // align) * align)
    return np.array(offsets), np.array([len(s) for s in slots]), rows, pos.reshape(np.shape(ids))


def combine(o, pos, weights):
    """(y, the sum of the terms' magnitudes)."""
    y, mag = np.zeros((len(pos), o.shape[1])), np.zeros((len(pos), o.shape[1]))
    for t in range(len(pos)):
        for j, r in enumerate(pos[t]):
            if 0 <= r < len(o):
                y[t] += weights[t, j] * o[r]
                mag[t] += np.abs(weights[t, j] * o[r])
    return y, mag


def combine_backward(dy, o, pos, weights):
    """(dweights, magnitude of its terms, do, rows of do that are written)."""
    dw, mag = np.zeros(weights.shape), np.zeros(weights.shape)
    do, written = np.zeros(o.shape), np.zeros(len(o), bool)
    for t in range(len(pos)):
        for j, r in enumerate(pos[t]):
            if 0 <= r < len(o):
                dw[t, j] = dy[t] @ o[r]
                mag[t, j] = np.abs(dy[t] * o[r]).sum()
                do[r] = weights[t, j] * dy[t]
                written[r] = True
    return dw, mag, do, written

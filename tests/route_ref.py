"""Plain binary64 forms of the routing and of its weights' gradient (numpy)."""
from __future__ import annotations

import numpy as np


def _clean(logits):
    l = np.array(logits, dtype=np.float64)
    l[np.isnan(l)] = -np.inf
    big = float(np.finfo(np.float32).max)
    return np.minimum(l, big)


def scores(logits, score):
    """(scores, available) of every expert: [T][E]."""
    l = _clean(logits)
    live = l > -np.inf
    s = np.zeros_like(l)
    for t in range(l.shape[0]):
        on = live[t]
        if not on.any():
            continue
        if score == "softmax":
            z = np.exp(l[t, on] - l[t, on].max())
            s[t, on] = z / z.sum()
        else:
            with np.errstate(over="ignore"):
                s[t, on] = 1.0 / (1.0 + np.exp(-l[t, on]))
    return s, live


def route(logits, k, score="softmax", bias=None, n_groups=1, keep_groups=1, group_top=1, renorm=True, scale=1.0):
    """idx [T][k], g [T][k] (binary64), one row at a time."""
    s, live = scores(logits, score)
    l = _clean(logits)
    T, E = l.shape
    gs = E // n_groups
    # without a bias the logits order the experts (both scores increase with them)
    key = s + bias if bias is not None else (s if group_top == 2 and n_groups > 1 else l)
    key = np.where(live, key, -np.inf)
    idx = np.full((T, k), -1, dtype=np.int64)
    g = np.zeros((T, k))
    for t in range(T):
        allowed = list(range(E))
        if n_groups > 1:
            rank = []
            for j in range(n_groups):
                v = sorted((key[t, e] for e in range(j * gs, (j + 1) * gs) if live[t, e]), reverse=True)[:group_top]
                rank.append(sum(v) if v else -np.inf)
            kept = sorted(range(n_groups), key=lambda j: (-rank[j], j))[:keep_groups]
            allowed = [e for e in range(E) if e // gs in kept]
        order = sorted((e for e in allowed if live[t, e]), key=lambda e: (-key[t, e], e))[:k]
        w = np.array([s[t, e] for e in order])
        if renorm and len(w):
            w = w / w.sum() if w.sum() > 0 else 0 * w
        idx[t, :len(order)] = order
        g[t, :len(order)] = w * scale
    return idx, g


def weights(logits, idx, score, renorm, scale):
    """The weights of a given choice, as a function of the logits alone (for differences)."""
    s, live = scores(logits, score)
    g = np.zeros(idx.shape)
    for t in range(idx.shape[0]):
        w = np.array([s[t, e] if e >= 0 and live[t, e] else 0.0 for e in idx[t]])
        if renorm:
            w = w / w.sum() if w.sum() > 0 else 0 * w
        g[t] = w * scale
    return g


def route_backward(logits, idx, dg, score="softmax", renorm=True, scale=1.0):
    """dLoss/dlogits [T][E] from the chain rule through the scores."""
    s, live = scores(logits, score)
    l = _clean(logits)
    T, E = l.shape
    out = np.zeros((T, E))
    for t in range(T):
        on = [(int(e), float(d)) for e, d in zip(idx[t], dg[t]) if 0 <= e < E and live[t, e]]
        tot = sum(s[t, e] for e, _ in on)
        if not on or (renorm and not tot > 0):
            continue
        ds = np.zeros(E)
        mean = sum(d * s[t, e] for e, d in on) / tot if renorm else 0.0
        for e, d in on:
            ds[e] += scale * ((d - mean) / tot if renorm else d)
        if score == "softmax":
            dl = s[t] * (ds - (ds * s[t]).sum())
        else:
            z = np.exp(-np.abs(np.where(live[t], l[t], 0.0)))
            dl = ds * z / (1 + z) ** 2
        out[t, live[t]] = dl[live[t]]
    return out

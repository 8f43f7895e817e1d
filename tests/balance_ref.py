"""Plain binary64 balance loss, its counts, and its gradient (torch, CPU)."""
from __future__ import annotations

import math

import torch


def scores(l, score):
    """(p, slope, log sum, available, live) of binary64 logits; slope: d s / d l over s."""
    l = torch.where(torch.isnan(l), -math.inf, l).clamp(max=3.402823466e38)
    on = l > -math.inf
    live = on.any(1)
    top = torch.where(live, l.amax(1), 0.0)[:, None]
    if score == "softmax":
        w, slope = torch.exp(l - top), torch.ones_like(l)
    else:  # over e^top where that is small: it cancels
        cut = top.clamp(max=0.0)
        w = torch.exp(torch.minimum(l, torch.zeros(())) - cut) / (1 + torch.exp(-l.abs()))
        slope = torch.sigmoid(-l)
    w = torch.where(on, w, 0.0)
    tot = w.sum(1, keepdim=True)
    p = torch.where(live[:, None], w / torch.where(tot > 0, tot, 1.0), 0.0)
    lse = torch.where(live, top[:, 0] + torch.log(torch.where(tot > 0, tot, 1.0))[:, 0], 0.0)
    return p, slope, lse, on, live


def borders(T, offsets):
    return [0, T] if offsets is None else [int(v) for v in offsets]


def balance(l, idx, score="softmax", alpha=1.0, zeta=0.0, offsets=None):
    """(loss [2], counts [S][E], rows [S], probs [S][E])."""
    T, E = l.shape
    k = idx.shape[1]
    p, _, lse, on, live = scores(l.double(), score)
    b = borders(T, offsets)
    S = len(b) - 1
    counts, rows = torch.zeros((S, E), dtype=torch.int64), torch.zeros(S, dtype=torch.int64)
    probs, loss = torch.zeros((S, E), dtype=torch.float64), torch.zeros(2, dtype=torch.float64)
    for q in range(S):
        for t in range(b[q], b[q + 1]):
            for e in idx[t].tolist():
                if 0 <= e < E and on[t, e]:
                    counts[q, e] += 1
        cut = slice(b[q], b[q + 1])
        n = int(live[cut].sum())
        rows[q] = n
        if n:
            probs[q] = p[cut].sum(0) / n
            loss[0] += alpha / S * (E / (k * n) * counts[q] * probs[q]).sum()
            loss[1] += zeta / S / n * lse[cut].square().sum()
    return loss, counts, rows, probs


def backward(l, counts, rows, k, score="softmax", alpha=1.0, zeta=0.0, offsets=None, dloss=(1.0, 1.0)):
    """(dlogits, a bound of fp32's errors in it), zero in rows of no sequence."""
    T, E = l.shape
    l = l.double()
    p, slope, lse, on, live = scores(l, score)
    b = borders(T, offsets)
    S = len(b) - 1
    dl, tol = torch.zeros_like(l), torch.zeros_like(l)
    U = 2.0 ** -24
    for q in range(S):
        cut = slice(b[q], b[q + 1])
        n = max(int(rows[q]), 1)
        u = dloss[0] * alpha / S * E / (k * n * n) * counts[q].double()
        z = 2 * dloss[1] * zeta / S / n * lse[cut, None]
        if score == "softmax":
            z = z + 0 * p[cut]
        else:
            z = 0 * p[cut]
        pc = p[cut]
        dot = (u * pc).sum(1, keepdim=True)
        dl[cut] = torch.where(on[cut], pc * slope[cut] * (u - dot) + z * pc, 0.0)
        rel, rel_dot = relative(l[cut], pc, score), None
        rel_dot = (u.abs() * pc * (rel + 16 * U)).sum(1, keepdim=True)
        # u and z are rounded once each, the difference, the products and the sum once more
        tol[cut] = pc * slope[cut] * ((rel + 6 * U) * (u - dot).abs() + rel_dot + 3 * U * (u.abs() + dot.abs()))
        tol[cut] += (rel + 6 * U) * (z * pc).abs() + 2 * U * abs(dloss[1] * zeta) * pc * 40 / n
    return dl, tol


def relative(l, p, score):
    """A bound of the relative error of an fp32 p: the exponent's rounding, |x| 2^-24 of the
    result, for e and on average over the row; the exponential, reciprocals, products and the
    row's sum (eight and six additions), 2^-23 or 2^-24 each: 48 of 2^-24 together."""
    top = torch.where(torch.isfinite(l), l, -math.inf).amax(1, keepdim=True)
    d = torch.where(l > -math.inf, (l - torch.where(top > -math.inf, top, 0.0)).abs(), 0.0)
    if score == "sigmoid":
        d = torch.maximum(d, torch.where(torch.isfinite(l), l.abs(), 0.0))
    d = d.clamp(max=200.0)
    return 2.0 ** -24 * (d + (p * d).sum(1, keepdim=True) + 48)

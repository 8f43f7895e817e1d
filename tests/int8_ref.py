"""Plain 8-bit products (torch, CPU): codes by exact comparisons, whole-number sums, binary64 factors."""
from __future__ import annotations

import torch


def codes(v):
    """(q, scale fp32) of binary64 rows: 127 for the largest magnitude, a half towards 0."""
    v = v.double()
    fin = torch.isfinite(v).all(1)
    v = torch.where(fin[:, None], v, 0.0)
    top = v.abs().amax(1, keepdim=True)
    at = v.abs() * 127 / torch.where(top > 0, top, 1.0)
    q = torch.ceil(at - 0.5) * torch.sign(v)
    return q.to(torch.int64), torch.where(fin, (top[:, 0] / 127).float(), float("nan"))


def product(q, s, W, w_scale):
    """s sum q W w_scale, exact sums (binary64: below 2^53)."""
    acc = q.double() @ W.double().t()
    return acc * s.double()[:, None] * (1.0 if w_scale is None else w_scale.double()[None, :])


def forward(x, W, w_scale):
    q, s = codes(x)
    return product(q, s, W, w_scale)


def backward(dys, Ws, w_scales):
    """dx of the problems that share an input."""
    q, s = codes(torch.cat([dy.double() * w.double() for dy, w in zip(dys, w_scales)], 1))
    return product(q, s, torch.cat([W for W in Ws]).t(), None)

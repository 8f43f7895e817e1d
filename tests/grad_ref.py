"""Plain binary64 gradients of the SGMM, with the magnitudes their error bounds go by (torch, CPU)."""
from __future__ import annotations

import torch


def backward(x, idx, g, A, B, dy, scale):
    """(dx share, dA, dB, dg) and the same sums over magnitudes, one row and slot at a time by expert."""
    x, A, B, dy, g = (t.detach().cpu().double() for t in (x, A, B, dy, g))
    idx = idx.cpu()
    T, E = x.shape[0], A.shape[0]
    out = [torch.zeros_like(x), torch.zeros_like(A), torch.zeros_like(B), torch.zeros((T, 2), dtype=torch.float64)]
    mag = [torch.zeros_like(t) for t in out]
    for e in range(E):
        for k in (0, 1):
            t = (idx[:, k] == e).nonzero().flatten()
            if not len(t):
                continue
            c = scale * g[t, k, None]
            u, w = x[t] @ A[e].t(), dy[t] @ B[e]
            out[0][t] += (c * w) @ A[e]
            out[1][e] += (c * w).t() @ x[t]
            out[2][e] += dy[t].t() @ (c * u)
            out[3][t, k] += scale * (u * w).sum(1)
            ua, wa = x[t].abs() @ A[e].abs().t(), dy[t].abs() @ B[e].abs()
            mag[0][t] += (c.abs() * wa) @ A[e].abs()
            mag[1][e] += (c.abs() * wa).t() @ x[t].abs()
            mag[2][e] += dy[t].abs().t() @ (c.abs() * ua)
            mag[3][t, k] += abs(scale) * (ua * wa).sum(1)
    return out, mag


def forward(x, idx, g, A, B, scale):
    """The product itself, for differences."""
    x, A, B, g = (t.detach().cpu().double() for t in (x, A, B, g))
    y = torch.zeros((x.shape[0], B.shape[1]), dtype=torch.float64)
    for t in range(x.shape[0]):
        for k in (0, 1):
            e = int(idx[t, k])
            if e >= 0:
                y[t] += scale * g[t, k] * (B[e] @ (A[e] @ x[t]))
    return y

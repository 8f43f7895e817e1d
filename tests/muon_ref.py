"""Plain forms of the orthogonalised momentum step (numpy, binary64): by the singular values, which the
polynomial acts on, and by the products themselves."""
from __future__ import annotations

import numpy as np

COEFS = (3.4445, -4.7750, 2.0315)


def by_values(u, eps, coefs):
    """X of a matrix from its singular value decomposition; coefs: one triple per step."""
    a, s, b = np.linalg.svd(u, full_matrices=False)
    s = s / (np.sqrt((u * u).sum()) + eps)
    for ca, cb, cc in coefs:
        s = s * (ca + cb * s ** 2 + cc * s ** 4)
    return (a * s) @ b


def by_products(u, eps, coefs):
    x = u / (np.sqrt((u * u).sum()) + eps)
    for ca, cb, cc in coefs:
        q = x @ x.T
        x = ca * x + (cb * q + cc * q @ q) @ x
    return x


def growth(coefs):
    """The largest factor that the steps put on a direction: the derivative at 0."""
    return float(np.prod([abs(c[0]) for c in coefs]))


def momentum(g, m, beta, nesterov, gscale=1.0):
    """(m, u) as fp32 arithmetic with fused multiply-adds gives them (in binary64, rounded once each)."""
    f = np.float32
    b, r = f(beta).astype(np.float64), f(1.0 - beta).astype(np.float64)
    inc = f(r * f(f(g) * f(gscale)).astype(np.float64)).astype(np.float64)
    m1 = f(b * m.astype(np.float64) + inc)
    return m1, (f(b * m1.astype(np.float64) + inc) if nesterov else m1)

"""Plain binary64 AdamW and the 8-bit moments' codes (numpy)."""
from __future__ import annotations

import numpy as np

BLOCK = 256
U32 = np.uint64(0xFFFFFFFF)


def mix(x):
    x = np.asarray(x, dtype=np.uint64) & U32
    x = ((x ^ (x >> np.uint64(16))) * np.uint64(0x85EBCA6B)) & U32
    x = ((x ^ (x >> np.uint64(13))) * np.uint64(0xC2B2AE35)) & U32
    return x ^ (x >> np.uint64(16))


def noise(seed, t, tensor, n):
    """The two 16-bit numbers of every element: functions of seed, step, tensor, block and place in the block."""
    i = np.arange(n, dtype=np.uint64)
    key = mix(np.uint64((seed + t * 0x9E3779B1) & 0xFFFFFFFF))
    key = mix(key + np.uint64((tensor * 0x85EBCA77) & 0xFFFFFFFF))
    key = mix(key + (i // np.uint64(BLOCK)) * np.uint64(0xC2B2AE3D))
    h = mix(key + (i % np.uint64(BLOCK)) * np.uint64(0x9E3779B1))
    return (h & np.uint64(0xFFFF)).astype(np.float64), (h >> np.uint64(16)).astype(np.float64)


def decode(q, c, ms, vs):
    n = len(q)
    b = np.arange(n) // BLOCK
    q, c = q.astype(np.float64), c.astype(np.float64)
    return (ms.astype(np.float64)[b] * (q * np.abs(q) / 127.0 ** 2),
            vs.astype(np.float64)[b] * (c ** 4 / 255.0 ** 4))


def _block_max(x):
    nb = -(-len(x) // BLOCK)
    pad = np.zeros(nb * BLOCK)
    pad[:len(x)] = x
    return pad.reshape(nb, BLOCK).max(1).astype(np.float32)


def encode(m, v, seed, t, tensor):
    """(q, c, ms, vs) of exact moments."""
    n = len(m)
    b = np.arange(n) // BLOCK
    hm, hv = noise(seed, t, tensor, n)
    ms, vs = _block_max(np.abs(m)), _block_max(v)
    with np.errstate(divide="ignore", invalid="ignore"):
        xm = np.where(ms[b] > 0, np.abs(m) * (127.0 ** 2 / ms.astype(np.float64)[b]), 0.0)
        xv = np.where(vs[b] > 0, v * (255.0 ** 4 / vs.astype(np.float64)[b]), 0.0)
    xm, xv = np.minimum(xm, 127.0 ** 2), np.minimum(xv, 255.0 ** 4)
    steps = np.arange(257, dtype=np.float64)
    q = np.searchsorted(steps ** 2, xm, side="right") - 1
    c = np.searchsorted(steps ** 4, xv, side="right") - 1
    q = q + ((xm - steps[q] ** 2) > (hm + 0.5) / 65536 * (2 * q + 1))
    c = c + ((xv - steps[c] ** 4) > (hv + 0.5) / 65536 * (steps[c + 1] ** 4 - steps[c] ** 4))
    c = np.where((v > 0) & (vs[b] > 0), np.maximum(c, 1), c)
    return (np.sign(m) * q).astype(np.int8), c.astype(np.uint8), ms, vs


def moments(g, m, v, beta1, beta2):
    return beta1 * m + (1 - beta1) * g, beta2 * v + (1 - beta2) * g * g


def update(w, m, v, t, lr, beta1, beta2, eps, wd):
    """(new weight, the step taken) in binary64."""
    s = (m / (1 - beta1 ** t)) / (np.sqrt(v / (1 - beta2 ** t)) + eps)
    return w * (1 - lr * wd) - lr * s, s

"""CPU oracles of the residual's norms and of dropout, written from their definitions in NumPy (float64); they share
no code with the library.

``add_norm`` and its gradient also return, per value, the sum of the magnitudes it is made of: what an fp32
computation's rounding errors are relative to."""
from __future__ import annotations

import math

import numpy as np


def philox(counters, offset, seed):
    """Philox4x32-10 under the key `seed`, counter words (low, high) of `counters` and of `offset`: uint32 [n, 4]."""
    low = np.uint64(0xFFFFFFFF)
    g = np.array(counters, np.uint64)
    half = np.uint64(32)
    c = [g & low, g >> half, np.full_like(g, offset & 0xFFFFFFFF), np.full_like(g, offset >> 32)]
    k = [seed & 0xFFFFFFFF, seed >> 32]
    for _ in range(10):
        a, b = c[0] * np.uint64(0xD2511F53), c[2] * np.uint64(0xCD9E8D57)
        c = [(b >> half) ^ c[1] ^ np.uint64(k[0]), b & low, (a >> half) ^ c[3] ^ np.uint64(k[1]), a & low]
        k = [(k[0] + 0x9E3779B9) & 0xFFFFFFFF, (k[1] + 0xBB67AE85) & 0xFFFFFFFF]
    return np.stack(c, 1).astype(np.uint32)


def factors(n, p, seed, offset=0):
    """What each of n elements is multiplied with: 0 or 1 / (1 - p), p in steps of 2^-16."""
    border = math.floor(p * 65536 + 0.5)
    w = philox(range(-(-n // 8)), offset, seed)
    bits = np.stack([w & 0xFFFF, w >> 16], 2).reshape(-1)[:n].astype(np.int64)
    return np.where(bits >= border, 65536 / (65536 - border) if border < 65536 else 0.0, 0.0)


def add_norm(y, r, w_pre, w_post, gate, f, eps):
    """(r_out, x, magnitudes of r_out, reciprocal rms of y and r_out); f: scale x dropout factors, of y's shape.
    Without w_pre x is None."""
    inv1 = 1 / np.sqrt((y * y).mean(1, keepdims=True) + eps) if w_post is not None else np.ones((len(y), 1))
    u = y * inv1 * (w_post if w_post is not None else 1.0)
    branch = f * (gate if gate is not None else 1.0) * u
    ro = r + branch
    inv2 = 1 / np.sqrt((ro * ro).mean(1, keepdims=True) + eps) if w_pre is not None else np.ones((len(y), 1))
    x = ro * inv2 * w_pre if w_pre is not None else None
    return ro, x, np.abs(r) + np.abs(branch), inv1, inv2


def add_norm_grad(y, r, w_pre, w_post, gate, f, eps, dx, dro):
    """{name: (value, magnitudes)} of dy, dr, dw_post, dw_pre, dgate (elementwise; sum its rows for a gate [d])."""
    ro, _, mro, inv1, inv2 = add_norm(y, r, w_pre, w_post, gate, f, eps)
    d = y.shape[1]
    g = gate if gate is not None else np.ones_like(y)
    w1 = w_post if w_post is not None else np.ones(d)
    n1, n2, m2 = y * inv1, ro * inv2, mro * inv2
    zero = np.zeros_like(y)
    dx = zero if dx is None else dx
    dro = zero if dro is None else dro
    a = dx * (w_pre if w_pre is not None else 0.0)
    mean = lambda v: v.mean(1, keepdims=True)  # noqa: E731
    D, mD = dro.copy(), np.abs(dro)
    if w_pre is not None:
        D = D + inv2 * (a - n2 * mean(a * n2))
        mD = mD + inv2 * (np.abs(a) + m2 * mean(np.abs(a) * m2))
    q = f * g * w1
    e = q * D
    dy, mdy = e, np.abs(q) * mD
    if w_post is not None:
        dy = inv1 * (e - n1 * mean(e * n1))
        mdy = inv1 * (np.abs(q) * mD + np.abs(n1) * mean(np.abs(q * n1) * mD))
    return {"dy": (dy, mdy), "dr": (D, mD), "dw_post": (f * g * D * n1, np.abs(f * g * n1) * mD),
            "dw_pre": (dx * n2, np.abs(dx) * m2), "dgate": (f * D * n1 * w1, np.abs(f * n1 * w1) * mD)}

"""CPU oracles of the operators around the vocabulary table, written from their
definitions in NumPy (float64, running sums in extended precision); they share
no code with the library."""
from __future__ import annotations

import numpy as np


def embed_rows(ids, W, scale):
    """scale x W[ids] in float64; zero rows for ids outside [0, V)."""
    ids = np.asarray(ids).reshape(-1)
    out = np.zeros((ids.size, W.shape[1]))
    for n, v in enumerate(ids):
        if 0 <= v < W.shape[0]:
            out[n] = np.float64(np.float32(scale)) * W[v].astype(np.float64)
    return out


def embed_grad(ids, dY, V, scale):
    """(dW [V, d], the sums of |scale dY| and the counts behind each row) in float64."""
    ids = np.asarray(ids).reshape(-1)
    dY = np.asarray(dY, np.float64).reshape(ids.size, -1)
    dW, mag, count = np.zeros((V, dY.shape[1])), np.zeros((V, dY.shape[1])), np.zeros(V, np.int64)
    for n, v in enumerate(ids):
        if 0 <= v < V:
            dW[v] += dY[n]
            mag[v] += np.abs(dY[n])
            count[v] += 1
    s = np.float64(np.float32(scale))
    return dW * s, mag * abs(s), count


def sample_row(logits, u, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0):
    """(id, log-probability) of one row by the definition: the tokens in the order
    (logit descending, id ascending), the shortest of the three prefixes, and the
    first token whose cumulative mass exceeds u times the prefix's."""
    x = np.where(np.isnan(logits), -np.inf, np.asarray(logits, np.float64))
    ids = np.flatnonzero(x > -np.inf)
    if ids.size == 0:
        return -1, -np.inf
    order = ids[np.lexsort((ids, -x[ids]))]
    top = x[order[0]]
    if not temperature > 0:
        return int(order[0]), 0.0
    if top == np.inf:
        e = (x[order] == np.inf).astype(np.longdouble)
    else:
        with np.errstate(over="ignore", under="ignore"):
            e = np.exp((x[order].astype(np.longdouble) - top) / np.longdouble(temperature))
    c = np.cumsum(e)
    n = order.size
    keep = min(int(top_k), n) if top_k > 0 else n
    mass_k = c[keep - 1]
    if top_p < 1:
        keep = min(keep, int(np.argmax(c >= np.longdouble(max(top_p, 0.0)) * mass_k)) + 1)
    if min_p > 0:
        keep = min(keep, max(1, int(np.sum(e >= min(min_p, 1.0)))))
    u = min(max(float(u), 0.0), 1.0 - 2.0 ** -24) if u == u else 0.0
    j = int(np.argmax(c[:keep] > np.longdouble(u) * c[keep - 1]))
    return int(order[j]), float(np.log(e[j] / c[keep - 1]))

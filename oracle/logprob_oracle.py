"""CPU oracle of the log-probabilities of given tokens, entropy, alternatives and their gradients, written from the
definitions in NumPy (float64); it shares no code with the library."""
from __future__ import annotations

import numpy as np


def row_stats(z):
    """(M, L, entropy, p, log p) of logits [N, V]; a row of -inf alone has M = -inf, L = 0, entropy 0, p 0."""
    z = np.asarray(z, np.float64)
    with np.errstate(invalid="ignore", divide="ignore", over="ignore"):
        M = z.max(1)
        none = M == -np.inf
        d = np.where(none[:, None], -np.inf, z - np.where(none, 0.0, M)[:, None])
        e = np.exp(d)
        S = e.sum(1)
        L = np.where(none, 0.0, np.log(np.where(none, 1.0, S)))
        logp = d - L[:, None]
        p = np.exp(logp)
        H = L - np.where(e > 0, e * d, 0.0).sum(1) / np.where(none, 1.0, S)
    return M, L, np.where(none, 0.0, H), p, logp


def given(logp, ids):
    """log p of the ids [N, T]; 0 for ids outside the vocabulary."""
    V = logp.shape[1]
    got = np.take_along_axis(logp, np.clip(ids, 0, V - 1).astype(np.int64), 1)
    return np.where((ids >= 0) & (ids < V), got, 0.0)


def top(z, logp, k):
    """Ids and log-probabilities of the k largest logits above -inf (equal logits by id), -1 and -inf past them."""
    N, V = z.shape
    ids, lp = np.full((N, k), -1, np.int64), np.full((N, k), -np.inf)
    for n in range(N):
        there = np.flatnonzero(z[n] > -np.inf)
        order = there[np.lexsort((there, -z[n][there]))][:k]
        ids[n, :order.size], lp[n, :order.size] = order, logp[n, order]
    return ids, lp


def weights(ids, dlogp, V, N):
    """[N, V]: the sum of dlogp over the entries with each id."""
    w = np.zeros((N, V))
    if ids is not None:
        for n in range(N):
            for i, v in zip(ids[n], dlogp[n]):
                if 0 <= i < V:
                    w[n, i] += v
    return w


def logits_grad(z, ids, dlogp, dentropy):
    """Gradient of sum dlogp logp + dentropy entropy at z [N, V]; zeros for rows of -inf alone."""
    M, _, H, p, logp = row_stats(z)
    w = weights(ids, dlogp, z.shape[1], z.shape[0])
    u = np.zeros(z.shape[0]) if dentropy is None else dentropy
    l = np.where(p > 0, logp, 0.0)
    G = w - p * (w.sum(1) + u * H)[:, None] - u[:, None] * p * l
    return np.where((M == -np.inf)[:, None], 0.0, G)

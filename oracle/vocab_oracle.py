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


def e4m3_values():
    """The 127 finite non-negative e4m3 values by code: sign, 4 exponent bits
    (bias 7), 3 mantissa bits; code 127 is NaN."""
    c = np.arange(127)
    e, m = c >> 3, c & 7
    return np.where(e == 0, m * 2.0 ** -9, (1 + m / 8) * 2.0 ** (e.astype(np.float64) - 7))


def e4m3_codes(x):
    """Codes of the e4m3 values nearest to x, ties to the even code (|x| <= 464; NaN -> 127)."""
    v = e4m3_values()
    mid = (v[1:] + v[:-1]) / 2
    a = np.abs(np.asarray(x, np.float64))
    c = np.searchsorted(mid, np.where(np.isnan(a), 0, a), side="left")
    tie = (c < 126) & (a == mid[np.minimum(c, 125)]) & (c % 2 == 1)
    c = np.minimum(c + tie, 126)
    c = np.where(np.isnan(a), 127, c)
    return (c | (np.signbit(x) << 7)).astype(np.uint8)


def quantize(x, block_rows):
    """(codes [R, C], scales) of fp32 x: scale = fp32(amax / 448) of the finite values
    of each block_rows x 128 block, code = e4m3 of the fp32 quotient; rows' scales
    are [blocks of columns, R]."""
    x = np.asarray(x, np.float32)
    R, C = x.shape
    rb, kb = -(-R // block_rows), -(-C // 128)
    codes, scales = np.zeros((R, C), np.uint8), np.ones((rb, kb), np.float32)
    for i in range(rb):
        for j in range(kb):
            b = x[i * block_rows:(i + 1) * block_rows, 128 * j:128 * j + 128]
            fin = np.isfinite(b)
            amax = np.max(np.abs(b), where=fin, initial=0.0).astype(np.float32)
            s = np.float32(max(np.float32(amax / np.float32(448)), np.float32(2.0 ** -126))) if amax > 0 else np.float32(1)
            with np.errstate(invalid="ignore"):
                q = np.where(fin, b / s, np.float32("nan")).astype(np.float32)
            codes[i * block_rows:(i + 1) * block_rows, 128 * j:128 * j + 128] = e4m3_codes(q)
            scales[i, j] = s
    return codes, (scales.T.copy() if block_rows == 1 else scales)


def dequantize(codes, scales, block_rows):
    """float64 values of codes and scales as ``quantize`` gives them."""
    v = np.concatenate([e4m3_values(), [np.nan]])
    x = v[codes & 127] * np.where(codes & 128, -1.0, 1.0)
    R, C = x.shape
    s = (scales.T if block_rows == 1 else scales).astype(np.float64)
    return x * np.repeat(np.repeat(s, block_rows, 0)[:R], 128, 1)[:, :C]

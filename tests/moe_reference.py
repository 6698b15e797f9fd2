"""Plain 64-bit implementations of the mixture-of-experts operators, on the CPU, choice by
choice, from their definitions."""
import numpy as np


def sort(ids, experts):
    """offsets, rows, slots of a 2-D array of expert numbers (outside 0..experts - 1: dropped)."""
    T, K = ids.shape
    offsets = np.zeros(experts + 1, np.int64)
    for e in ids.reshape(-1):
        if 0 <= e < experts:
            offsets[e + 1] += 1
    offsets = np.cumsum(offsets)
    nxt = offsets[:-1].copy()
    rows, slots = np.full(T * K, -1, np.int64), np.full((T, K), -1, np.int64)
    for t in range(T):
        for k in range(K):
            e = ids[t, k]
            if 0 <= e < experts:
                slots[t, k] = nxt[e]
                rows[nxt[e]] = t
                nxt[e] += 1
    return offsets, rows, slots


def dispatch(x, slots, nrows):
    """Row -> token's values; rows no choice names are NaN."""
    y = np.full((nrows, x.shape[1]), np.nan)
    for t in range(slots.shape[0]):
        for s in slots[t]:
            if 0 <= s < nrows:
                y[s] = x[t]
    return y


def combine(y, slots, weights):
    """Sums, and the sums of magnitudes that bound their rounding."""
    T, K = slots.shape
    out, size = np.zeros((T, y.shape[1])), np.zeros((T, y.shape[1]))
    for t in range(T):
        for k in range(K):
            s = slots[t, k]
            if 0 <= s < y.shape[0]:
                term = (1.0 if weights is None else float(weights[t, k])) * y[s]
                out[t] += term
                size[t] += np.abs(term)
    return out, size


def combine_backward(dout, y, slots, weights):
    T, K = slots.shape
    dy = np.full(y.shape, np.nan)
    dw, size = np.zeros((T, K)), np.zeros((T, K))
    for t in range(T):
        for k in range(K):
            s = slots[t, k]
            if 0 <= s < y.shape[0]:
                dy[s] = float(weights[t, k]) * dout[t]
                terms = dout[t] * y[s]
                dw[t, k] = terms.sum()
                size[t, k] = np.abs(terms).sum()
    return dy, dw, size


def quantize(x):
    """q (whole numbers) and scale of each row of finite values, or 0 and NaN."""
    peak = np.abs(x).max(axis=1)
    bad = ~np.isfinite(peak)
    safe = np.where((peak == 0) | bad, 1.0, peak)
    q = np.rint(np.where(bad[:, None], 0.0, 127.0 * np.where(np.isfinite(x), x, 0.0)) / safe[:, None])
    return q.astype(np.int64), np.where(bad, np.nan, peak / 127.0)


def product(q, scales, w, w_scales, offsets):
    """Rows outside every expert's range are NaN."""
    out = np.full((q.shape[0], w.shape[1]), np.nan)
    for e in range(w.shape[0]):
        a, b = int(offsets[e]), int(offsets[e + 1])
        if a < b:
            sums = (q[a:b].astype(np.float64) @ w[e].astype(np.float64).T)   # whole numbers below 2^53: exact
            out[a:b] = sums * scales[a:b, None].astype(np.float64) * w_scales[e].astype(np.float64)
    return out

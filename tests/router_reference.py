"""Plain 64-bit implementations of the router's operators and of the product with 4-bit
weights, on the CPU, token by token, from their definitions."""
import numpy as np


def counted(z, mask):
    """Tokens that take part: not masked, some logit above minus infinity."""
    open_ = ~(z == -np.inf).all(axis=1)
    return open_ if mask is None else open_ & (mask != 0)


def softmax(z):
    with np.errstate(invalid="ignore", over="ignore"):
        e = np.exp(z - z.max())
        return e / e.sum()


def choices(z, mask, top_k):
    live = counted(z, mask)
    ids = np.full((z.shape[0], top_k), -1, np.int64)
    for t in np.flatnonzero(live):
        nan = np.isnan(z[t])
        rank = np.where(nan, np.inf, z[t])
        order = sorted(range(z.shape[1]), key=lambda e: (not nan[e], -rank[e], e))
        for k in range(top_k):
            if nan[order[k]] or rank[order[k]] > -np.inf:
                ids[t, k] = order[k]
    return ids


def over_choices(row, ids):
    """Softmax over a token's choices (0 for dropped ones, and where all are closed)."""
    w = np.zeros(len(ids))
    kept = ids >= 0
    if kept.any() and not (row[ids[kept]] == -np.inf).all():
        w[kept] = softmax(row[ids[kept]])
    return w


def weights(z, mask, ids, renormalize):
    live, w = counted(z, mask), np.zeros(ids.shape)
    for t in np.flatnonzero(live):
        kept = ids[t] >= 0
        if renormalize:
            w[t] = over_choices(z[t], ids[t])
        else:
            w[t, kept] = softmax(z[t])[ids[t, kept]]
    return w


def balance(z, mask, ids):
    """counts (and n), sums, loss."""
    live, (T, E), K = counted(z, mask), z.shape, ids.shape[1]
    counts, sums = np.zeros(E + 1, np.int64), np.zeros(E)
    for t in np.flatnonzero(live):
        sums += softmax(z[t])
        for e in ids[t]:
            if 0 <= e < E:
                counts[e] += 1
    n = counts[E] = live.sum()
    return counts, sums, float(E / (K * float(n) ** 2) * (counts[:E] * sums).sum()) if n else 0.0


def backward(z, mask, ids, renormalize, dweights, counts, dloss):
    """dlogits and the sums of magnitudes that bound its rounding."""
    (T, E), K = z.shape, ids.shape[1]
    grad, size = np.zeros((T, E)), np.zeros((T, E))
    for t in np.flatnonzero(counted(z, mask)):
        p = softmax(z[t])
        if counts is not None and counts[E]:
            f = dloss * E / (K * float(counts[E]) ** 2) * counts[:E]
            grad[t] += p * (f - (p * f).sum())
            size[t] += p * (np.abs(f) + (p * np.abs(f)).sum())
        if dweights is None:
            continue
        ok = (ids[t] >= 0) & (ids[t] < E)
        if renormalize:
            w = over_choices(z[t], np.where(ok, ids[t], -1))
            dw = np.where(ok, dweights[t], 0.0)
            for k in np.flatnonzero(ok):
                grad[t, ids[t, k]] += w[k] * (dw[k] - (w * dw).sum())
                size[t, ids[t, k]] += w[k] * (abs(dw[k]) + (w * np.abs(dw)).sum())
        else:
            g, a = np.zeros(E), np.zeros(E)
            for k in np.flatnonzero(ok):
                g[ids[t, k]] += dweights[t, k]
                a[ids[t, k]] += abs(dweights[t, k])
            grad[t] += p * (g - (p * g).sum())
            size[t] += p * (a + (p * a).sum())
    return grad, size


# ------------------------------------------------------------------------------------
# 4-bit weights
# ------------------------------------------------------------------------------------
def unpack4(q, E, N, H):
    """Values (E x N x H) of packed tiles, place by place; and whether all other places are 0."""
    tiles, slabs = -(-N // 16), -(-H // 128)
    words = np.frombuffer(np.ascontiguousarray(q).tobytes(), "<u4").reshape(E, tiles, slabs, 256)
    full = np.zeros((E, tiles * 16, slabs * 128), np.int64)
    for o in range(16):
        for g in range(4):
            for i in range(4):
                for j in range(8):
                    v = (words[:, :, :, 4 * (16 * g + o) + i] >> (4 * j)) & 15
                    full[:, o::16, 32 * i + 8 * g + j::128] = np.where(v > 7, v.astype(np.int64) - 16, v)
    inside = full[:, :N, :H].copy()
    full[:, :N, :H] = 0
    return inside, not full.any()


def quantize4(w, group, round_scale):
    """Values and scales (E x groups x N) of float32 weights; round_scale rounds to the scales' type."""
    E, N, H = w.shape
    groups = -(-H // group)
    values, scales = np.zeros((E, N, H), np.int64), np.zeros((E, groups, N))
    for g in range(groups):
        part = w[:, :, g * group:(g + 1) * group]
        peak = np.abs(part).max(axis=2)
        bad = ~np.isfinite(peak)
        s = round_scale(np.where(bad, 0, peak).astype(np.float32) / np.float32(7))
        safe = np.where(s == 0, np.float32(1), s)[:, :, None]
        q = np.clip(np.rint(np.where(np.isfinite(part), part, 0).astype(np.float32) / safe), -8, 7)
        values[:, :, g * group:(g + 1) * group] = np.where(((s == 0) | bad)[:, :, None], 0, q)
        scales[:, g, :] = np.where(bad, np.nan, s)
    return values, scales


def product4(x, index, values, scales, group, offsets):
    """out, and the sums of magnitudes; rows outside every expert's range are NaN."""
    E, N, H = values.shape
    M = len(index)
    out, size = np.full((M, N), np.nan), np.zeros((M, N))
    for e in range(E):
        w = values[e] * np.repeat(scales[e].T, group, axis=1)[:, :H]
        at = slice(int(offsets[e]), int(offsets[e + 1]))
        there = (index[at] >= 0) & (index[at] < x.shape[0])
        rows = np.where(there[:, None], x[np.where(there, index[at], 0)], 0.0)
        with np.errstate(invalid="ignore"):
            out[at] = rows @ w.T
            size[at] = np.abs(rows) @ np.abs(w).T
    return out, size

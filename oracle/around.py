"""The operators around the products, in fp64 numpy: the router and its
gradient, the row layouts, the quantising scatter, the weighted gather and its
weights' gradient, and low-rank adapters.  Definitions as in include/dg.h."""
import numpy as np

E4M3_MAX = 448.0
LEAST_AMAX = 2.0 ** -100


# ---- router ------------------------------------------------------------------
def _scores(x, score):
    x = np.where(np.isnan(x), -np.inf, np.minimum(np.asarray(x, dtype=np.float64), np.finfo(np.float32).max))
    with np.errstate(over="ignore", invalid="ignore", divide="ignore"):
        if score == "sigmoid":
            return x, 1.0 / (1.0 + np.exp(-x))
        top = x.max(axis=1, keepdims=True)
        e = np.where(x > -np.inf, np.exp(x - np.where(top > -np.inf, top, 0.0)), 0.0)
        z = e.sum(axis=1, keepdims=True)
        return x, np.divide(e, z, out=np.zeros_like(e), where=z > 0)


def route(x, bias, top_k, score, num_groups=1, topk_groups=1, group_top=1, renormalize=True, scale=1.0):
    """(ids [T][top_k], weights, margin [T]): margin is the least gap between two neighbours of a
    sorted list whose order shows in the answer (inf where nothing was near)."""
    x, s = _scores(x, score)
    T, E = x.shape
    with np.errstate(invalid="ignore"):
        key = s if bias is None else s + np.asarray(bias, dtype=np.float64)
    key = np.where((x > -np.inf) & (key > -np.inf), key, -np.inf)
    ids = np.full((T, top_k), -1, dtype=np.int64)
    weights = np.zeros((T, top_k))
    margin = np.full(T, np.inf)

    def order(v):                        # falling, lowest index first among equals
        o = np.lexsort((np.arange(v.size), -v))
        return [i for i in o if v[i] > -np.inf]

    def gap(t, v, o, n):
        for i in range(min(n, len(o) - 1)):
            margin[t] = min(margin[t], v[o[i]] - v[o[i + 1]])

    for t in range(T):
        k = key[t].copy()
        if topk_groups < num_groups:
            per = k.reshape(num_groups, -1)
            best = -np.sort(-per, axis=1)[:, :group_top]
            g = np.where(best[:, 0] > -np.inf, np.where(best > -np.inf, best, 0.0).sum(axis=1), -np.inf)
            o = order(g)
            gap(t, g, o, topk_groups)
            keep = np.zeros(num_groups, dtype=bool)
            keep[o[:topk_groups]] = True
            k[np.repeat(~keep, E // num_groups)] = -np.inf
        o = order(k)
        gap(t, k, o, top_k)
        o = o[:top_k]
        ids[t, :len(o)] = o
        w = s[t, o]
        if renormalize:
            w = w / w.sum() if w.sum() > 0 else np.zeros_like(w)
        weights[t, :len(o)] = scale * w
    return ids, weights, margin


def route_weights(x, ids, score, renormalize, scale):
    """The weights of a given choice, for differences: x fp64 [T][E]."""
    x, s = _scores(x, score)
    has = (ids >= 0) & (ids < x.shape[1])
    w = np.where(has, np.take_along_axis(s, np.where(has, ids, 0), axis=1), 0.0)
    if renormalize:
        z = w.sum(axis=1, keepdims=True)
        w = np.divide(w, z, out=np.zeros_like(w), where=z > 0)
    return scale * w


def route_backward(x, ids, grad_weights, score, renormalize, scale):
    x, s = _scores(x, score)
    T, E = x.shape
    has = (ids >= 0) & (ids < E)
    at = np.where(has, ids, 0)
    chosen = np.where(has, np.take_along_axis(s, at, axis=1), 0.0)
    g = np.where(chosen > 0, np.asarray(grad_weights, dtype=np.float64), 0.0) * scale
    z = chosen.sum(axis=1, keepdims=True)
    z = np.where(z > 0, z, 1.0)
    ds = np.zeros((T, E))                # gradient with respect to the scores
    for j in range(ids.shape[1]):
        gj = g[:, j:j + 1]
        d = (gj - (g * chosen).sum(axis=1, keepdims=True) / z) / z if renormalize else gj
        for t in np.nonzero(has[:, j])[0]:
            ds[t, ids[t, j]] += d[t, 0]
    if score == "sigmoid":
        return ds * s * (1.0 - s)
    return s * (ds - (ds * s).sum(axis=1, keepdims=True))


# ---- rows --------------------------------------------------------------------
def rows_bound(choices, groups):
    return (choices + 127 * min(choices, groups)) // 128 * 128


def layout_contiguous(ids, first, groups, M):
    """(grouped_layout, row_of, slot_of, counts)"""
    flat = np.asarray(ids, dtype=np.int64).ravel() - first
    counts = np.array([(flat == g).sum() for g in range(groups)], dtype=np.int64)
    start = np.concatenate([[0], np.cumsum((counts + 127) // 128 * 128)])
    layout, slot = np.full(M, -1, dtype=np.int32), np.full(M, -1, dtype=np.int32)
    row = np.full(flat.size, -1, dtype=np.int32)
    seen = np.zeros(groups, dtype=np.int64)
    for i, g in enumerate(flat):
        if 0 <= g < groups:
            r = start[g] + seen[g]
            seen[g] += 1
            if r < M:
                row[i], slot[r], layout[r] = r, i, g
    return layout, row.reshape(np.shape(ids)), slot, counts.astype(np.int32)


def layout_masked(ids, first, groups, max_m):
    """(masked_m, row_of, slot_of)"""
    flat = np.asarray(ids, dtype=np.int64).ravel() - first
    slot = np.full((groups, max_m), -1, dtype=np.int32)
    row = np.full(flat.size, -1, dtype=np.int32)
    seen = np.zeros(groups, dtype=np.int64)
    for i, g in enumerate(flat):
        if 0 <= g < groups:
            if seen[g] < max_m:
                row[i], slot[g, seen[g]] = g * max_m + seen[g], i
            seen[g] += 1
    return np.minimum(seen, max_m).astype(np.int32), row.reshape(np.shape(ids)), slot


def block_scales(amax, pow2):
    """fp64 scales of block maxima (finite)."""
    sf = np.maximum(amax, LEAST_AMAX) / E4M3_MAX
    if pow2:
        m, e = np.frexp(sf)
        sf = np.ldexp(1.0, np.where(m == 0.5, e - 1, e))
    return np.where(amax > 0, sf, 1.0)


def e4m3_step(v):
    """The distance between neighbouring e4m3 values at |v| (2^-9 below 2^-6)."""
    v = np.minimum(np.abs(v), E4M3_MAX)
    e = np.where(v > 0, np.frexp(v)[1], -5)
    return np.ldexp(1.0, np.maximum(e, -5) - 4)


def gather(rows, row_of, weights, c):
    """(sum, sum of magnitudes) in fp64."""
    T, k = row_of.shape
    out = np.zeros((T, rows.shape[1])) if c is None else c.astype(np.float64)
    mag = np.abs(out)
    for j in range(k):
        ok = (row_of[:, j] >= 0) & (row_of[:, j] < rows.shape[0])
        v = rows[row_of[ok, j]].astype(np.float64)
        if weights is not None:
            v = v * weights[ok, j].astype(np.float64)[:, None]
        out[ok] += v
        mag[ok] += np.abs(v)
    return out, mag


def gather_weight_grad(rows, row_of, grad_d):
    T, k = row_of.shape
    out, mag = np.zeros((T, k)), np.zeros((T, k))
    for j in range(k):
        ok = (row_of[:, j] >= 0) & (row_of[:, j] < rows.shape[0])
        v = rows[row_of[ok, j]].astype(np.float64) * grad_d[ok].astype(np.float64)
        out[ok, j] = v.sum(axis=1)
        mag[ok, j] = np.abs(v).sum(axis=1)
    return out, mag


# ---- adapters ----------------------------------------------------------------
def lora(x, a, b, scales, ids, c):
    """(result, |adapter term| with every product's magnitude) in fp64."""
    T, N = x.shape[0], b.shape[1]
    out = np.zeros((T, N)) if c is None else c.astype(np.float64)
    mag = np.zeros((T, N))
    for t in range(T):
        i = ids[t]
        if 0 <= i < a.shape[0]:
            s = 1.0 if scales is None else float(scales[i])
            A, B, v = a[i].astype(np.float64), b[i].astype(np.float64), x[t].astype(np.float64)
            out[t] += s * (B @ (A @ v))
            mag[t] = abs(s) * (np.abs(B) @ (np.abs(A) @ np.abs(v)))
    return out, mag

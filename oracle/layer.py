"""The router's balance loss and its gradient, products with 4-bit weights, and
the gradients' norm and clipping, in fp64 numpy.  Definitions as in
include/dg.h."""
import numpy as np


# ---- balance loss --------------------------------------------------------------
def _spans(seq_starts, T):
    if seq_starts is None:
        return [(0, T)]
    s = np.clip(np.asarray(seq_starts, dtype=np.int64), 0, T)
    return list(zip(s[:-1], s[1:]))


def shares(x, score):
    """(p [T][E], sigmoid(-x)): 0 in p for masked experts (NaN or -inf)."""
    x = np.where(np.isnan(x), -np.inf, np.minimum(np.asarray(x, dtype=np.float64), np.finfo(np.float32).max))
    with np.errstate(over="ignore", invalid="ignore", divide="ignore"):
        logs = x if score == "softmax" else -np.logaddexp(0.0, -x)
        logs = np.where(x > -np.inf, logs, -np.inf)
        top = logs.max(axis=1, keepdims=True)
        e = np.where(x > -np.inf, np.exp(logs - np.where(top > -np.inf, top, 0.0)), 0.0)
        z = e.sum(axis=1, keepdims=True)
        rest = np.exp(-np.logaddexp(0.0, x))
    return np.divide(e, z, out=np.zeros_like(e), where=z > 0), rest


def balance(x, ids, seq_starts, score, scale=1.0):
    """(loss [S], counts [S][E])"""
    T, E = x.shape
    k = ids.shape[1]
    p, _ = shares(x, score)
    losses, counts = [], []
    for a, b in _spans(seq_starts, T):
        chosen = ids[a:b].ravel()
        n = np.bincount(chosen[(chosen >= 0) & (chosen < E)], minlength=E)
        counts.append(n)
        losses.append(scale * E / (k * float(b - a) ** 2) * float(n @ p[a:b].sum(axis=0)) if b > a else 0.0)
    return np.array(losses), np.array(counts).reshape(-1, E)


def balance_backward(x, counts, seq_starts, grad_loss, c, top_k, score, scale=1.0):
    """(gradient [T][E] with c added, the magnitudes that its rounding is measured by)"""
    T, E = x.shape
    p, rest = shares(x, score)
    if score == "softmax":
        rest = np.ones_like(rest)
    out = np.zeros((T, E)) if c is None else np.array(c, dtype=np.float64)
    mag = np.zeros((T, E))
    for s, (a, b) in enumerate(_spans(seq_starts, T)):
        if b <= a:
            continue
        w = scale * E / (top_k * float(b - a) ** 2) * (1.0 if grad_loss is None else float(grad_loss[s]))
        for t in range(a, b):
            n = counts[s].astype(np.float64)
            n = n - n[np.argmax(p[t])]
            with np.errstate(invalid="ignore"):
                g = w * p[t] * rest[t] * (n - p[t] @ n)
                m = abs(w) * p[t] * rest[t] * (np.abs(n) + p[t] @ np.abs(n))
            out[t] += np.where(p[t] > 0, g, 0.0)
            mag[t] = np.where(p[t] > 0, m, 0.0)
    return out, mag


# ---- 4-bit weights --------------------------------------------------------------
E2M1 = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6, -0.0, -0.5, -1, -1.5, -2, -3, -4, -6])


def nibbles(b):
    """[..., K/2] bytes -> [..., K] values of 0 to 15, the low nibble first"""
    b = np.asarray(b, dtype=np.uint8)
    return np.stack([b & 15, b >> 4], axis=-1).reshape(*b.shape[:-1], -1)


def fp4_weights(b, sfb):
    """[N][K] of b uint8 [N][K/2] and sfb int32 [K/128][N] (four E8M0 exponents each)"""
    w = E2M1[nibbles(b)]
    e = np.ascontiguousarray(sfb).view(np.uint8).reshape(*sfb.shape, 4).astype(np.float64)
    e = np.moveaxis(e, 1, 0).reshape(w.shape[0], -1)                # [N][K/32]
    power = np.where(e == 255, np.nan, 2.0 ** (e - 127))
    return w * np.repeat(power, 32, axis=1)


def int4_weights(b, scales, zeros):
    """([N][K], the same with q + zero in place of q - zero: what its sums' rounding is measured by)"""
    q = nibbles(b).astype(np.float64)
    group = q.shape[1] // scales.shape[0]
    z = np.full(scales.shape, 8.0) if zeros is None else np.asarray(zeros, dtype=np.float64)
    z = np.repeat(z.T, group, axis=1)
    s = np.repeat(np.asarray(scales, dtype=np.float64).T, group, axis=1)
    return (q - z) * s, (q + z) * np.abs(s)


def gemv(x, w, c, most=None):
    """(c + x w^T, sum of magnitudes); most: magnitudes in place of |w|"""
    x = np.asarray(x, dtype=np.float64)
    d = x @ w.T
    mag = np.abs(x) @ (np.abs(w) if most is None else most).T
    return (d, mag) if c is None else (d + np.asarray(c, dtype=np.float64), mag + np.abs(np.asarray(c, dtype=np.float64)))


# ---- gradients -------------------------------------------------------------------
def grad_norm(grads):
    return float(np.sqrt(sum(float(np.sum(np.asarray(g, dtype=np.float64) ** 2)) for g in grads)))


def grad_factor(norm, max_norm):
    return min(1.0, max_norm / (norm + 1e-6))

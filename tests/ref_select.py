"""64-bit references of the expert choice and of the 4-bit experts (numpy; not
collected as tests): plain loops and sums from the definitions.

Rounding units: U = 2^-24 is half an ulp of fp32 relative to the value, 2 U
what a truncating fp32 accumulation loses per addition.
"""
from __future__ import annotations

import numpy as np

U = 2.0 ** -24


def half_ulp_bf16(x):
    """Half the spacing of bf16 (8 significant bits) at |x|."""
    x = np.maximum(np.abs(x), 2.0 ** -126)
    return np.exp2(np.floor(np.log2(x)) - 8.0)


def scores(z, score):
    z = np.asarray(z, np.float64)
    with np.errstate(over="ignore", invalid="ignore"):
        if score == "sigmoid":
            return 1.0 / (1.0 + np.exp(-z))
        m = z.max(axis=1, keepdims=True)
        m = np.where(np.isneginf(m), 0.0, m)
        e = np.where(np.isneginf(z), 0.0, np.exp(z - m))
        tot = e.sum(axis=1, keepdims=True)
        return np.where(tot > 0, e / np.where(tot > 0, tot, 1.0), 0.0)


def weights_of(z, ids, score, renorm, scale):
    """w [T, k] of a given choice."""
    s = scores(z, score)
    p = np.take_along_axis(s, ids, 1)
    if renorm:
        tot = p.sum(1, keepdims=True)
        p = np.where(tot > 0, p / np.where(tot > 0, tot, 1.0), 0.0)
    return scale * p


def select(z, k, bias=None, score="softmax", n_groups=1, top_groups=1, group_score="top2", renorm=True, scale=1.0):
    """dict ids, w, gap: gap[t] is the smallest distance between two values
    that the choice compares with different outcomes for the result."""
    z = np.asarray(z, np.float64)
    T, E = z.shape
    per = E // n_groups
    s = scores(z, score)
    by_score = bias is not None or (group_score == "top2" and n_groups > 1 and per > 1)
    a = s + (0.0 if bias is None else np.asarray(bias, np.float64)) if by_score else z
    a = np.where(np.isneginf(z), -np.inf, a)
    ids = np.zeros((T, k), np.int64)
    gap = np.full(T, np.inf)
    for t in range(T):
        order_g = [0]
        if n_groups > 1:
            best = []
            for g in range(n_groups):
                v = sorted(a[t, g * per:(g + 1) * per], reverse=True)
                if group_score == "top2" and per > 1 and v[1] > -np.inf:
                    best.append(v[0] + v[1])
                else:
                    best.append(v[0])
            rank = sorted(range(n_groups), key=lambda g: (-best[g], g))
            order_g = sorted(rank[:top_groups])
            if top_groups < n_groups and best[rank[top_groups]] > -np.inf:
                gap[t] = abs(best[rank[top_groups - 1]] - best[rank[top_groups]])
        cand = [e for g in order_g for e in range(g * per, (g + 1) * per)]
        cand.sort(key=lambda e: (-a[t, e], e))
        ids[t] = cand[:k]
        for x, y in zip(cand[:k], cand[1:k + 1]):
            if a[t, y] > -np.inf:
                gap[t] = min(gap[t], abs(a[t, x] - a[t, y]))
    return dict(ids=ids, w=weights_of(z, ids, score, renorm, scale), gap=gap, a=a)


def select_bwd(dw, z, ids, score, renorm, scale):
    """d_logits [T, E] by the chain rule through the Jacobians, one factor at a time."""
    z, dw = np.asarray(z, np.float64), np.asarray(dw, np.float64)
    T, E = z.shape
    s = scores(z, score)
    out = np.zeros((T, E))
    for t in range(T):
        p = s[t, ids[t]]
        dp = scale * dw[t]
        if renorm:
            tot = p.sum()
            dp = (dp - (dp * p).sum() / tot) / tot if tot > 0 else np.zeros_like(dp)
        ds = np.zeros(E)
        ds[ids[t]] = dp
        if score == "sigmoid":
            out[t] = ds * s[t] * (1.0 - s[t])
        else:
            out[t] = s[t] * (ds - (ds * s[t]).sum())
    return out


def unpack(q, scales, zeros, K, N, group):
    """[E, K, N] fp64 weights from words [E*K/8, N] (int32 or uint32)."""
    q = np.ascontiguousarray(q).view(np.uint32)
    codes = np.stack([(q >> np.uint32(4 * i)) & np.uint32(15) for i in range(8)], 1).reshape(-1, N).astype(np.float64)
    zero = 8.0 if zeros is None else np.repeat(np.asarray(zeros, np.float64), group, 0)
    w = (codes - zero) * np.repeat(np.asarray(scales, np.float64), group, 0)
    return w.reshape(-1, K, N)


def silu(g):
    return g / (1.0 + np.exp(-g))


def experts(rows, ids, W):
    """rows [T, k, K] through W[ids]: (sum, sum of |terms|) [T, k, N]; empty slots 0."""
    T, k, _ = rows.shape
    N = W.shape[2]
    y, mag = np.zeros((T, k, N)), np.zeros((T, k, N))
    for t in range(T):
        for j in range(k):
            e = ids[t, j]
            if e >= 0:
                y[t, j] = rows[t, j] @ W[e]
                mag[t, j] = np.abs(rows[t, j]) @ np.abs(W[e])
    return y, mag

"""The operators on 8-bit codes with a scale for each token and channel in plain
numpy, fp64: selection of experts from scores, grouping of the routed pairs,
codes of rows, grouped products, the weighted sum of the pairs.
"""
from __future__ import annotations

import numpy as np

TINY = 2.0 ** -100


def group_scores(v, groups, top2):
    """Scores of the groups of v [T, E] (-inf: expert takes no part): the best, or the sum of the two best."""
    t, e = v.shape
    s = -np.sort(-v.reshape(t, groups, e // groups), axis=-1)
    if not top2 or s.shape[-1] == 1:
        return s[..., 0]
    second = np.where(np.isneginf(s[..., 1]), 0.0, s[..., 1])
    return s[..., 0] + second


def scores(logits, softmax):
    l = np.asarray(logits, np.float64)
    with np.errstate(over="ignore", invalid="ignore"):
        if not softmax:
            return np.where(l >= 0, 1.0 / (1.0 + np.exp(-np.abs(l))), np.exp(-np.abs(l)) / (1.0 + np.exp(-np.abs(l))))
        m = l.max(-1, keepdims=True)
        x = np.exp(l - np.where(np.isneginf(m), 0.0, m))
        total = x.sum(-1, keepdims=True)
        return np.where(total > 0, x / np.where(total > 0, total, 1.0), 0.0)


def select(logits, k, bias=None, softmax=True, groups=1, keep=1, top2=True, renorm=True, scaling=1.0):
    """-> ids [T, k] (-1 where no expert takes part), weights [T, k], and bad [T] (non-finite input)."""
    l = np.asarray(logits, np.float64)
    t, e = l.shape
    b = np.zeros(e) if bias is None else np.asarray(bias, np.float64)
    bad = ~(l < np.inf).all(-1) | ~(b < np.inf).all()
    ids, w = np.full((t, k), -1, np.int64), np.zeros((t, k))
    s = scores(np.where(bad[:, None], 0.0, l), softmax)
    for i in range(t):
        if bad[i]:
            continue
        v = np.where(np.isneginf(l[i]), -np.inf, s[i] + b)
        rank = (l[i] if bias is None else v).copy()
        if keep < groups:
            g = group_scores(v[None], groups, top2)[0]
            kept = sorted(range(groups), key=lambda j: (-g[j], j))[:keep]
            rank[[x for x in range(e) if x // (e // groups) not in kept]] = -np.inf
        order = [x for x in sorted(range(e), key=lambda x: (-rank[x], x)) if rank[x] > -np.inf][:k]
        ids[i, :len(order)] = order
        w[i, :len(order)] = s[i, order]
    if renorm:
        total = w.sum(-1, keepdims=True)
        w = np.where(total > 0, w / np.where(total > 0, total, 1.0), 0.0)
    return ids, w * scaling, bad


def group(idx, experts, rank=0, shards=1):
    """-> offsets [groups + 1], rows [pairs], slots like idx: the pairs of idx [T, k] in expert order."""
    t, k = idx.shape
    mine = range(rank, experts, shards)
    pairs = [(g, i) for g, e in enumerate(mine) for i in np.flatnonzero(idx.reshape(-1) == e)]
    offsets = np.zeros(len(mine) + 1, np.int64)
    slots = np.full(t * k, -1, np.int64)
    for p, (g, i) in enumerate(pairs):
        offsets[g + 1] += 1
        slots[i] = p
    return np.cumsum(offsets), np.array([i // k for _, i in pairs], np.int64), slots.reshape(t, k)


def swiglu(x):
    g, u = np.split(np.asarray(x, np.float64), 2, axis=-1)
    return scores(g, False) * g * u


def quantize(x):
    """-> codes [T, K] (whole numbers), scales [T]; x in fp64, the scale unrounded."""
    x = np.asarray(x, np.float64)
    top = np.abs(x).max(-1)
    lost = ~np.isfinite(top)
    some = (top >= TINY) & ~lost
    q = np.where(some[:, None], np.rint(np.where(some[:, None], x, 0.0) * 127.0 / np.where(some, top, 1.0)[:, None]), 0.0)
    return q, np.where(lost, np.nan, np.where(some, top / 127.0, 0.0))


def sums(x, w, offsets, rows):
    """The exact integer sums [P, N] of codes x [X, K], w [G, N, K]; rows of no group (or out of range) are 0."""
    x, w = np.asarray(x, np.int64), np.asarray(w, np.int64)
    out = np.zeros((len(rows), w.shape[1]), np.int64)
    top = 0
    for g in range(w.shape[0]):
        a = top = max(top, min(max(offsets[g], 0), len(rows)))
        for p in range(a, max(a, min(max(offsets[g + 1], 0), len(rows)))):
            if 0 <= rows[p] < len(x):
                out[p] = w[g] @ x[rows[p]]
    return out


def combine(o, slots, w, add=None):
    """-> y [T, H] and the sum of magnitudes behind each value."""
    y = np.zeros((len(slots), o.shape[1])) if add is None else np.array(add, np.float64)
    mag = np.abs(y)
    for t, j in np.ndindex(*slots.shape):
        if 0 <= slots[t, j] < len(o):
            term = np.float64(w[t, j]) * np.asarray(o[slots[t, j]], np.float64)
            y[t] += term
            mag[t] += np.abs(term)
    return y, mag

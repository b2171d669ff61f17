"""64-bit definitions of the 16-bit block around the experts: router, grouping, grouped products,
norms.  Plain numpy, one token / expert / row at a time where that is the definition."""
from __future__ import annotations

import numpy as np


def sigmoid(x):
    x = np.asarray(x, np.float64)
    with np.errstate(over="ignore"):
        return 1.0 / (1.0 + np.exp(-x))


# ------------------------------------------------------------------------------------ router

def choose(keys, topk):
    """Indices of the topk largest keys (descending, equal keys in ascending index); -inf and NaN
    are never chosen (id -1)."""
    keys = np.asarray(keys)
    left = [(-(k + 0.0), i) for i, k in enumerate(keys) if k > -np.inf]
    left.sort()
    ids = [i for _, i in left[:topk]]
    return ids + [-1] * (topk - len(ids))


def router(logits, topk, score="softmax", bias=None, n_group=1, topk_group=1, renormalize=True,
           scale=1.0, keys=None):
    """(ids [M, topk] int32, weights [M, topk] float64).  keys: the selection keys to use instead
    of the 64-bit ones (a sigmoid's 32-bit keys can tie or swap where 64-bit ones do not)."""
    l = np.asarray(logits, np.float64)
    M, E = l.shape
    ids = np.full((M, topk), -1, np.int32)
    w = np.zeros((M, topk))
    for t in range(M):
        live = l[t] > -np.inf                                  # False for NaN too
        if score == "sigmoid":
            # a score is an fp32 value: one below its range is 0
            s = np.where(live, sigmoid(np.where(live, l[t], 0.0)), 0.0).astype(np.float32).astype(np.float64)
            k = s + (0.0 if bias is None else np.asarray(bias, np.float64))
        else:
            s = np.zeros(E)
            if live.any():
                top = l[t][live].max()
                d = np.where(live & (l[t] != top), l[t] - top if np.isfinite(top) else -np.inf, 0.0)
                s = np.where(live, np.exp(d), 0.0)
                s /= s.sum()
            k = l[t]
        if keys is not None:
            k = np.asarray(keys[t])
        k = np.where(live & ~np.isnan(k), k, -np.inf)
        if n_group > 1:
            runs = k.reshape(n_group, E // n_group)
            best = -np.sort(-runs, axis=1)
            rk = best[:, 0] if score == "softmax" or runs.shape[1] == 1 else best[:, 0] + best[:, 1]
            order = sorted(range(n_group), key=lambda g: (-rk[g], g))
            stay = np.zeros(n_group, bool)
            stay[order[:topk_group]] = True
            k = np.where(np.repeat(stay, E // n_group), k, -np.inf)
        ids[t] = choose(k, topk)
        got = ids[t] >= 0
        w[t, got] = s[ids[t][got]]
        if renormalize:
            total = w[t].sum()
            w[t] = w[t] / total if total > 0 else 0.0
    return ids, w * scale


# ------------------------------------------------------------------------------------ grouping

def group(ids, E, first=0):
    """(offsets [E + 1], perm [S], slot_of like ids)."""
    flat = np.asarray(ids, np.int64).reshape(-1) - first
    lists = [[] for _ in range(E)]
    for f, e in enumerate(flat):
        if 0 <= e < E:
            lists[e].append(f)
    order = [f for l in lists for f in l]
    offsets = np.concatenate([[0], np.cumsum([len(l) for l in lists])]).astype(np.int32)
    perm = np.full(flat.size, -1, np.int32)
    perm[:len(order)] = order
    slot_of = np.full(flat.size, -1, np.int32)
    slot_of[order] = np.arange(len(order))
    return offsets, perm, slot_of.reshape(np.shape(ids))


# ------------------------------------------------------------------------------------ products

def grouped(x, w, offsets, S, perm=None, topk=1):
    """(product [S, N], sum of |terms| [S, N]) in 64 bits; rows past offsets[E] are zero."""
    x, w = np.asarray(x, np.float64), np.asarray(w, np.float64)
    out = np.zeros((S, w.shape[1]))
    mag = np.zeros_like(out)
    for e in range(w.shape[0]):
        a, b = int(offsets[e]), int(offsets[e + 1])
        rows = x[a:b] if perm is None else x[np.asarray(perm[a:b]) // topk]
        out[a:b] = rows @ w[e].T
        mag[a:b] = np.abs(rows) @ np.abs(w[e]).T
    return out, mag


def swiglu(up, gate, limit=np.inf, alpha=1.0, beta=0.0):
    g = np.minimum(gate, limit)
    u = np.clip(up, -limit, limit)
    return g * sigmoid(alpha * g) * (u + beta)


# ------------------------------------------------------------------------------------ norms

def norm(v, weight, bias=None, kind="rms", eps=1e-6, offset=0.0):
    if kind == "layer":
        v = v - v.mean(axis=-1, keepdims=True)
    n = v / np.sqrt(np.mean(v * v, axis=-1, keepdims=True) + eps)
    n = n * (np.asarray(weight, np.float64) + offset)
    return n if bias is None else n + np.asarray(bias, np.float64)


def combine(rows, slot_of, weights, shared=None):
    """(combination [M, H], sum of |terms|)."""
    rows = np.asarray(rows, np.float64)
    M, k = slot_of.shape
    y = np.zeros((M, rows.shape[1]))
    mag = np.zeros_like(y)
    for t in range(M):
        for j in range(k):
            s = slot_of[t, j]
            if 0 <= s < rows.shape[0]:
                y[t] += float(weights[t, j]) * rows[s]
                mag[t] += np.abs(float(weights[t, j]) * rows[s])
    if shared is not None:
        y, mag = y + shared, mag + np.abs(shared)
    return y, mag

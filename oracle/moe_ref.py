"""Plain CPU oracle of a block of experts: the router, pairs sorted by expert, rows there and back,
the packed product with its epilogue, and their gradients.  Test infrastructure only; everything in
64 bits, one loop for one definition.
"""

from __future__ import annotations

import math

import numpy as np

from . import awq_ref


def scores(logits, score, bias=None):
    """What the choice goes by, [T, E]: without a bias a sigmoid orders as its logit."""
    s = np.asarray(logits, dtype=np.float64)
    if bias is not None:
        if score == "sigmoid":
            s = 1 / (1 + np.exp(-s))
        s = s + np.asarray(bias, dtype=np.float64)
    return s


def choose(logits, k, score="softmax", bias=None):
    """[T, k] experts: the largest score, the lowest number of equals, NaN after all others."""
    s = scores(logits, score, bias)
    out = np.empty((s.shape[0], k), dtype=np.int64)
    for t, row in enumerate(s):
        left = list(range(len(row)))
        for j in range(k):
            best = left[0]
            for e in left[1:]:
                if row[e] > row[best] or (np.isnan(row[best]) and not np.isnan(row[e])):
                    best = e
            out[t, j] = best
            left.remove(best)
    return out


def route_weights(logits, experts, score="softmax", normalise=True, scale=1.0):
    x = np.asarray(logits, dtype=np.float64)
    w = np.zeros(experts.shape)
    for t in range(x.shape[0]):
        c = x[t, experts[t]]
        if score == "sigmoid":
            p = 1 / (1 + np.exp(-c))
            total = p.sum() if normalise else 1.0
        else:
            among = c if normalise else x[t]
            top = among.max()
            if top == -np.inf:
                continue
            p, total = np.exp(c - top), np.exp(among - top).sum()
        w[t] = scale * p / total if total != 0 else 0.0
    return w


def route_grad(logits, experts, dweights, score="softmax", normalise=True, scale=1.0):
    x = np.asarray(logits, dtype=np.float64)
    d = np.zeros_like(x)
    for t in range(x.shape[0]):
        e, g = experts[t], scale * np.asarray(dweights[t], dtype=np.float64)
        if score == "sigmoid":
            p = 1 / (1 + np.exp(-x[t]))
            inner = p * (1 - p)
            if normalise:
                total = p[e].sum()
                g = (g - (g * p[e]).sum() / total) / total
            for j in range(len(e)):
                d[t, e[j]] += g[j] * inner[e[j]]
        else:
            among = e if normalise else np.arange(x.shape[1])
            p = np.zeros(x.shape[1])
            p[among] = np.exp(x[t, among] - x[t, among].max())
            p /= p.sum()
            dot = sum(g[j] * p[e[j]] for j in range(len(e)))
            for j in range(len(e)):
                d[t, e[j]] += g[j] * p[e[j]]
            d[t] -= p * dot
    return d


def sort_pairs(experts, first, count):
    """offsets [count + 1], order [n], place of experts' shape."""
    flat = np.asarray(experts, dtype=np.int64).ravel()
    rows = [[] for _ in range(count + 1)]
    for p, e in enumerate(flat):
        rows[e - first if 0 <= e - first < count else count].append(p)
    order = np.array([p for r in rows for p in r], dtype=np.int64)
    place = np.empty_like(order)
    place[order] = np.arange(len(order))
    offsets = np.cumsum([0] + [len(r) for r in rows[:count]])
    return offsets, order, place.reshape(np.shape(experts))


def gather(x, offsets, place, weights=None):
    T, k = place.shape
    out = np.zeros((T * k, x.shape[1]))
    for t in range(T):
        for j in range(k):
            if place[t, j] < offsets[-1]:
                out[place[t, j]] = x[t] * (1.0 if weights is None else weights[t, j])
    return out


def combine(rows, offsets, place, weights=None, residual=None):
    T, k = place.shape
    out = np.zeros((T, rows.shape[1])) if residual is None else residual.astype(np.float64)
    for t in range(T):
        for j in range(k):
            if place[t, j] < offsets[-1]:
                out[t] += rows[place[t, j]] * (1.0 if weights is None else weights[t, j])
    return out


def dots(tokens, rows, offsets, place):
    """<tokens[t], rows[place[t, j]]>, 0 for pairs that no expert has: what weights' gradients are."""
    T, k = place.shape
    out = np.zeros((T, k))
    for t in range(T):
        for j in range(k):
            if place[t, j] < offsets[-1]:
                out[t, j] = tokens[t] @ rows[place[t, j]]
    return out


def activate(v, act):
    if act == "relu":
        return np.maximum(v, 0)
    if act == "silu":
        return v / (1 + np.exp(-v))
    if act == "gelu":
        return 0.5 * v * (1 + np.vectorize(math.erf)(v / math.sqrt(2)))
    if act == "gelu_tanh":
        return 0.5 * v * (1 + np.tanh(math.sqrt(2 / math.pi) * (v + 0.044715 * v ** 3)))
    return v


def finish(v, act="none", gated=False, residual=None):
    if gated:
        half = v.shape[1] // 2
        y = activate(v[:, :half], act) * v[:, half:]
    else:
        y = activate(v, act)
    return y if residual is None else y + residual


def weights_of(codes, steps, zeros, group):
    """(c - z) step, [rows, K], from codes [rows, K] and [rows, K/group] of steps and zero points."""
    z = np.repeat(np.asarray(zeros, dtype=np.float64), group, 1)
    return (np.asarray(codes, dtype=np.float64) - z) * np.repeat(np.asarray(steps, dtype=np.float64), group, 1)


def repack(codes, steps, zeros, bits):
    """The layout that the products read: words [K/32, rows, bits] and (step, zero) [K/group, rows, 2]."""
    rows, K = codes.shape
    words = awq_ref.pack_codes(codes, bits).reshape(rows, K // 32, bits).transpose(1, 0, 2)
    meta = np.stack((np.asarray(steps, np.float32), np.asarray(zeros, np.float32)), -1).transpose(1, 0, 2)
    return np.ascontiguousarray(words), np.ascontiguousarray(meta)


def experts_product(x, W, offsets, source=None):
    """Rows [offsets[e], offsets[e+1]) times W[e]^T; row r is x[source[r]] (None: x[r]); the rest zero."""
    n = len(x) if source is None else len(source)
    v = np.zeros((n, W.shape[1]))
    for e in range(W.shape[0]):
        for r in range(offsets[e], offsets[e + 1]):
            v[r] = W[e] @ x[r if source is None else source[r]]
    return v

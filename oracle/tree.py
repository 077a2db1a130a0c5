"""A step of speculative decoding over the paged cache, in float64: appending normed and rotated rows,
attention of drafted trees, sampling, and the trees' bookkeeping.

TEST INFRASTRUCTURE (see oracle/__init__.py): never imported by the product path.
"""
from __future__ import annotations

import numpy as np


def append_rows(x, gain, pos, kind, theta, base, exp, eps, query):
    """Rows x [T, heads, D] normed by gain [D] (None: not) and rotated ("rope") or, queries only, scaled ("ssmax")."""
    x = np.asarray(x, np.float64)
    D = x.shape[-1]
    p = np.asarray(pos, np.float64)[:, None, None]
    if gain is not None:
        x = x / np.sqrt(np.mean(x * x, -1, keepdims=True) + eps) * gain
    if kind == "rope":
        angle = (p - 1) * theta ** (-2.0 * np.arange(D // 2) / D)
        a, b = x[..., :D // 2], x[..., D // 2:]
        return np.concatenate([a * np.cos(angle) - b * np.sin(angle), b * np.cos(angle) + a * np.sin(angle)], -1)
    return x * (1 + np.maximum(p, 0) / base) ** exp if query else x


def masks(parent):
    """Each node's ancestors and itself, as sets, for one tree; None where a parent is not an earlier node."""
    out = []
    for j, up in enumerate(parent):
        if up < -1 or up >= j or (up >= 0 and out[up] is None):
            out.append(None)
        else:
            out.append((out[up] if up >= 0 else frozenset()) | {j})
    return out


def bits(nodes):
    """A set of nodes as a signed 64-bit word."""
    m = sum(1 << j for j in nodes or ())
    return m - (1 << 64) if m >> 63 else m


def accept(parent, token, sampled):
    """(path, next token) of one tree. Tokens below 0 match nothing; without a root there is no path."""
    if len(parent) == 0 or parent[0] != -1:
        return [], -1
    path = [0]
    while True:
        at = path[-1]
        child = [j for j in range(at + 1, len(parent)) if parent[j] == at and token[j] == sampled[at] >= 0]
        if not child:
            return path, sampled[at]
        path.append(child[0])


def tree_attention(n_q, q, cache, seq, base, nodes, g=None, bias=None):
    """Rows q [n, n_q, D] of one tree of sequence `seq` behind `base` tokens: row j sees the context and `nodes`[j]
    (a set), with the cache's window its nearest ancestors and the context above its position less the window.
    Returns, before any rounding, og, sum p|v| (gated too), the keys seen per row, and per row
    and head max sum|q k| / sqrt(D) and max|v|."""
    n, _, D = q.shape
    out, mag = np.zeros((n, n_q * D)), np.zeros((n, n_q * D))
    counts, logit, most = np.zeros(n, int), np.zeros((n, n_q)), np.zeros((n, n_q))
    for j in range(n):
        tree = sorted(nodes[j])
        depth = len(tree)
        if depth == 0:
            continue
        W = cache.window
        first = max(1, base + depth - W + 1) if W else 1
        keys = list(range(first, base + 1)) + [base + 1 + a for a in (tree[-W:] if W else tree)]
        page = cache.table[seq, (np.array(keys) - 1) // cache.page_size]
        keys = np.array(keys)[(page >= 0) & (page < cache.k.shape[0])]   # those in a page
        counts[j] = len(keys)
        if len(keys) == 0:
            continue
        K, V = cache.load(seq, keys)
        for h in range(n_q):
            kv = h // (n_q // K.shape[0])
            x = K[kv] @ q[j, h] / np.sqrt(D)
            w = np.exp(x - np.max(x))
            w /= w.sum()
            out[j, h * D:(h + 1) * D] = w @ V[kv]
            mag[j, h * D:(h + 1) * D] = w @ np.abs(V[kv])
            logit[j, h] = np.max(np.abs(K[kv]) @ np.abs(q[j, h])) / np.sqrt(D)
            most[j, h] = np.max(np.abs(V[kv]))
    if g is not None:
        gate = 1 / (1 + np.exp(-(g.reshape(n, n_q, D) + bias[None, :, None]))).reshape(n, n_q * D)
        out, mag = out * gate, mag * gate
    return out, mag, counts, logit, most


def kept(z, t, k, p, m):
    """Indices that sampling from logits z may give, in ascending order."""
    z = np.asarray(z, np.float64)
    order = np.lexsort((np.arange(len(z)), -z))
    if not t >= 1e-30:
        return order[:1]
    if k > 0:
        order = order[:k]
    w = np.exp((z[order] - z[order[0]]) / t)
    if not p >= 1:
        order = order[:max(1, int(np.argmax(np.cumsum(w) >= max(p, 0) * w.sum())) + 1)]
    if m > 0:
        order = order[z[order] >= min(z[order[0]], z[order[0]] + t * np.log(m))]
    return np.sort(order)


def sample(z, u, t=1.0, k=0, p=1.0, m=0.0):
    """(token, log of its share of the kept weights). For the token weights count in steps of 2^-44 of the largest."""
    z = np.asarray(z, np.float64)
    if np.any(np.isnan(z)) or np.any(z == np.inf) or not np.any(np.isfinite(z)):
        return -1, np.nan
    at = kept(z, t, k, p, m)
    w = np.exp((z[at] - z[at].max()) / (t if t >= 1e-30 else 1.0))
    steps = np.floor(w * 2.0 ** 44)
    run = np.cumsum(steps)
    over = np.nonzero(run > u * run[-1])[0]
    j = over[0] if len(over) else np.nonzero(steps)[0][-1]
    return int(at[j]), float(np.log(w[j] / w.sum()))


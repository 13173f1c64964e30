"""Plain 64-bit forms of tree verification, its acceptance and append, the tokens' weights and the eviction."""
from __future__ import annotations

from fractions import Fraction

import numpy as np


# ---------------------------------------------------------------- trees

def random_tree(rng, T, kind="random", nodes=None):
    """Parents [T] of a tree of `nodes` nodes (the rest -2)."""
    n = T if nodes is None else nodes
    p = np.full(T, -2, np.int64)
    for v in range(n):
        p[v] = v - 1 if kind == "chain" else (v - 1) // 3 if kind == "wide" else int(rng.integers(max(0, v - 5), v)) if v else -1
    if n:
        p[0] = -1
    return p


def sees(parents):
    """[T][T] truth values: whether node v sees node u; none for what is no node."""
    T = len(parents)
    m = np.zeros((T, T), bool)
    alive = np.zeros(T, bool)
    for v, p in enumerate(parents):
        if p == -1:
            m[v, v] = alive[v] = True
        elif 0 <= p < v and alive[p]:
            m[v] = m[p]
            m[v, v] = alive[v] = True
    return m


# ---------------------------------------------------------------- acceptance

def grid(v):
    """floor(2^40 min(v, 1)) of float32 numbers as Python ints (0 for v <= 0, NaN and subnormals)."""
    v = np.asarray(v, np.float32).astype(np.float64)
    v = np.where(np.isnan(v), 0.0, np.clip(v, 0.0, 1.0))
    return np.floor(v * 2.0 ** 40).astype(np.int64)


def floor_of(u, total):
    """floor(u * total) for a float32 u in [0, 1)."""
    return int(Fraction(float(np.float32(u))) * int(total))


def accept_tree(q, draft, parents, u_acc, u_res):
    """One sequence: q [T][n] float32; (n_path, path [T], tokens [T])."""
    T, n = q.shape
    path, tokens = np.full(T, -1, np.int64), np.full(T, -1, np.int64)
    if parents[0] != -1:
        return 0, path, tokens
    node, count = 0, 0
    while True:
        path[count] = node
        count += 1
        w = grid(q[node])
        left, nxt = int(w.sum()), None
        for c in range(node + 1, T):
            if parents[c] != node or not 0 <= draft[c] < n:
                continue
            if floor_of(u_acc[c], left) < w[draft[c]]:
                nxt = c
                break
            left -= int(w[draft[c]])
            w[draft[c]] = 0
        if nxt is None:
            break
        tokens[count - 1] = draft[nxt]
        node = nxt
    if left:
        mark = min(floor_of(u_res, left), left - 1)
        tokens[count - 1] = int(np.searchsorted(np.cumsum(w), mark, side="right"))
    return count, path, tokens


# ---------------------------------------------------------------- weights and eviction

def weights(q, lse, keys, scale, first, visible=None):
    """q [rows][G][D], lse [rows][G], keys [n][D] of one KV head: sums [n] over the rows, row i at position first + i,
    and what the tolerance is made of: sum of p times the magnitude |scale| sum |q| |k| of its logit."""
    n = len(keys)
    total, spread = np.zeros(n), np.zeros(n)
    for i in range(len(q)):
        seen = np.arange(n) <= first + i
        if visible is not None:
            seen &= visible
        for g in range(q.shape[1]):
            if np.isneginf(lse[i, g]):
                continue
            p = np.where(seen, np.exp(scale * (keys @ q[i, g]) - lse[i, g]), 0.0)
            total += p
            spread += p * (abs(scale) * (np.abs(keys) @ np.abs(q[i, g])) + abs(lse[i, g]))
    return total, spread


def kept(w, length, budget, n_sink, n_recent):
    """Positions that one KV head keeps."""
    if length <= budget:
        return np.arange(length)
    inner = [t for t in range(n_sink, length - n_recent)]
    key = lambda t: (np.isnan(w[t]), -(0.0 if np.isnan(w[t]) else float(w[t])), t)
    best = sorted(inner, key=key)[: budget - n_sink - n_recent]
    return np.array(sorted([*range(n_sink), *best, *range(length - n_recent, length)]), np.int64)

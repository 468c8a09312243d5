"""fp64 reference for attention with shared key heads, the attention weight of cached tokens and
eviction by it.  TEST INFRASTRUCTURE ONLY (see the package docstring).

Every function takes values already upcast to float64 (eviction: any values, which it moves) and
loops over the sequences as the definitions are written; nothing here is shared with the library.
"""

from __future__ import annotations

import numpy as np


def rows_of(cache, table, length, head):
    """Rows ``[length, D]`` of one head of a sequence."""
    bs = cache.shape[2]
    return np.stack([cache[int(table[t // bs]), head, t % bs] for t in range(length)]) if length else (
        np.zeros((0, cache.shape[3])))


def softmax_rows(q, k_cache, table, length, places, scale):
    """Softmax weights ``[R, Hq, length]`` of rows q ``[R, Hq, D]``, row r over the places 0 ..
    places[r]; the logarithm of each row's sum ``[R, Hq]``; and the largest of scale * sum_d |q_d k_td|
    over the places it sees ``[R, Hq]`` (for error bounds)."""
    r, hq, _ = q.shape
    group = hq // k_cache.shape[1]
    w, lse, reach = np.zeros((r, hq, length)), np.full((r, hq), -np.inf), np.zeros((r, hq))
    for h in range(k_cache.shape[1]):
        k = rows_of(k_cache, table, length, h)
        for g in range(h * group, (h + 1) * group):
            for i in range(r):
                n = int(places[i]) + 1
                if n <= 0:
                    continue
                s = k[:n] @ q[i, g] * scale
                top = s.max()
                e = np.exp(s - top)
                w[i, g, :n], lse[i, g] = e / e.sum(), top + np.log(e.sum())
                reach[i, g] = (np.abs(k[:n]) @ np.abs(q[i, g])).max() * abs(scale)
    return w, lse, reach


def weighted(w, v_cache, table, length):
    """``[R, Hq, D]``: sum_t w_t v_t, and sum_t w_t |v_t| and sum_t |v_t| (for error bounds)."""
    r, hq, _ = w.shape
    h, d = v_cache.shape[1], v_cache.shape[3]
    out, spread, size = (np.zeros((r, hq, d)) for _ in range(3))
    for head in range(h):
        v = rows_of(v_cache, table, length, head)
        for g in range(head * (hq // h), (head + 1) * (hq // h)):
            out[:, g], spread[:, g], size[:, g] = w[:, g] @ v, w[:, g] @ np.abs(v), np.abs(v).sum(0)
    return out, spread, size


def by_key_head(w, kv_heads):
    """``[R, Hq, L]`` summed over rows and over the query heads of a key head: ``[H, L]``."""
    r, hq, length = w.shape
    return w.reshape(r, kv_heads, hq // kv_heads, length).sum((0, 2))


def evict(k_cache, v_cache, tables, seq_lens, kept, weights=None, new_tables=None):
    """In place: place j of (sequence, key head) takes the rows and the weight that place
    kept[i][h][j] held; places without an entry keep their rows, in a new block too, and their
    weights become 0."""
    old_k, old_v, bs = k_cache.copy(), v_cache.copy(), k_cache.shape[2]
    to = tables if new_tables is None else new_tables
    for i, length in enumerate(seq_lens):
        for h in range(k_cache.shape[1]):
            if weights is not None:
                old_w = weights[i, h].copy()
                weights[i, h, :int(length)] = 0
            for j in range(min(int(length), kept.shape[2])):
                entry = int(kept[i, h, j])
                s = j if entry < 0 else entry
                if entry < 0 and (j // bs >= len(to[i]) or to[i][j // bs] < 0):
                    continue                            # a place that the sequence does not keep
                a, b = int(tables[i][s // bs]), int(to[i][j // bs])
                k_cache[b, h, j % bs] = old_k[a, h, s % bs]
                v_cache[b, h, j % bs] = old_v[a, h, s % bs]
                if weights is not None and entry >= 0:
                    weights[i, h, j] = old_w[s]

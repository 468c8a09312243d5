"""fp64 reference for the append with rotary positions and for decode attention over
selected blocks.  TEST INFRASTRUCTURE ONLY (see the package docstring).

Every function takes values already upcast to float64 and loops over the sequences as
the definitions are written; nothing here is shared with the library.
"""

from __future__ import annotations

import numpy as np


def rotate(x, cos_sin, positions, pair_axis=None, interleaved=False):
    """x ``[T, H, D]`` rotated: pair j of token t turns by the angle whose cosine and sine
    are ``cos_sin[P][j]`` and ``cos_sin[P][R/2 + j]``, P the token's position on the pair's
    axis (positions ``[T]`` or ``[axes, T]``).  Pairs are dims (j, j + R/2), or (2 j, 2 j + 1)
    when interleaved; dims R and up are left alone."""
    x = np.array(x, dtype=np.float64)
    table = np.asarray(cos_sin, dtype=np.float64)
    half = table.shape[1] // 2
    pos = np.atleast_2d(np.asarray(positions, dtype=np.int64))
    for j in range(half):
        at = pos[0 if pair_axis is None else int(pair_axis[j])]
        c, s = table[at, j][:, None], table[at, half + j][:, None]
        d0, d1 = (2 * j, 2 * j + 1) if interleaved else (j, j + half)
        a, b = x[:, :, d0].copy(), x[:, :, d1].copy()
        x[:, :, d0], x[:, :, d1] = a * c - b * s, b * c + a * s
    return x


def new_places(query_start, seq_lens):
    """For every new token: (row of q/k/v, sequence, place in the sequence)."""
    out = []
    for i, length in enumerate(seq_lens):
        a, b = int(query_start[i]), int(query_start[i + 1])
        out.extend((a + j, i, int(length) - (b - a) + j) for j in range(b - a))
    return out


def block_bounds(k_cache, block_tables, seq_lens, k_min, k_max, first_token=None):
    """In place: k_min, k_max ``[B, H, D]`` of every block that holds a token at or past
    first_token, over the rows of tokens below the sequence's length."""
    bs = k_cache.shape[2]
    for i, length in enumerate(seq_lens):
        first = 0 if first_token is None else max(int(first_token[i]), 0)
        for b in range(first // bs, -(-int(length) // bs)):
            rows = k_cache[int(block_tables[i][b]), :, :min(bs, int(length) - b * bs)]
            k_min[int(block_tables[i][b])] = rows.min(axis=1)
            k_max[int(block_tables[i][b])] = rows.max(axis=1)


def block_scores(q, k_min, k_max, block_tables, seq_lens, scale, block_size):
    """``[N, H, MB]``: scale times the largest, over the query heads g of key head h, of
    sum_d max(q_d, 0) k_max_d + min(q_d, 0) k_min_d; -inf past a sequence's blocks.  The
    second result is the sum of the terms' magnitudes (for error bounds)."""
    n, mb = np.shape(block_tables)
    h = k_min.shape[1]
    group = q.shape[1] // h
    out = np.full((n, h, mb), -np.inf)
    size = np.zeros((n, h, mb))
    for i in range(n):
        for b in range(-(-int(seq_lens[i]) // block_size)):
            blk = int(block_tables[i][b])
            for hh in range(h):
                x = q[i, hh * group:(hh + 1) * group]
                terms = np.maximum(x, 0) * k_max[blk, hh], np.minimum(x, 0) * k_min[blk, hh]
                out[i, hh, b] = scale * (terms[0] + terms[1]).sum(axis=1).max()
                size[i, hh, b] = scale * (np.abs(terms[0]) + np.abs(terms[1])).sum(axis=1).max()
    return out, size


def block_select(scores, seq_lens, block_size, num_selected, sink=0, recent=0):
    """``[N, H, num_selected]``: all blocks if they fit, else the first ``sink``, the last
    ``recent`` and the best of the others (NaN above every number, ties to the lower
    block), ascending, padded with -1."""
    n, h, _ = scores.shape
    out = np.full((n, h, num_selected), -1, dtype=np.int32)
    for i in range(n):
        held = -(-int(seq_lens[i]) // block_size)
        for hh in range(h):
            if held <= num_selected:
                keep = list(range(held))
            else:
                forced = list(range(sink)) + list(range(held - recent, held))
                s = [float(x) for x in scores[i, hh, :held]]
                rest = sorted(range(sink, held - recent),
                              key=lambda b: (0 if s[b] != s[b] else 1, -s[b] if s[b] == s[b] else 0, b))
                keep = sorted(forced + rest[:num_selected - sink - recent])
            out[i, hh, :len(keep)] = keep
    return out


def sparse_attention(q, k_cache, v_cache, block_tables, seq_lens, selected, scale):
    """Attention of each query head over the tokens (below the length) of the blocks its key
    head lists; -1 and blocks past the end hold none; no token at all: zeros.  Returns
    ``(out, spread, reach)`` ``[N, Hq, D]``, ``[N, Hq, D]``, ``[N, Hq]``: the result,
    sum_t w_t |v_t|, and max_t of scale * sum_d |q_d k_td| (for error bounds)."""
    n, hq, d = q.shape
    h, bs = k_cache.shape[1:3]
    group = hq // h
    out, spread, reach = np.zeros((n, hq, d)), np.zeros((n, hq, d)), np.zeros((n, hq))
    for i in range(n):
        length = int(seq_lens[i])
        for hh in range(h):
            ks, vs = [], []
            for b in selected[i][hh]:
                if b < 0 or b * bs >= length:
                    continue
                rows = min(bs, length - int(b) * bs)
                blk = int(block_tables[i][int(b)])
                ks.append(k_cache[blk, hh, :rows])
                vs.append(v_cache[blk, hh, :rows])
            if not ks:
                continue
            k, v = np.concatenate(ks), np.concatenate(vs)
            for g in range(hh * group, (hh + 1) * group):
                s = k @ q[i, g] * scale
                w = np.exp(s - s.max())
                w /= w.sum()
                out[i, g], spread[i, g] = w @ v, w @ np.abs(v)
                reach[i, g] = (np.abs(k) @ np.abs(q[i, g])).max() * abs(scale)
    return out, spread, reach

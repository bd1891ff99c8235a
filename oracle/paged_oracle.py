"""Plain fp64 statement of the paged key-value cache's operators (numpy).

``append``: the call's tokens go to their pages.  ``attend``: causal softmax attention of a
sequence's last tokens over all of its tokens, or over a window of them and the first ``sinks``
positions.  No kernel's order of summation, tiling or page walk appears here.
"""
from __future__ import annotations

import math

import numpy as np

__all__ = ["append", "gather", "visible", "attend"]


def append(pool, table, lens, new, new_start, page_size):
    """pool [pages][heads][page_size][d] gets rows of new [tokens][heads][d]; returns a copy."""
    pool = pool.copy()
    for b, n in enumerate(lens):
        rows = range(new_start[b], new_start[b + 1])
        for i, row in enumerate(rows):
            p = n - len(rows) + i
            pool[table[b][p // page_size], :, p % page_size] = new[row]
    return pool


def gather(pool, table_row, n, page_size):
    """The first n tokens of a sequence, [heads][n][d]."""
    rows = [pool[table_row[p // page_size], :, p % page_size] for p in range(n)]
    return np.stack(rows, axis=1) if rows else np.zeros((pool.shape[1], 0, pool.shape[3]))


def visible(positions, n, window, sinks):
    """[len(positions)][n]: does the query at that position see key j?"""
    p = np.asarray(positions)[:, None]
    j = np.arange(n)[None]
    see = j <= p
    if window > 0:
        see &= (j > p - window) | (j < sinks)
    return see


def attend(q, k, v, see):
    """q [rows][q_heads][d], k and v [kv_heads][n][d], see [rows][n].

    Returns out [rows][q_heads][d], lse [rows][q_heads], and two sizes that bounds on rounding
    need: sum_j p_j |v_j| (shape of out) and max_j sum_i |q_i k_ji| / sqrt(d) over the keys that a
    row sees [rows][q_heads]."""
    q, k, v = (np.asarray(x, dtype=np.float64) for x in (q, k, v))
    rows, heads, d = q.shape
    group = heads // k.shape[0]
    out, size = np.zeros((rows, heads, d)), np.zeros((rows, heads, d))
    lse, dots = np.full((rows, heads), -math.inf), np.zeros((rows, heads))
    for i in range(rows):
        at = np.flatnonzero(see[i])
        if at.size == 0:
            continue
        for h in range(heads):
            kk, vv = k[h // group][at], v[h // group][at]
            s = kk @ q[i, h] / math.sqrt(d)
            m = s.max()
            w = np.exp(s - m)
            out[i, h] = w @ vv / w.sum()
            size[i, h] = w @ np.abs(vv) / w.sum()
            lse[i, h] = m + math.log(w.sum())
            dots[i, h] = (np.abs(kk) @ np.abs(q[i, h])).max() / math.sqrt(d)
    return out, lse, size, dots

"""Attention over a sliding window and the first tokens of a sequence, stated
plainly (test oracle).

TEST INFRASTRUCTURE ONLY -- see the package docstring.  Imports: numpy.

The query at absolute position p attends to key j iff j <= p and (j > p -
window or j < num_sinks); otherwise this is the attention of
paged_attention.py.  Only the pages that hold a key some query row of the
sequence attends to are read from the pool.
"""
from __future__ import annotations

import numpy as np


def visible_keys(position, window, num_sinks):
    """The keys the query at `position` attends to, ascending (none below 0)."""
    return [j for j in range(position + 1) if j > position - window or j < num_sinks]


def _one_row(key_pool, value_pool, q, row, position, scale, window, num_sinks):
    hq, d = q.shape
    ps, hkv = key_pool.shape[1], key_pool.shape[2]
    keys = visible_keys(position, window, num_sinks)
    out = np.zeros((hq, d))
    if not keys:
        return out
    K = np.stack([key_pool[int(row[j // ps]), j % ps] for j in keys]).astype(np.float64)
    V = np.stack([value_pool[int(row[j // ps]), j % ps] for j in keys]).astype(np.float64)
    for h in range(hq):
        s = scale * (K[:, h // (hq // hkv)] @ q[h])
        w = np.exp(s - s.max())
        out[h] = (w @ V[:, h // (hq // hkv)]) / w.sum()
    return out


def paged_attention_decode_window(key_pool, value_pool, q, block_table, seq_lens, scale, window, num_sinks):
    """One query token per sequence at position L_b - 1: ``q [B, Hq, D]`` ->
    ``[B, Hq, D]``; an empty sequence gives 0."""
    q = np.asarray(q, dtype=np.float64)
    return np.stack([_one_row(key_pool, value_pool, q[b], block_table[b], int(seq_lens[b]) - 1, scale, window,
                              num_sinks) for b in range(q.shape[0])])


def paged_attention_prefill_window(key_pool, value_pool, q, query_start_loc, block_table, seq_lens, scale, window,
                                   num_sinks):
    """Packed new tokens: row i of sequence b at position L_b - n_b + i; a row
    below position 0 gives 0."""
    q = np.asarray(q, dtype=np.float64)
    out = np.zeros(q.shape)
    for b in range(len(query_start_loc) - 1):
        s0, s1 = int(query_start_loc[b]), int(query_start_loc[b + 1])
        for r in range(s0, s1):
            out[r] = _one_row(key_pool, value_pool, q[r], block_table[b], int(seq_lens[b]) - (s1 - r), scale, window,
                              num_sinks)
    return out

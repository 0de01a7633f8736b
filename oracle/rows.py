"""What happens to rows around attention, stated plainly (test oracle): the
per-head norm and the rotation of queries and keys, page copies and in-place
compaction of a sequence's rows.

TEST INFRASTRUCTURE ONLY -- see the package docstring.  Imports: numpy.
"""
from __future__ import annotations

import numpy as np


def rms_norm(x, weight, eps):
    """x / sqrt(mean(x^2) + eps) * weight over the last axis (x itself without a weight)."""
    x = np.asarray(x, dtype=np.float64)
    if weight is None:
        return x.copy()
    return x / np.sqrt((x * x).mean(axis=-1, keepdims=True) + eps) * np.asarray(weight, dtype=np.float64)


def rotate(x, cos, sin, interleaved):
    """Turn the pairs of the first 2 * len(cos) dims of ``x [H, D]``."""
    x = np.asarray(x, dtype=np.float64).copy()
    half = len(cos)
    for i in range(half):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
        xa, xb = x[:, a].copy(), x[:, b].copy()
        x[:, a] = xa * cos[i] - xb * sin[i]
        x[:, b] = xb * cos[i] + xa * sin[i]
    return x


def qk_norm_rope(q, key, positions, cos_sin, q_weight, k_weight, eps, interleaved):
    """fp64 normed and rotated rows of ``q [T, Hq, D]`` and ``key [T, Hkv, D]``."""
    outs = []
    for x, w in ((q, q_weight), (key, k_weight)):
        y = rms_norm(x, w, eps)
        if cos_sin is not None:
            half = cos_sin.shape[1] // 2
            for t in range(y.shape[0]):
                row = np.asarray(cos_sin[int(positions[t])], dtype=np.float64)
                y[t] = rotate(y[t], row[:half], row[half:], interleaved)
        outs.append(y)
    return outs


def paged_kv_copy_pages(pool, src_pages, dst_pages):
    """A copy of ``pool [P, ...]`` in which page dst becomes the old page src for
    each pair; pairs with a negative entry do nothing."""
    pool = np.asarray(pool)
    out = pool.copy()
    for s, d in zip(src_pages, dst_pages):
        if s >= 0 and d >= 0:
            out[int(d)] = pool[int(s)]
    return out


def paged_kv_compact(pool, block_table, base, keep_indptr, keep):
    """A copy of ``pool [P, ps, ...]`` in which row base[b] + i of sequence b is
    its old row keep[keep_indptr[b] + i]."""
    pool = np.asarray(pool)
    ps = pool.shape[1]
    out = pool.copy()
    for b in range(len(keep_indptr) - 1):
        for i, old in enumerate(keep[int(keep_indptr[b]):int(keep_indptr[b + 1])]):
            new = int(base[b]) + i
            out[int(block_table[b][new // ps]), new % ps] = pool[int(block_table[b][int(old) // ps]), int(old) % ps]
    return out


def rope_table(max_position, rotary_dim, theta=10000.0):
    """[max_position, rotary_dim]: cosines, then sines, of p * theta^(-2i / rotary_dim)."""
    inv = np.array([theta ** (-2.0 * i / rotary_dim) for i in range(rotary_dim // 2)])
    ang = np.arange(max_position, dtype=np.float64)[:, None] * inv[None, :]
    return np.concatenate([np.cos(ang), np.sin(ang)], axis=1)

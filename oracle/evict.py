"""Attention weights of cached keys and the choice of what to evict by them, stated
plainly (test oracle).

TEST INFRASTRUCTURE ONLY -- see the package docstring.  Imports: numpy.
"""
from __future__ import annotations

import numpy as np


def key_weights(key_pool, q, block_table, seq_lens, scale):
    """Per sequence, the softmax weights of its keys summed over the query heads
    (fp64 ``[L_b]`` each): q ``[B, Hq, D]``, key_pool ``[P, page_size, Hkv, D]``."""
    P, ps, hkv, d = key_pool.shape
    hq = q.shape[1]
    out = []
    for b, L in enumerate(np.asarray(seq_lens).tolist()):
        total = np.zeros(L)
        j = np.arange(L)
        K = np.asarray(key_pool[np.asarray(block_table)[b, j // ps], j % ps], dtype=np.float64)
        for h in range(hq):
            if L == 0:
                continue
            x = scale * (K[:, h // (hq // hkv)] @ np.asarray(q[b, h], dtype=np.float64))
            w = np.exp(x - x.max())
            total += w / w.sum()
        out.append(total)
    return out


def _heaviest(weights, first, last, count):
    """The `count` indices of [first, last) with the largest weights (NaN lightest,
    ties: the lower index)."""
    w = [(-np.inf if np.isnan(x) else float(x), not np.isnan(x)) for x in weights[first:last]]
    order = sorted(range(len(w)), key=lambda i: (not w[i][1], -w[i][0], i))
    return [first + i for i in order[:count]]


def evict_rows(mass, seq_lens, budget, num_sinks, num_recent):
    """Per sequence ``(base, kept rows at or past base)``."""
    out = []
    for row, L in zip(mass, np.asarray(seq_lens).tolist()):
        if L <= budget:
            out.append((L, []))
            continue
        top = _heaviest(row, num_sinks, L - num_recent, budget - num_sinks - num_recent)
        out.append((num_sinks, sorted(top) + list(range(L - num_recent, L))))
    return out


def page_weight(row):
    """Halves added again and again, in float32."""
    x = np.asarray(row, dtype=np.float32)
    while len(x) > 1:
        x = x[:len(x) // 2] + x[len(x) // 2:]
    return x[0]


def evict_pages(mass, seq_lens, page_size, budget, num_sinks, num_recent):
    """Per sequence ``(pages that stay, pages that go)``, ascending."""
    out = []
    for row, L in zip(mass, np.asarray(seq_lens).tolist()):
        n = -(-L // page_size)
        if n <= budget:
            out.append((list(range(n)), []))
            continue
        x = np.zeros(n * page_size, dtype=np.float32)
        x[:L] = row[:L]
        with np.errstate(all="ignore"):
            weights = [page_weight(x[i * page_size:(i + 1) * page_size]) for i in range(n)]
        front, back = -(-num_sinks // page_size), max(0, L - max(1, num_recent)) // page_size
        stay = sorted(list(range(front)) + _heaviest(weights, front, back, budget - front - (n - back))
                      + list(range(back, n)))
        gone = set(range(n)) - set(stay)
        out.append((stay, sorted(gone)))
    return out


def moved(row, kept, width):
    """The masses of the kept rows in front, zeros up to `width`."""
    out = np.zeros(width, dtype=np.float32)
    out[:len(kept)] = np.asarray(row)[kept]
    return out

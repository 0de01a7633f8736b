"""int8 KV pools with a scale for each block of tokens and KV head, stated plainly
(test oracle).

A pool ``codes [P, page_size, Hkv, D]`` int8 and its ``scales [P, page_size /
block, Hkv]`` float32: code c of slot s and head h stands for ``c * scales[s //
block, h]``, a scale counting as at least 2**-40 and at most 2**40.

The append's arithmetic is that of float32 (numpy's, IEEE): it decides which code
a value gets, so it belongs to the definition.

TEST INFRASTRUCTURE ONLY -- see the package docstring.  Imports: numpy.
"""
from __future__ import annotations

import numpy as np

SCALE_MIN, SCALE_MAX = np.float32(2.0 ** -40), np.float32(2.0 ** 40)


def clamp_scale(s):
    """NaN counts as the least scale."""
    s = np.asarray(s, dtype=np.float32)
    return np.minimum(np.where(s > SCALE_MIN, s, SCALE_MIN), SCALE_MAX)


def dequantize(codes, scales):
    """fp64 values of a pool."""
    P, ps, hkv, d = codes.shape
    blocks = scales.shape[1]
    s = clamp_scale(scales).astype(np.float64)
    x = np.asarray(codes, dtype=np.float64).reshape(P, blocks, ps // blocks, hkv, d)
    return (x * s[:, :, None, :, None]).reshape(P, ps, hkv, d)


def _round(x):
    """Nearest integer, ties to even, within +-127; NaN becomes 0."""
    y = np.rint(np.nan_to_num(x, nan=0.0, posinf=1e9, neginf=-1e9))
    return np.clip(y, -127, 127).astype(np.int8)


def append_int8(codes, scales, rows, slot_mapping):
    """(codes, scales) after the rows ``[T, Hkv, D]`` float32 are written at their
    slots (negative: skipped)."""
    codes, scales = np.array(codes), np.array(scales, dtype=np.float32)
    P, ps, hkv, d = codes.shape
    block = ps // scales.shape[1]
    flat, sc = codes.reshape(-1, block, hkv, d), scales.reshape(-1, hkv)
    rows = np.asarray(rows, dtype=np.float32)
    written = {}
    for t, s in enumerate(np.asarray(slot_mapping).tolist()):
        if s >= 0:
            written.setdefault(s // block, []).append((t, s % block))
    for b, places in written.items():
        tokens, at = [t for t, _ in places], [o for _, o in places]
        for h in range(hkv):
            x = rows[tokens, h]
            a = np.abs(x[~np.isnan(x)]).max(initial=np.float32(0))
            with np.errstate(all="ignore"):
                s = clamp_scale(np.float32(a) / np.float32(127))
                if 0 not in at:
                    old = clamp_scale(sc[b, h])
                    if s > old:
                        flat[b, :, h] = _round(flat[b, :, h].astype(np.float32) * (old / s))
                    s = max(s, old)
                flat[b, at, h] = _round(x / s)
            sc[b, h] = s
    return codes, scales

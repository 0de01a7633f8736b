"""The attention over an int8 pool judged row by row and head by head: nothing that a row
does not see may show in it, however far apart the scales of its tile's blocks are.

Tolerance of an element, with w_j the row's weights of the keys that it sees, v_j their
scales, c_j their codes, V_j = v_j c_j and A = sum_j w_j |V_j|:
  its rounding to bf16: 2^-8 |y|;
  the weights times scales of the product, rounded to f16: 2^-11 A, and, as f16 has steps of
  2^-24 below 2^-14, relative to the largest w_j v_j: 2^-25 max_j (w_j v_j) sum_j |c_j|;
  fp32 products, sums, logarithms and exponentials of arguments up to 2^8: 2^-12 A;
  the scores: fp32 sums of d products of codes and f16 queries, d <= 128, each addition off by
  2^-23 of sum_d |q_d K_d| at most, so e = 2^-16 scale max_j sum_d |q_d K_jd|, which moves the
  row by (exp(2 e) - 1) (A + |y|), and by no more than 2 max_j |V_j| (both are means)."""
from __future__ import annotations

import numpy as np

import oracle
from _int8 import Case
from _parity import bits, to_f64


class RowCase(Case):
    def rows(self):
        """(y, tol, e): per row and head, [T, Hq, D], [T, Hq, D], [T, Hq]; rows in the order of q."""
        assert self.dtype == "int8" and not self.bad
        K, V = self.values()
        sv = oracle.kv_int8.clamp_scale(self.vs.numpy()).astype(np.float64)
        codes = self.vp.numpy().astype(np.float64)
        q = to_f64(bits(self.q))
        G = q.shape[1] // K.shape[2]
        y, tol, e = np.zeros_like(q), np.zeros_like(q), np.zeros(q.shape[:2])
        for b, L in enumerate(self.lens.tolist()):
            n = int(self.n[b])
            j = np.arange(L)
            page, off = self.seen[b, j // self.ps], j % self.ps
            for i in range(n):
                t, see = int(self.qsl[b]) + i, L - n + i + 1
                if self.is_decode:
                    t, see = b, L
                if see <= 0:
                    continue
                p, o = page[:see], off[:see]
                for h in range(q.shape[1]):
                    k, v = K[p, o, h // G], V[p, o, h // G]
                    x = self.scale * (k @ q[t, h])
                    w = np.exp(x - x.max())
                    w /= w.sum()
                    y[t, h] = w @ v
                    a = w @ np.abs(v)
                    small = (w * sv[p, o // self.blk, h // G]).max() * np.abs(codes[p, o, h // G]).sum(axis=0)
                    e[t, h] = 2.0 ** -16 * abs(self.scale) * (np.abs(k) @ np.abs(q[t, h])).max()
                    moved = np.expm1(min(2 * e[t, h], 50.0)) * (a + np.abs(y[t, h]))
                    tol[t, h] = (2.0 ** -8 * np.abs(y[t, h]) + (2.0 ** -11 + 2.0 ** -12) * a + 2.0 ** -25 * small +
                                 np.minimum(moved, 2 * np.abs(v).max(axis=0)))
        return y, tol, e

    def compare(self, out, exp=None, judged=0.75):
        """All rows within tolerance; at least `judged` of the rows are such that zeros, or any
        other answer that misses them, would not pass."""
        y, tol, e = exp or self.rows()
        got = to_f64(bits(out))
        assert np.isfinite(got).all()
        err = np.abs(got - y)
        worst = (err / np.maximum(tol, 1e-300)).max(axis=(1, 2))
        assert (err <= tol).all(), f"row {worst.argmax()}: {worst.max():.3g} of its tolerance, {(worst > 1).sum()} rows past it"
        told = (np.abs(y) > tol).mean(axis=2) > 0.75
        assert told.mean() >= judged, f"zeros would pass in {1 - told.mean():.2f} of the rows"

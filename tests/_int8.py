"""Inputs of the tests of int8 pools: codes and scales in which every slot that holds
no live key has garbage codes and every block without one a garbage scale, the
oracle's result on the values that the codes stand for, and a tolerance.

Tolerance, per output element, with A = sum_j w_j |v_j| (the oracle's attention over
|V|) and n keys: the output's rounding to bf16 is off by at most 2^-8 |y|; the
weights of the PV product are rounded to f16, at most 2^-11 each, so 2^-11 A; f16
weights below 2^-14 have steps of 2^-24, half of that per key, beside codes of at most
127 and relative to the row's largest weight times scale: 2^-25 * 127 n max s; fp32
products, sums, the logarithm of a scale and the exponential: 2^-12 A.  The prefill
rounds a code times its scale to f16 in two steps (ratio, product): 2^-10 of V, so
2^-10 A, and 2^-10 of K, which moves a score by at most e = 2^-10 scale sum_d |q_d K_d|
and a row's result by at most (exp(2 e) - 1) (A + |y|), and, however far the scores
move, by no more than 2 max_j |v_j|: both results are means of the v_j."""
from __future__ import annotations

import numpy as np
import torch

import oracle
from _parity import bits, to_f64


class Case:
    """Sequences of cached + new tokens (new all 1: a decode; cached -1: no key)."""

    score_error = 0.0

    def __init__(self, new, cached, hq=8, hkv=2, d=64, ps=16, blk=16, seed=0, scale=None, spread=0.5, dtype="int8",
                 bad=(), k_scale=0.02, v_scale=0.03, room=0):
        rng = np.random.default_rng(seed)
        self.ps, self.blk, self.d, self.dtype = ps, blk, d, dtype
        self.n = np.asarray(new, dtype=np.int64)
        self.lens = np.maximum(np.asarray(cached, dtype=np.int64) + self.n, 0).astype(np.int32)
        B = len(self.lens)
        self.qsl = np.concatenate([[0], np.cumsum(self.n)]).astype(np.int32)
        # room: more columns than the sequences need, and a bound on their lengths as wide: a
        # decode then takes the kernel for long contexts
        mb = max(1, int((self.lens.max(initial=0) + ps - 1) // ps)) + 1 + room
        self.max_len = mb * ps if room else max(1, int(self.lens.max(initial=0)))
        pages = [int(-(-int(L) // ps)) for L in self.lens]
        P = sum(pages) + 4
        ids = iter(rng.permutation(P))
        self.table = np.full((B, mb), -7, dtype=np.int32)
        live = np.zeros((P, ps), dtype=bool)
        for b in range(B):
            for m in range(pages[b]):
                p = next(ids)
                self.table[b, m] = p
                live[p, :max(0, min(ps, int(self.lens[b]) - m * ps))] = True
        self.live = live
        self.scale = d ** -0.5 if scale is None else scale
        self.k_scale, self.v_scale = (k_scale, v_scale) if dtype == "e4m3" else (1.0, 1.0)
        self.kp, self.ks = self._pool(rng, P, ps, blk, hkv, d, live, spread)
        self.vp, self.vs = self._pool(rng, P, ps, blk, hkv, d, live, spread)
        g = torch.Generator().manual_seed(seed)
        self.q = torch.randn(B if self.is_decode else int(self.n.sum()), hq, d, generator=g).to(torch.bfloat16)
        self.seen = self.table.copy()          # what the oracle reads
        self.bad = list(bad)                   # (sequence, page) whose entry is out of range
        for i, (b, m) in enumerate(self.bad):
            self.table[b, m] = (P, -1, 1 << 30)[i % 3]

    def _pool(self, rng, P, ps, blk, hkv, d, live, spread):
        x = rng.standard_normal((P, ps, hkv, d)).astype(np.float32)
        if self.dtype != "int8":
            x[~live] = np.nan
            t = torch.from_numpy(x)
            s = self.k_scale if not hasattr(self, "kp") else self.v_scale
            return (t.to(torch.bfloat16) if self.dtype == "bf16" else (t / s).clamp(-448, 448).to(torch.float8_e4m3fn)), None
        size = np.exp(spread * rng.standard_normal((P, ps // blk, 1, hkv, 1))).astype(np.float32)
        x = (x.reshape(P, ps // blk, blk, hkv, d) * size)
        s = np.abs(x).max(axis=(2, 4), keepdims=True) / np.float32(127)
        codes = np.rint(x / s).astype(np.int8).reshape(P, ps, hkv, d)
        scales = s.reshape(P, ps // blk, hkv).astype(np.float32)
        junk = rng.integers(-128, 128, size=codes.shape, dtype=np.int8)
        codes[~live] = junk[~live]
        dead = ~live.reshape(P, ps // blk, blk).any(axis=2)
        odd = np.asarray([np.nan, np.inf, -np.inf, 0.0, -1.0, 3e38], dtype=np.float32)
        scales[dead] = odd[rng.integers(0, len(odd), size=scales.shape)][dead]
        return torch.from_numpy(codes), torch.from_numpy(scales)

    @property
    def is_decode(self):
        return bool((self.n == 1).all())

    def values(self):
        out = []
        for x, s, t in ((self.kp, self.ks, self.k_scale), (self.vp, self.vs, self.v_scale)):
            if self.dtype == "int8":
                v = oracle.kv_int8.dequantize(x.numpy(), s.numpy())
            elif self.dtype == "e4m3":
                v = oracle.kv_fp8.dequantize(bits(x), t)
            else:
                v = to_f64(bits(x))
            out.append(np.where(self.live[:, :, None, None], v, 0.0))
        return out

    def _compact(self, V):
        """Tables and lengths without the keys of pages that are out of range (decode)."""
        lens, table = self.lens.copy(), self.seen.copy()
        for b in range(len(lens)):
            gone = sorted(m for bb, m in self.bad if bb == b)
            keep = [m for m in range(-(-int(lens[b]) // self.ps)) if m not in gone]
            for m in gone:
                assert (m + 1) * self.ps <= lens[b]   # whole pages here: the last one moves up unchanged
            lens[b] -= self.ps * len(gone)
            table[b, :len(keep)] = self.seen[b, keep]
        return table, lens

    def oracle(self):
        K, V = self.values()
        q = to_f64(bits(self.q))
        A = lambda k, v, qq, s: (oracle.paged_attention_decode(k, v, qq, *self._compact(v), s) if self.is_decode else
                                 oracle.paged_attention_prefill(k, v, qq, self.qsl, self.seen, self.lens, s))
        y, a = A(K, V, q, self.scale), A(K, np.abs(V), q, self.scale)
        n = int(self.lens.max(initial=0))
        w = 2.0 ** -8 if self.dtype == "bf16" else 2.0 ** -11
        if self.dtype == "int8":
            s = oracle.kv_int8.clamp_scale(self.vs.numpy())
            alive = self.live.reshape(s.shape[0], s.shape[1], -1).any(axis=2)
            smax = float(s[alive].max(initial=0.0))
        else:
            smax = self.v_scale
        small = 2.0 ** -25 * (448 if self.dtype == "e4m3" else 127) * n * smax if self.dtype != "bf16" else 0.0
        tol = 2.0 ** -8 * np.abs(y) + (w + 2.0 ** -12) * a + small
        if not self.is_decode:
            G = q.shape[1] // K.shape[2]
            e = np.zeros(q.shape[:2])
            for b in range(len(self.lens)):   # largest of sum_d |q_d K_d| over the sequence's keys
                j = np.arange(int(self.lens[b]))
                k = np.abs(K[self.seen[b, j // self.ps], j % self.ps]) if len(j) else np.zeros((1,) + K.shape[2:])
                for h in range(q.shape[1]):
                    rows = np.abs(q[self.qsl[b]:self.qsl[b + 1], h])
                    e[self.qsl[b]:self.qsl[b + 1], h] = (rows @ k[:, h // G].T).max(axis=1, initial=0.0)
            e *= 2.0 ** -10 * abs(self.scale)
            moved = np.expm1(np.minimum(2 * e, 50.0))[:, :, None] * (a + np.abs(y))
            tol += 2.0 ** -10 * a + np.minimum(moved, 2 * np.abs(V).max())
            self.score_error = float(e.max(initial=0.0))
        return y, tol

    def tensors(self, device):
        dev = lambda a: (a if torch.is_tensor(a) else torch.from_numpy(np.ascontiguousarray(a))).to(device)
        return [None if t is None else dev(t) for t in (self.kp, self.vp, self.ks, self.vs, self.q, self.table, self.lens,
                                                        self.qsl)]

    def run(self, capi, device, **k):
        kp, vp, ks, vs, q, bt, L, qsl = self.args = self.tensors(device)
        k.setdefault("max_seq_len", self.max_len)
        k.setdefault("out", torch.full_like(q, float("nan")))
        if self.is_decode:
            return capi.paged_attention_decode_int8(kp, vp, ks, vs, q, bt, L, self.scale, **k)
        return capi.paged_attention_prefill_int8(kp, vp, ks, vs, q, qsl, bt, L, self.scale, int(self.n.max()), **k)

    def compare(self, out, exp=None):
        got = to_f64(bits(out))
        y, tol = exp or self.oracle()
        assert np.isfinite(got).all()
        err = np.abs(got - y)
        assert (err <= tol).all(), f"error {err.max():.3e}, {(err / np.maximum(tol, 1e-30)).max():.2f} of the tolerance"
        # all of it, as a norm: the output's own rounding is the largest part, 2^-8 at most
        # (unless a prefill's scores are so large that their roundings turn the weights)
        assert self.score_error > 2.0 ** -4 or np.linalg.norm(err) <= 2.0 ** -7 * np.linalg.norm(y) + 1e-30

    def check(self, capi, device, error=(0, 0), **k):
        out = self.run(capi, device, **k)
        torch.cuda.synchronize()
        code, detail = capi.device_error()
        assert code == error[0] and (code == 0 or error[1] is None or detail == error[1])
        self.compare(out)
        return out

"""Inputs of the sliding-window tests: pools in which every slot that no query
row of its sequence sees holds NaN and every page without a visible key is
freed (its block_table entry is garbage), the oracle's result and a tolerance.

Tolerance, per output element, with A = sum_j w_j |v_j| / sum_j w_j (the
oracle's attention over |V|): the output's rounding to bf16 is off by at most
2^-8 |y|; the weights of a PV product are rounded to bf16 (e4m3 pools: f16), at
most 2^-8 (2^-11) each, so their sum over the row by that times A; f16 weights
below 2^-14 have steps of 2^-24, half of that per key, relative to a weight sum
of at least 1: 2^-25 sum_j |v_j|; fp32 products, sums and the exponential are
covered by 2^-12 A (scores of a few units, sums over a few hundred dims and a
few thousand keys)."""
from __future__ import annotations

import numpy as np
import torch

import oracle
from _parity import bits, to_f64

GARBAGE = (-1, 1 << 29)


class Case:
    def __init__(self, new, cached, window, sinks, hq=8, hkv=2, d=64, ps=16, dtype="bf16", seed=0, scale=None,
                 k_scale=0.02, v_scale=0.03, poison=float("nan")):
        rng = np.random.default_rng(seed)
        self.window, self.sinks, self.dtype, self.ps = window, sinks, dtype, ps
        self.n = np.asarray(new, dtype=np.int64)
        # a sequence's keys: those cached and the new ones, never below 0 (rows without a key)
        self.lens = np.maximum(np.asarray(cached, dtype=np.int64) + self.n, 0).astype(np.int32)
        B = len(self.lens)
        self.qsl = np.concatenate([[0], np.cumsum(self.n)]).astype(np.int32)
        mb = max(1, int((self.lens.max(initial=0) + ps - 1) // ps))
        seen = np.zeros((B, mb * ps), dtype=bool)          # keys that a row of the sequence attends to
        for b in range(B):
            for i in range(self.n[b]):
                seen[b, oracle.visible_keys(int(self.lens[b] - self.n[b] + i), window, sinks)] = True
        live = seen.reshape(B, mb, ps).any(axis=2)
        P = int(live.sum()) + 5
        ids = iter(rng.permutation(P))
        self.table = np.empty((B, mb), dtype=np.int32)
        dead = np.ones((P, ps), dtype=bool)
        for b in range(B):
            for m in range(mb):
                self.table[b, m] = next(ids) if live[b, m] else GARBAGE[(b + m) % 2]
                if live[b, m]:
                    dead[self.table[b, m]] = ~seen[b].reshape(mb, ps)[m]
        g = torch.Generator().manual_seed(seed)
        self.scale = d ** -0.5 if scale is None else scale
        self.k_scale, self.v_scale = (k_scale, v_scale) if dtype == "e4m3" else (1.0, 1.0)
        pools = []
        for s in (self.k_scale, self.v_scale):
            x = torch.randn(P, ps, hkv, d, generator=g)
            x[torch.from_numpy(dead)] = poison
            if dtype == "e4m3":
                x = (x / s).clamp(-448, 448).to(torch.float8_e4m3fn)
            else:
                x = x.to(torch.bfloat16 if dtype == "bf16" else torch.float32)
            pools.append(x)
        self.kp, self.vp = pools
        rows = B if self.is_decode else int(self.n.sum())
        self.q = torch.randn(rows, hq, d, generator=g).to(torch.float32 if dtype == "f32" else torch.bfloat16)

    @property
    def is_decode(self):
        return bool((self.n <= 1).all())

    def oracle(self):
        if self.dtype == "e4m3":
            K = oracle.kv_fp8.dequantize(bits(self.kp), self.k_scale)
            V = oracle.kv_fp8.dequantize(bits(self.vp), self.v_scale)
        else:
            K, V = to_f64(bits(self.kp)), to_f64(bits(self.vp))
        q = to_f64(bits(self.q))
        if self.is_decode:
            f = lambda v: oracle.paged_attention_decode_window(K, v, q, self.table, self.lens, self.scale, self.window,
                                                               self.sinks)
        else:
            f = lambda v: oracle.paged_attention_prefill_window(K, v, q, self.qsl, self.table, self.lens, self.scale,
                                                                self.window, self.sinks)
        y, A = f(V), f(np.abs(V))
        if self.dtype == "f32":
            return y, 1e-5 * (1 + A)
        w = 2.0 ** -8 if self.dtype == "bf16" else 2.0 ** -11
        small = 2.0 ** -25 * int(self.lens.max()) * 4 if self.dtype == "e4m3" else 0.0   # |v| of a few units
        return y, 2.0 ** -8 * np.abs(y) + (w + 2.0 ** -12) * A + small

    def run(self, capi, device, **k):
        dev = lambda a: torch.from_numpy(np.ascontiguousarray(a)).to(device)
        kp, vp, q = self.kp.to(device), self.vp.to(device), self.q.to(device)
        self.args = (kp, vp, q)
        msl = k.pop("max_seq_len", max(1, int(self.lens.max())))
        common = dict(max_seq_len=msl, k_scale=self.k_scale, v_scale=self.v_scale, **k)
        if "out" not in common:
            common["out"] = torch.full_like(q, float("nan"))
        if self.is_decode:
            return capi.paged_attention_decode_window(kp, vp, q, dev(self.table), dev(self.lens), self.scale,
                                                      self.window, self.sinks, **common)
        return capi.paged_attention_prefill_window(kp, vp, q, dev(self.qsl), dev(self.table), dev(self.lens),
                                                   self.scale, int(self.n.max()), self.window, self.sinks, **common)

    def check(self, capi, device, **k):
        out = self.run(capi, device, **k)
        torch.cuda.synchronize()
        assert capi.device_error() == (0, 0)
        got = to_f64(bits(out))
        y, tol = self.oracle()
        assert np.isfinite(got).all()
        err = np.abs(got - y)
        assert (err <= tol).all(), f"error {err.max():.3e}, {(err / np.maximum(tol, 1e-30)).max():.2f} of the tolerance"
        return out

"""The calls of a sliding-window layer together, as a serving loop makes them:
norm-rotate-append and prefill of a first chunk, decode steps with pages freed
behind the window, a fork (shared pages and a copied one), eviction by compaction
and decode after it -- on two layers, without a synchronisation between the
calls.  Every output is compared with the oracle on the pools as they stand, and
the whole run with one that synchronises after every call, bit for bit."""
import numpy as np
import pytest
import torch

import oracle
from serving_slot_mapping_gb300 import build as build_mod
from serving_slot_mapping_gb300 import capi

from _parity import bits, to_f64

pytestmark = pytest.mark.gpu

HQ, HKV, D, PS, WINDOW, SINKS, SCALE = 8, 2, 64, 16, 40, 3, 0.125
LAYERS, PAGES, MB = 2, 48, 16


@pytest.fixture(scope="module", autouse=True)
def _lib(cuda_device):
    build_mod.build()
    capi.lib()
    capi.device_error()  # clear


class Run:
    def __init__(self, device, sync, dtype):
        self.device, self.sync = device, sync
        self.gen = torch.Generator(device=device).manual_seed(5)
        self.row = torch.bfloat16
        self.scales = 0.02 if dtype == "e4m3" else 1.0
        pool = lambda: torch.randn(PAGES, PS, HKV, D, generator=self.gen, device=device)
        t = torch.float8_e4m3fn if dtype == "e4m3" else torch.bfloat16
        self.layers = [(pool().to(t), pool().to(t)) for _ in range(LAYERS)]
        self.pools = capi.make_pools(self.layers)
        self.weights = [torch.randn(2, D, generator=self.gen, device=device).to(self.row) for _ in range(LAYERS)]
        self.table_cs = torch.from_numpy(oracle.rope_table(600, D).astype(np.float32)).to(device)
        rng = np.random.default_rng(1)
        self.free = list(rng.permutation(PAGES))
        self.tables, self.lens, self.log = [], [], []

    def step(self):
        if self.sync:
            torch.cuda.synchronize()

    def dev(self, a, dtype=np.int32):
        return torch.from_numpy(np.ascontiguousarray(a, dtype=dtype)).to(self.device)

    def grow(self, b, n):
        """Pages for n more tokens of sequence b; their slots and positions."""
        slots, pos = [], []
        for p in range(self.lens[b], self.lens[b] + n):
            if p % PS == 0:
                self.tables[b][p // PS] = self.free.pop()
            slots.append(self.tables[b][p // PS] * PS + p % PS)
            pos.append(p)
        self.lens[b] += n
        return slots, pos

    def forward(self, new):
        """One pass of the layers over `new[b]` tokens of every sequence."""
        slots, pos = [], []
        for b, n in enumerate(new):
            s, p = self.grow(b, n)
            slots += s
            pos += p
        T = len(slots)
        table, lens = self.dev(self.tables), self.dev(self.lens)
        slots, pos = self.dev(slots, np.int64), self.dev(pos)
        qsl = self.dev(np.concatenate([[0], np.cumsum(new)]))
        for i, (kp, vp) in enumerate(self.layers):
            qkv = torch.randn(T, HQ + 2 * HKV, D, generator=self.gen, device=self.device).to(self.row)
            q = capi.paged_qk_norm_rope_append(kp, vp, qkv[:, :HQ], qkv[:, HQ:HQ + HKV], qkv[:, HQ + HKV:], slots, pos,
                                               self.table_cs, q_weight=self.weights[i][0], k_weight=self.weights[i][1],
                                               k_scale=self.scales, v_scale=self.scales)
            self.step()
            common = dict(max_seq_len=MB * PS, k_scale=self.scales, v_scale=self.scales)
            if max(new) == 1:
                out = capi.paged_attention_decode_window(kp, vp, q, table, lens, SCALE, WINDOW, SINKS, **common)
            else:
                out = capi.paged_attention_prefill_window(kp, vp, q, qsl, table, lens, SCALE, max(new), WINDOW, SINKS,
                                                          **common)
            self.step()
            self.log += [q, out]
            if self.sync:
                self.check(kp, vp, q, out, qsl.cpu().numpy(), table.cpu().numpy(), lens.cpu().numpy())

    def values(self, pool):
        if pool.dtype == torch.float8_e4m3fn:
            return oracle.kv_fp8.dequantize(bits(pool), self.scales)
        return to_f64(bits(pool))

    def check(self, kp, vp, q, out, qsl, table, lens):
        K, V, qf = self.values(kp), self.values(vp), to_f64(bits(q))
        f = lambda v: oracle.paged_attention_prefill_window(K, v, qf, qsl, table, lens, SCALE, WINDOW, SINKS)
        y, A = f(V), f(np.abs(V))
        # output and weights rounded to 8 bits each, fp32 sums (_window.py)
        assert (np.abs(to_f64(bits(out)) - y) <= 2.0 ** -8 * np.abs(y) + (2.0 ** -8 + 2.0 ** -12) * A).all()

    def free_behind(self, b):
        """Free the pages that no later token of sequence b sees; their slots hold anything."""
        for m in range(MB):
            if self.tables[b][m] >= 0 and m * PS >= SINKS and (m + 1) * PS <= self.lens[b] + 1 - WINDOW:
                for kp, vp in self.layers:
                    for pool in (kp, vp):
                        pool.view(torch.uint8)[int(self.tables[b][m])] = 255   # NaN in either type
                self.tables[b][m] = -1

    def fork(self, b):
        """A new sequence that shares b's full pages and copies the last, partial one."""
        last = self.lens[b] // PS
        row = list(self.tables[b])
        row[last] = self.free.pop()
        capi.paged_kv_copy_pages(self.pools, self.dev([self.tables[b][last]]), self.dev([row[last]]))
        self.step()
        self.tables.append(row)
        self.lens.append(self.lens[b])

    def evict(self, b, keep):
        base = [n for n in self.lens]
        base[b] = SINKS
        counts = np.zeros(len(self.lens) + 1, dtype=np.int64)
        counts[b + 1:] = len(keep)
        new = capi.paged_kv_compact(self.pools, self.dev(self.tables), self.dev(self.lens), self.dev(counts),
                                    self.dev(keep), base=self.dev(base))
        self.step()
        self.log.append(new)
        self.lens[b] = SINKS + len(keep)
        return new

    def all(self):
        for n in (50, 9, 100):
            self.tables.append([-1] * MB)
            self.lens.append(0)
        self.forward([50, 9, 100])
        for _ in range(9):
            self.forward([1, 1, 1])
        self.free_behind(2)
        self.forward([30, 5, 20])
        self.free_behind(2)
        for _ in range(3):
            self.forward([1, 1, 1])
        # sequence 0 is 92 tokens: a partial last page
        self.fork(0)
        self.forward([1, 1, 1, 1])
        # evict from sequence 1 (27 tokens, all its pages its own)
        new = self.evict(1, np.array([4, 5, 9, 17, 18, 19, 20, 25], dtype=np.int32))
        for _ in range(3):
            self.forward([1, 1, 1, 1])
        # the lengths written by the call are those a next call may use at once
        q = self.log[-2]
        lens2 = new + 3
        lens2[3] += 0
        self.log.append(capi.paged_attention_decode_window(*self.layers[1], q, self.dev(self.tables), lens2, SCALE, WINDOW,
                                                           SINKS, max_seq_len=MB * PS, k_scale=self.scales,
                                                           v_scale=self.scales))
        torch.cuda.synchronize()
        return self.log + [t for pair in self.layers for t in pair]


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
def test_serving_loop(cuda_device, dtype):
    runs = [Run(cuda_device, sync, dtype).all() for sync in (True, False, False)]
    assert capi.device_error() == (0, 0)
    for other in runs[1:]:
        assert len(other) == len(runs[0])
        for a, b in zip(runs[0], other):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
    # the last call repeats the step before it with lengths taken from the compaction
    assert torch.equal(runs[0][-2 * LAYERS - 1].view(torch.int16), runs[0][-2 * LAYERS - 2].view(torch.int16))

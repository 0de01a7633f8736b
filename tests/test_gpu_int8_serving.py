"""The operators of a long-context cache used together, as a serving loop does: prompts
into an int8 cache, decode steps that add up the attention weights of their keys,
eviction by page when a sequence is over its budget; and the same over a bf16 cache with
eviction by row.  Every output is compared with the oracle fed with what the pools hold."""
import numpy as np
import pytest
import torch

import oracle
from serving_slot_mapping_gb300 import build as build_mod
from serving_slot_mapping_gb300 import capi

from _parity import bits, to_f64

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib(cuda_device):
    build_mod.build()
    capi.lib()
    capi.device_error()  # clear


def close(out, y, K, q, scale):
    """Tolerance: bf16 output, f16 weights (2^-8 + 2^-11 of values of a few units), and a
    prefill's f16 keys (2^-10 of a score's sum of magnitudes)."""
    e = np.expm1(2 * 2.0 ** -10 * scale * np.abs(q).max() * np.abs(K).sum(-1).max())
    v = np.abs(y).max() + 4
    assert np.abs(to_f64(bits(out)) - y).max() <= (2.0 ** -8 + 2.0 ** -9 + e) * v


class Loop:
    def __init__(self, device, prompts, ps=16, hq=8, hkv=2, d=64, P=200, seed=0):
        self.dev, self.ps, self.hq, self.hkv, self.d, self.scale = device, ps, hq, hkv, d, d ** -0.5
        self.rng = np.random.default_rng(seed)
        self.g = torch.Generator().manual_seed(seed)
        self.lens = np.asarray(prompts, dtype=np.int32)
        self.B, self.mb = len(prompts), 16
        self.free = self.rng.permutation(P).tolist()
        self.table = np.full((self.B, self.mb), -1, dtype=np.int32)
        self.P = P
        self.mass = torch.zeros(self.B, self.mb * ps, device=device)

    def rows(self, n, heads):
        return torch.randn(n, heads, self.d, generator=self.g).to(torch.bfloat16).to(self.dev)

    def grow(self, b):
        """Pages for sequence b's length; the slots of its positions."""
        for m in range(-(-int(self.lens[b]) // self.ps)):
            if self.table[b, m] < 0:
                self.table[b, m] = self.free.pop()

    def slot(self, b, j):
        return int(self.table[b, j // self.ps]) * self.ps + j % self.ps

    def t(self, a, dtype=np.int32):
        return torch.from_numpy(np.ascontiguousarray(a, dtype=dtype)).to(self.dev)


def test_int8_cache_with_page_eviction(cuda_device):
    L = Loop(cuda_device, [40, 97, 1, 150])
    kp, vp = (torch.randint(-128, 128, (L.P, L.ps, L.hkv, L.d), device=cuda_device, dtype=torch.int8) for _ in range(2))
    ks, vs = (torch.full((L.P, 1, L.hkv), float("nan"), device=cuda_device) for _ in range(2))
    values = lambda: [oracle.kv_int8.dequantize(x.cpu().numpy(), s.cpu().numpy()) for x, s in ((kp, ks), (vp, vs))]
    # prompts, in two chunks each
    done = np.zeros(L.B, dtype=np.int32)
    full = L.lens.copy()
    for part in ((full + 1) // 2, full - (full + 1) // 2):
        L.lens = done + part
        for b in range(L.B):
            L.grow(b)
        slots = [L.slot(b, j) for b in range(L.B) for j in range(done[b], L.lens[b])]
        key, value, q = L.rows(len(slots), L.hkv), L.rows(len(slots), L.hkv), L.rows(len(slots), L.hq)
        capi.paged_kv_append_int8(kp, vp, ks, vs, key, value, L.t(slots, np.int64))
        qsl = np.concatenate([[0], np.cumsum(part)])
        out = capi.paged_attention_prefill_int8(kp, vp, ks, vs, q, L.t(qsl), L.t(L.table), L.t(L.lens), L.scale,
                                                int(part.max()))
        torch.cuda.synchronize()
        K, V = values()
        close(out, oracle.paged_attention_prefill(K, V, to_f64(bits(q)), qsl, L.table, L.lens, L.scale), K, to_f64(bits(q)),
              L.scale)
        done = L.lens.copy()
    ws = capi.decode_mass_workspace(L.B, L.hq, kp, L.mb * L.ps)
    want = np.zeros((L.B, L.mb * L.ps))
    for step in range(12):
        L.lens = L.lens + 1
        for b in range(L.B):
            L.grow(b)
        key, value, q = L.rows(L.B, L.hkv), L.rows(L.B, L.hkv), L.rows(L.B, L.hq)
        capi.paged_kv_append_int8(kp, vp, ks, vs, key, value, L.t([L.slot(b, L.lens[b] - 1) for b in range(L.B)], np.int64))
        bt, sl = L.t(L.table), L.t(L.lens)
        out = capi.paged_attention_decode_mass(kp, vp, q, bt, sl, L.scale, L.mass, mass_in=L.mass, workspace=ws,
                                               key_scales=ks, value_scales=vs)
        assert torch.equal(out, capi.paged_attention_decode_int8(kp, vp, ks, vs, q, bt, sl, L.scale))
        K, V = values()
        close(out, oracle.paged_attention_decode(K, V, to_f64(bits(q)), L.table, L.lens, L.scale), K, to_f64(bits(q)), L.scale)
        for b, w in enumerate(oracle.evict.key_weights(K, to_f64(bits(q)), L.table, L.lens, L.scale)):
            want[b, :len(w)] += w
        assert np.abs(L.mass.cpu().numpy() - want).max() < 1e-4 * L.hq
        if step % 4 == 3:        # at most 6 pages a sequence
            nbt, nsl, mass = capi.paged_kv_evict_pages(L.mass, bt, sl, L.ps, 6, 4, 20)
            picked = oracle.evict.evict_pages(L.mass.cpu().numpy(), L.lens, L.ps, 6, 4, 20)
            nbt, nsl = nbt.cpu().numpy(), nsl.cpu().numpy()
            for b, (stay, go) in enumerate(picked):
                assert nbt[b, :len(stay)].tolist() == L.table[b, stay].tolist()
                old = len(stay) + len(go)
                kept = -(-int(nsl[b]) // L.ps)
                L.free += nbt[b, kept:old].tolist()
                nbt[b, kept:] = -1
                rows = [p * L.ps + i for p in stay for i in range(L.ps) if p * L.ps + i < L.lens[b]]
                want[b] = np.concatenate([want[b, rows], np.zeros(want.shape[1] - len(rows))])
            L.table, L.lens, L.mass = nbt.copy(), nsl.copy(), mass
            assert (L.lens <= 6 * L.ps).all()
    assert capi.device_error() == (0, 0)


def test_bf16_cache_with_row_eviction(cuda_device):
    L = Loop(cuda_device, [60, 33, 120], seed=1)
    layers = [tuple(torch.randn(L.P, L.ps, L.hkv, L.d, device=cuda_device).bfloat16() for _ in range(2)) for _ in range(2)]
    for b in range(L.B):
        L.grow(b)
    for step in range(6):
        L.lens = L.lens + 1
        for b in range(L.B):
            L.grow(b)
        bt, sl = L.t(L.table), L.t(L.lens)
        for kp, vp in layers:     # one mass for the layers that share the block table
            key, value, q = L.rows(L.B, L.hkv), L.rows(L.B, L.hkv), L.rows(L.B, L.hq)
            capi.paged_kv_append(kp, vp, key, value, L.t([L.slot(b, L.lens[b] - 1) for b in range(L.B)], np.int64))
            out = capi.paged_attention_decode_mass(kp, vp, q, bt, sl, L.scale, L.mass, mass_in=L.mass, decay=0.9)
            assert torch.equal(out, capi.paged_attention_decode(kp, vp, q, bt, sl, L.scale))
        if step % 3 == 2:
            before = [(to_f64(bits(k)), to_f64(bits(v))) for k, v in layers]
            m = L.mass.cpu().numpy()
            ptr, keep, base, L.mass = capi.paged_kv_evict_rows(L.mass, sl, 48, 4, 16)
            new = capi.paged_kv_compact(layers, bt, sl, ptr, keep, base=base)
            picked = oracle.evict.evict_rows(m, L.lens, 48, 4, 16)
            torch.cuda.synchronize()
            for b, (bs, kept) in enumerate(picked):
                rows = list(range(bs)) + kept
                assert int(new[b]) == len(rows)
                assert np.array_equal(L.mass[b].cpu().numpy(), oracle.evict.moved(m[b], rows, m.shape[1]))
                for (k, v), (ok, ov) in zip(layers, before):
                    k, v = to_f64(bits(k)).reshape(-1, L.hkv, L.d), to_f64(bits(v)).reshape(-1, L.hkv, L.d)
                    to, frm = [L.slot(b, i) for i in range(len(rows))], [L.slot(b, j) for j in rows]
                    assert np.array_equal(k[to], ok.reshape(k.shape)[frm]) and np.array_equal(v[to], ov.reshape(v.shape)[frm])
            L.lens = new.cpu().numpy()
            assert (L.lens <= 48).all()
    assert capi.device_error() == (0, 0)


def test_a_fork_of_an_int8_cache(cuda_device):
    """Pages and their scales copied by the same call, the scales as an f32 pool."""
    ps, blk = 64, 16
    kp, vp = (torch.randint(-128, 128, (20, ps, 2, 64), device=cuda_device, dtype=torch.int8) for _ in range(2))
    ks, vs = (torch.rand(20, ps // blk, 2, device=cuda_device) for _ in range(2))
    src, dst = (torch.tensor(x, dtype=torch.int32, device=cuda_device) for x in ([3, 7], [11, 12]))
    want = [x.clone() for x in (kp, vp, ks, vs)]
    for x in want:
        x[dst.long()] = x[src.long()]
    capi.paged_kv_copy_pages([(kp, vp)], src, dst)
    capi.paged_kv_copy_pages([(ks.unsqueeze(-1), vs.unsqueeze(-1))], src, dst)
    for x, y in zip((kp, vp, ks, vs), want):
        assert torch.equal(x, y)
    assert capi.device_error() == (0, 0)


def test_pages_past_2_31_codes(cuda_device):
    """A pool of more than 2^31 codes a tensor: its last pages."""
    P, ps, hkv, d = 140000, 16, 8, 128
    kp, vp = (torch.empty(P, ps, hkv, d, device=cuda_device, dtype=torch.int8) for _ in range(2))
    ks, vs = (torch.empty(P, 1, hkv, device=cuda_device) for _ in range(2))
    pages = [P - 1, 3, P - 2]
    table = torch.tensor([pages], dtype=torch.int32, device=cuda_device)
    lens = torch.tensor([40], dtype=torch.int32, device=cuda_device)
    slots = torch.tensor([pages[j // ps] * ps + j % ps for j in range(40)], device=cuda_device)
    g = torch.Generator().manual_seed(2)
    key, value, q = (torch.randn(n, h, d, generator=g).bfloat16().to(cuda_device) for n, h in ((40, hkv), (40, hkv), (40, 32)))
    small = [torch.empty(3, ps, hkv, d, device=cuda_device, dtype=torch.int8) for _ in range(2)] + \
        [torch.empty(3, 1, hkv, device=cuda_device) for _ in range(2)]
    near = torch.tensor([[0, 1, 2]], dtype=torch.int32, device=cuda_device)
    capi.paged_kv_append_int8(kp, vp, ks, vs, key, value, slots)
    capi.paged_kv_append_int8(*small, key, value, torch.arange(40, device=cuda_device))
    for i, p in enumerate(pages):
        n = min(ps, 40 - ps * i)
        assert torch.equal(kp[p, :n], small[0][i, :n]) and torch.equal(vs[p], small[3][i])
    qsl = torch.tensor([0, 40], dtype=torch.int32, device=cuda_device)
    m, m2 = torch.zeros(1, 48, device=cuda_device), torch.zeros(1, 48, device=cuda_device)
    assert torch.equal(capi.paged_attention_decode_int8(kp, vp, ks, vs, q[:1], table, lens, 0.1),
                       capi.paged_attention_decode_int8(*small, q[:1], near, lens, 0.1))
    assert torch.equal(capi.paged_attention_prefill_int8(kp, vp, ks, vs, q, qsl, table, lens, 0.1, 40),
                       capi.paged_attention_prefill_int8(*small, q, qsl, near, lens, 0.1, 40))
    a = capi.paged_attention_decode_mass(kp, vp, q[:1], table, lens, 0.1, m, key_scales=ks, value_scales=vs)
    b = capi.paged_attention_decode_mass(small[0], small[1], q[:1], near, lens, 0.1, m2, key_scales=small[2],
                                         value_scales=small[3])
    assert torch.equal(a, b) and torch.equal(m, m2)
    assert capi.device_error() == (0, 0)

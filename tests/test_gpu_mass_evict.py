"""Attention weights of cached keys and eviction by them, against the oracle."""
import numpy as np
import pytest
import torch

import oracle
from serving_slot_mapping_gb300 import build as build_mod
from serving_slot_mapping_gb300 import capi

from _int8 import Case
from _parity import bits, to_f64

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib(cuda_device):
    build_mod.build()
    capi.lib()
    capi.device_error()  # clear


def decode(lens, **k):
    lens = np.asarray(lens)
    return Case(np.ones_like(lens), lens - 1, **k)


RAGGED = [1, 15, 16, 17, 0, 33, 64, 129, 500, 31]


def run_mass(c, device, mass_in=None, decay=1.0, stride=None, **k):
    kp, vp, ks, vs, q, bt, L, _ = c.tensors(device)
    msl = c.max_len
    B = len(c.lens)
    store = torch.full((B, stride or msl + 3), -7.0, device=device)
    m = store[:, :msl + 1] if stride else store
    out = capi.paged_attention_decode_mass(kp, vp, q, bt, L, c.scale, m, mass_in=mass_in, decay=decay,
                                           max_seq_len=k.pop("max_seq_len", msl), k_scale=c.k_scale, v_scale=c.v_scale,
                                           key_scales=ks, value_scales=vs, **k)
    torch.cuda.synchronize()
    return out, m


def check_mass(c, device, before=None, decay=1.0, **k):
    """A weight's error: its score's, from fp32 sums of d products (at most (d + 4) 2^-24
    sum_d |q_d K_d| scale; e below, on the weight and on its row's sum), the exponential's
    and the sums' (2^-20, far above both), relative to the weight; e4m3 and int8 pools
    round q to f16, which is exact here."""
    out, m = run_mass(c, device, decay=decay, **k)
    assert capi.device_error() == (0, 0)
    c.compare(out)
    K, _ = c.values()
    q = to_f64(bits(c.q))
    want = oracle.evict.key_weights(K, q, c.seen, c.lens, c.scale)
    got = m.cpu().numpy()
    for b, L in enumerate(c.lens.tolist()):
        e = 2 * (c.d + 4) * 2.0 ** -24 * abs(c.scale) * np.abs(q[b]).sum(-1).max() * np.abs(K).max() + 2.0 ** -20
        w = want[b] + (0.0 if before is None else decay * before[b, :L].astype(np.float64))
        assert (np.abs(got[b, :L] - w) <= e * want[b] + 2.0 ** -22 * np.abs(w)).all()
        assert (got[b, L:] == -7.0).all()     # behind the sequence nothing is written
        if L and before is None:
            assert abs(got[b, :L].sum() - q.shape[1]) <= 1e-4 * q.shape[1]
    return out, m


@pytest.mark.parametrize("dtype", ["bf16", "e4m3", "int8"])
@pytest.mark.parametrize("hq,hkv,d", [(1, 1, 64), (8, 2, 64), (32, 8, 128), (12, 3, 128), (32, 1, 128), (16, 16, 64), (64, 2, 64)])
def test_mass_head_layouts(cuda_device, dtype, hq, hkv, d):
    check_mass(decode(RAGGED, hq=hq, hkv=hkv, d=d, dtype=dtype, seed=hq), cuda_device)
    if dtype == "int8":   # the kernel for long contexts too
        check_mass(decode(RAGGED, hq=hq, hkv=hkv, d=d, dtype=dtype, seed=hq, room=2400), cuda_device)


@pytest.mark.parametrize("dtype,ps,blk", [("bf16", 8, 8), ("bf16", 64, 64), ("e4m3", 8, 8), ("e4m3", 32, 32), ("int8", 64, 32)])
def test_mass_page_sizes(cuda_device, dtype, ps, blk):
    check_mass(decode(RAGGED + [1500], ps=ps, blk=blk, dtype=dtype, seed=ps), cuda_device)


@pytest.mark.parametrize("lens", [[1], [4096], [1] * 40, [5000, 3, 700], [0, 0], list(range(1, 300, 5))])
@pytest.mark.parametrize("dtype", ["bf16", "int8"])
def test_mass_batches(cuda_device, lens, dtype):
    check_mass(decode(lens, hq=32, hkv=8, d=128, dtype=dtype, seed=len(lens)), cuda_device)
    if dtype == "int8":
        check_mass(decode(lens, hq=32, hkv=8, d=128, dtype=dtype, seed=len(lens), room=2400), cuda_device)


def test_mass_of_steps_before(cuda_device):
    c = decode([40, 7, 300], dtype="bf16")
    before = torch.rand(3, 400, device=cuda_device)
    for decay in (1.0, 0.5, 0.0, -1.0):
        check_mass(c, cuda_device, before=before.cpu().numpy(), decay=decay, mass_in=before[:, :301], stride=400)
    nan = torch.full((3, 400), float("nan"), device=cuda_device)
    check_mass(c, cuda_device, before=np.zeros((3, 400)), decay=0.0, mass_in=nan[:, :301], stride=400)
    # in place, twice
    m = torch.zeros(3, 300, device=cuda_device)
    kp, vp, ks, vs, q, bt, L, _ = c.tensors(cuda_device)
    for _ in range(2):
        capi.paged_attention_decode_mass(kp, vp, q, bt, L, c.scale, m, mass_in=m, max_seq_len=300)
    once = torch.zeros(3, 300, device=cuda_device)
    capi.paged_attention_decode_mass(kp, vp, q, bt, L, c.scale, once, max_seq_len=300)
    assert torch.equal(m, 2 * once)


def test_mass_rows_of_one_sequence_and_two_widths(cuda_device):
    """One sequence has no row stride: the masses before may lie in a wider tensor."""
    c = decode([40], dtype="bf16")
    kp, vp, ks, vs, q, bt, L, _ = c.tensors(cuda_device)
    before = torch.rand(1, 53, device=cuda_device)
    got, once = torch.zeros(1, 41, device=cuda_device), torch.zeros(1, 53, device=cuda_device)
    capi.paged_attention_decode_mass(kp, vp, q, bt, L, c.scale, got, mass_in=before, max_seq_len=40)
    capi.paged_attention_decode_mass(kp, vp, q, bt, L, c.scale, once, mass_in=before, max_seq_len=40)
    assert torch.equal(got[:, :40], once[:, :40]) and float(got[0, 40]) == 0


def test_mass_is_that_of_the_plain_decode(cuda_device):
    """The attention beside it is bit for bit that of the plain call."""
    for room in (0, 2400):
        c = decode([300, 41, 900], hq=32, hkv=8, d=128, dtype="int8", room=room)
        out, _ = check_mass(c, cuda_device)
        assert torch.equal(out, c.run(capi, cuda_device))


def test_a_sequence_past_max_seq_len_is_cut_to_it(cuda_device):
    c = decode([30, 100], dtype="bf16")
    kp, vp, ks, vs, q, bt, L, _ = c.tensors(cuda_device)
    m = torch.full((2, 80), -7.0, device=cuda_device)
    out = capi.paged_attention_decode_mass(kp, vp, q, bt, L, c.scale, m, max_seq_len=70)
    torch.cuda.synchronize()
    assert capi.device_error()[0] == 3
    want = capi.paged_attention_decode(kp, vp, q, bt, L.clamp(max=70), c.scale, max_seq_len=70)
    assert torch.equal(out, want) and (m[:, 70:] == -7.0).all() and abs(float(m[1, :70].sum()) - 8) < 1e-3


def test_mass_skips_keys_of_bad_pages_int8(cuda_device):
    for room in (0, 2400):
        c = decode([100, 75], bad=[(0, 2)], room=room)
        out, m = run_mass(c, cuda_device)
        assert capi.device_error()[0] == 1
        c.compare(out)
        assert (m[0, 32:48] == 0).all() and abs(float(m[0, :100].sum()) - 8) < 1e-3


# ---- eviction --------------------------------------------------------------------

def masses(B, width, seed, ties=0.2, odd=False):
    rng = np.random.default_rng(seed)
    m = rng.exponential(size=(B, width)).astype(np.float32)
    m[rng.random((B, width)) < ties] = 0.0
    m[rng.random((B, width)) < ties / 2] = -0.0
    if odd:
        for v in (np.nan, np.inf, -np.inf, 1e-42, 2.5, 2.5):
            m[rng.random((B, width)) < 0.05] = v
    return m


def check_rows(device, mass, lens, budget, sinks, recent, stride=None, **k):
    B, width = mass.shape
    store = torch.zeros((B, stride or width), device=device)
    store[:, :width] = torch.from_numpy(mass).to(device)
    L = torch.tensor(lens, dtype=torch.int32, device=device)
    ptr, keep, base, new = capi.paged_kv_evict_rows(store[:, :width], L, budget, sinks, recent, **k)
    torch.cuda.synchronize()
    assert capi.device_error() == (0, 0)
    want = oracle.evict.evict_rows(mass, lens, budget, sinks, recent)
    ptr, keep = ptr.tolist(), keep.cpu().numpy()
    assert ptr[0] == 0 and base.tolist() == [b for b, _ in want]
    for b, (bs, kept) in enumerate(want):
        assert keep[ptr[b]:ptr[b + 1]].tolist() == kept
        exp = oracle.evict.moved(mass[b], list(range(bs)) + kept, width)
        assert np.array_equal(new[b].cpu().numpy(), exp, equal_nan=True)


def check_pages(device, mass, lens, ps, budget, sinks, recent, extra=0, **k):
    B, width = mass.shape
    mb = max(1, -(-width // ps)) + extra
    table = np.random.default_rng(B).permutation(B * mb).reshape(B, mb).astype(np.int32)
    L = torch.tensor(lens, dtype=torch.int32, device=device)
    bt, nl, new = capi.paged_kv_evict_pages(torch.from_numpy(mass).to(device), torch.from_numpy(table).to(device), L, ps,
                                            budget, sinks, recent, **k)
    torch.cuda.synchronize()
    assert capi.device_error() == (0, 0)
    for b, (stay, go) in enumerate(oracle.evict.evict_pages(mass, lens, ps, budget, sinks, recent)):
        n = len(stay) + len(go)
        assert bt[b].tolist() == table[b, stay + go].tolist() + table[b, n:].tolist()
        assert int(nl[b]) == lens[b] - ps * len(go)
        rows = [p * ps + i for p in stay for i in range(ps) if p * ps + i < lens[b]]
        assert np.array_equal(new[b].cpu().numpy(), oracle.evict.moved(mass[b], rows, width), equal_nan=True)


LENS = [0, 1, 99, 100, 101, 500, 333, 128]


@pytest.mark.parametrize("budget,sinks,recent", [(100, 4, 32), (100, 0, 0), (100, 0, 100), (100, 100, 0), (1, 0, 0),
                                                 (1, 0, 1), (0, 0, 0), (499, 3, 5), (500, 1, 1), (600, 0, 0)])
@pytest.mark.parametrize("odd", [False, True])
def test_evict_rows(cuda_device, budget, sinks, recent, odd):
    check_rows(cuda_device, masses(8, 500, budget, odd=odd), LENS, budget, sinks, recent, stride=517)


def test_evict_rows_all_equal(cuda_device):
    for v in (0.0, 1.5, float("nan")):
        check_rows(cuda_device, np.full((8, 500), v, dtype=np.float32), LENS, 77, 3, 9)


@pytest.mark.parametrize("B,width", [(1, 1), (1, 9000), (2, 70001), (3, 20000), (1, 400000), (200, 300)])
def test_evict_rows_sizes(cuda_device, B, width):
    """From one row to those that a cluster shares, and past what fits in shared memory."""
    rng = np.random.default_rng(width)
    lens = [width] + rng.integers(0, width + 1, size=B - 1).tolist()
    for budget in {max(1, width // 3), max(1, width - 1)}:
        check_rows(cuda_device, masses(B, width, B, ties=0.4), lens, budget, 0 if budget < 9 else 4, 0 if budget < 9 else 5)


@pytest.mark.parametrize("ps", [1, 2, 8, 16, 32, 64, 256, 1024])
@pytest.mark.parametrize("odd", [False, True])
def test_evict_pages(cuda_device, ps, odd):
    width = 9 * ps + 5
    lens = [0, 1, ps, ps + 1, 5 * ps, 5 * ps + 1, 9 * ps - 1 if ps > 1 else 9, 9 * ps + 3 if ps > 3 else 9]
    check_pages(cuda_device, masses(8, width, ps, odd=odd), lens, ps, 5, 1, 2, extra=3)
    check_pages(cuda_device, masses(8, width, ps + 1), lens, ps, 2, 0, 0)
    # rows that start on 16 bytes: vectors
    check_pages(cuda_device, masses(8, 9 * ps + 8 - ps % 4, ps + 2, odd=odd), lens, ps, 4, 1, 1, extra=1)


@pytest.mark.parametrize("B,pages,ps", [(1, 30000, 4), (2, 9000, 16), (40, 300, 16), (1, 100000, 1)])
def test_evict_pages_sizes(cuda_device, B, pages, ps):
    rng = np.random.default_rng(pages)
    width = pages * ps
    lens = [width - ps // 2] + rng.integers(0, width + 1, size=B - 1).tolist()
    check_pages(cuda_device, masses(B, width, 3, ties=0.5), lens, ps, pages // 3, 4, 3 * ps + 1)


def test_evict_lengths_out_of_range(cuda_device):
    m = torch.rand(2, 64, device=cuda_device)
    L = torch.tensor([70, -3], dtype=torch.int32, device=cuda_device)
    ptr, keep, base, new = capi.paged_kv_evict_rows(m, L, 32, 4, 4)
    torch.cuda.synchronize()
    assert capi.device_error()[0] == 3
    want = oracle.evict.evict_rows(m.cpu().numpy(), [64, 0], 32, 4, 4)
    assert ptr.tolist() == [0, 28, 28] and keep.tolist()[:28] == want[0][1] and base.tolist() == [4, 0]
    bt = torch.arange(8, dtype=torch.int32, device=cuda_device).view(2, 4)
    nbt, nl, _ = capi.paged_kv_evict_pages(m, bt, L, 16, 3, 1, 1)
    torch.cuda.synchronize()
    assert capi.device_error()[0] == 3 and nl.tolist() == [48, 0] and sorted(nbt[0].tolist()) == [0, 1, 2, 3]


def test_evict_replayed_on_other_inputs(cuda_device):
    m, L = torch.empty(3, 300, device=cuda_device), torch.empty(3, dtype=torch.int32, device=cuda_device)
    bt = torch.arange(60, dtype=torch.int32, device=cuda_device).view(3, 20)
    rows = [torch.zeros(4, dtype=torch.int32, device=cuda_device), torch.zeros(300, dtype=torch.int32, device=cuda_device),
            torch.zeros(3, dtype=torch.int32, device=cuda_device), torch.zeros(3, 300, device=cuda_device)]
    pages = [torch.zeros_like(bt), torch.zeros_like(L), torch.zeros(3, 300, device=cuda_device)]
    m.fill_(1.0)
    L.fill_(5)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        capi.paged_kv_evict_rows(m, L, 100, 4, 20, keep_indptr=rows[0], keep=rows[1], base=rows[2], new_mass=rows[3])
        capi.paged_kv_evict_pages(m, bt, L, 16, 7, 4, 20, new_block_table=pages[0], new_seq_lens=pages[1], new_mass=pages[2])
    for seed in range(3):
        m.copy_(torch.from_numpy(masses(3, 300, seed)))
        L.copy_(torch.tensor([300, 17 + seed, 150 + 30 * seed]))
        g.replay()
        torch.cuda.synchronize()
        for got, want in zip(rows, capi.paged_kv_evict_rows(m, L, 100, 4, 20)):
            n = int(rows[0][-1]) if got is rows[1] else None
            assert torch.equal(got[:n], want[:n])
        for got, want in zip(pages, capi.paged_kv_evict_pages(m, bt, L, 16, 7, 4, 20)):
            assert torch.equal(got, want)
    assert capi.device_error() == (0, 0)


def test_evict_of_nothing(cuda_device):
    """No column, or nothing over the budget."""
    L = torch.zeros(2, dtype=torch.int32, device=cuda_device)
    ptr, keep, base, new = capi.paged_kv_evict_rows(torch.empty(2, 0, device=cuda_device), L, 5, 1, 1)
    assert ptr.tolist() == [0, 0, 0] and base.tolist() == [0, 0] and new.shape == (2, 0) and keep.numel() == 0
    check_rows(cuda_device, masses(2, 8, 1), [8, 3], 8, 0, 0)
    check_pages(cuda_device, masses(2, 8, 1), [8, 3], 4, 2, 0, 0)
    assert capi.device_error() == (0, 0)

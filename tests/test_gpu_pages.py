"""paged_kv_copy_pages and paged_kv_compact against the oracle, bit for bit,
over whole pools."""
import numpy as np
import pytest
import torch

import oracle
from serving_slot_mapping_gb300 import build as build_mod
from serving_slot_mapping_gb300 import capi

pytestmark = pytest.mark.gpu

TYPES = {"bf16": torch.bfloat16, "f32": torch.float32, "e4m3": torch.float8_e4m3fn}


@pytest.fixture(scope="module", autouse=True)
def _lib(cuda_device):
    build_mod.build()
    capi.lib()
    capi.device_error()  # clear


def _pools(dev, layers, P, ps, hkv, d, dtype, seed=0):
    """Pools of random bytes (any bit pattern, NaN included)."""
    g = torch.Generator().manual_seed(seed)
    n = P * ps * hkv * d * TYPES[dtype].itemsize
    make = lambda: torch.randint(0, 256, (n,), generator=g, dtype=torch.uint8).to(dev).view(TYPES[dtype]).view(P, ps, hkv, d)
    return [(make(), make()) for _ in range(layers)]


def _bytes(t):
    return t.contiguous().view(torch.uint8).cpu().numpy()


def _dev(a, dev, dtype=np.int32):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=dtype)).to(dev)


@pytest.mark.parametrize("dtype", ["bf16", "f32", "e4m3"])
@pytest.mark.parametrize("layers,P,ps,hkv,d,n", [(1, 3, 16, 8, 128, 1), (5, 40, 16, 8, 128, 20), (3, 70, 8, 1, 64, 35),
                                                 (130, 6, 4, 1, 32, 3), (2, 50, 1, 3, 5, 25), (2, 9, 12, 1, 7, 4),
                                                 (1, 9, 64, 8, 256, 4)])
def test_copy_pages(cuda_device, dtype, layers, P, ps, hkv, d, n):
    pairs = _pools(cuda_device, layers, P, ps, hkv, d, dtype, seed=P)
    rng = np.random.default_rng(P)
    ids = rng.permutation(P)[:2 * n]
    src, dst = ids[:n].copy(), ids[n:].copy()
    if n > 3:
        src[1] = -1                 # padding pairs, a page onto itself, one source twice
        dst[2] = -5
        src[3] = dst[3]
        src[0] = src[n - 1]
    before = [[_bytes(t) for t in p] for p in pairs]
    capi.paged_kv_copy_pages(capi.make_pools(pairs), _dev(src, cuda_device), _dev(dst, cuda_device))
    torch.cuda.synchronize()
    assert capi.device_error() == (0, 0)
    for old, pair in zip(before, pairs):
        for o, t in zip(old, pair):
            assert np.array_equal(_bytes(t), oracle.paged_kv_copy_pages(o, src, dst))


def test_copy_no_pairs_and_bad_pages(cuda_device):
    pairs = _pools(cuda_device, 2, 10, 16, 2, 64, "bf16")
    before = [[_bytes(t) for t in p] for p in pairs]
    none = torch.zeros(0, dtype=torch.int32, device=cuda_device)
    capi.paged_kv_copy_pages(pairs, none, none)
    capi.paged_kv_copy_pages(pairs, _dev([3, 10, 4], cuda_device), _dev([10, 2, 5], cuda_device))
    torch.cuda.synchronize()
    assert capi.device_error() == (1, 10)
    for old, pair in zip(before, pairs):
        for o, t in zip(old, pair):
            assert np.array_equal(_bytes(t), oracle.paged_kv_copy_pages(o, [4], [5]))


def _sequences(rng, lens, ps, spare=3):
    mb = max(1, max((n + ps - 1) // ps for n in lens))
    P = sum((n + ps - 1) // ps for n in lens) + spare
    ids = iter(rng.permutation(P))
    bt = np.full((len(lens), mb), -1, dtype=np.int32)
    for b, n in enumerate(lens):
        for m in range((n + ps - 1) // ps):
            bt[b, m] = next(ids)
    return bt, P


def _lists(rng, lens, base, frac):
    keep, ptr = [], [0]
    for n, s in zip(lens, base):
        m = int(round((n - s) * frac))
        keep.extend(np.sort(rng.permutation(n - s)[:m]) + s)
        ptr.append(len(keep))
    return np.asarray(keep, dtype=np.int32), np.asarray(ptr, dtype=np.int32)


def _check_compact(dev, pairs, bt, lens, base, ptr, keep, pools=None):
    before = [[t.clone() for t in p] for p in pairs]
    new = capi.paged_kv_compact(pools or capi.make_pools(pairs), _dev(bt, dev), _dev(lens, dev), _dev(ptr, dev),
                                _dev(keep, dev), base=None if base is None else _dev(base, dev))
    torch.cuda.synchronize()
    assert capi.device_error() == (0, 0)
    at = np.zeros(len(lens), dtype=np.int64) if base is None else np.asarray(base)
    assert np.array_equal(new.cpu().numpy(), at + np.diff(ptr))
    for old, pair in zip(before, pairs):
        for o, t in zip(old, pair):
            P, ps = o.shape[:2]
            exp = oracle.paged_kv_compact(_bytes(o).reshape(P, ps, -1), bt, at, ptr, keep)
            assert np.array_equal(_bytes(t).reshape(P, ps, -1), exp)


@pytest.mark.parametrize("dtype", ["bf16", "f32", "e4m3"])
@pytest.mark.parametrize("layers,ps,hkv,d", [(1, 16, 8, 128), (3, 16, 1, 128), (2, 8, 2, 64), (130, 4, 1, 16),
                                             (1, 1, 3, 5), (2, 12, 1, 7), (1, 64, 4, 256)])
def test_compact(cuda_device, dtype, layers, ps, hkv, d):
    rng = np.random.default_rng(ps + d)
    lens = [0, 1, 5, 100, 17, 333] if layers < 100 else [9, 20]
    bt, P = _sequences(rng, lens, ps)
    base = [min(n, k) for n, k in zip(lens, [0, 1, 2, 4, 17, 0])]
    ptr_keep = _lists(rng, lens, base, 0.6)
    pairs = _pools(cuda_device, layers, P, ps, hkv, d, dtype, seed=d)
    _check_compact(cuda_device, pairs, bt, lens, base, ptr_keep[1], ptr_keep[0])


@pytest.mark.parametrize("frac", [0.0, 0.02, 0.5, 0.97, 1.0])
@pytest.mark.parametrize("layers,lens", [(1, [4000]), (12, [2000, 1, 700]), (2, [37] * 40)])
def test_compact_many_rows(cuda_device, layers, lens, frac):
    # long lists (many tiles that read rows the same tile overwrites), wide and narrow grids
    rng = np.random.default_rng(len(lens))
    bt, P = _sequences(rng, lens, 16)
    keep, ptr = _lists(rng, lens, [0] * len(lens), frac)
    pairs = _pools(cuda_device, layers, P, 16, 8, 64, "bf16", seed=3)
    _check_compact(cuda_device, pairs, bt, lens, None, ptr, keep)


def test_compact_shifts_by_one(cuda_device):
    # every row moves onto the place of the one before it
    rng = np.random.default_rng(1)
    bt, P = _sequences(rng, [3000], 16)
    keep = np.arange(1, 3000, dtype=np.int32)
    pairs = _pools(cuda_device, 1, P, 16, 2, 64, "bf16")
    _check_compact(cuda_device, pairs, bt, [3000], [0], np.array([0, 2999], dtype=np.int32), keep)


def test_compact_bad_lists_leave_memory_in_range(cuda_device):
    rng = np.random.default_rng(2)
    lens = [40, 40, 40, 40]
    bt, P = _sequences(rng, lens, 16)
    pairs = _pools(cuda_device, 1, P, 16, 2, 64, "bf16")
    run = lambda lens, base, ptr, keep, table=bt: capi.paged_kv_compact(
        pairs, _dev(table, cuda_device), _dev(lens, cuda_device), _dev(ptr, cuda_device), _dev(keep, cuda_device),
        base=_dev(base, cuda_device))
    before = [_bytes(t) for t in pairs[0]]

    def same():
        torch.cuda.synchronize()
        return all(np.array_equal(_bytes(t), o) for t, o in zip(pairs[0], before))

    zero = [0, 0, 0, 0]
    new = run([40, -1, 1000, 40], zero, [0, 1, 2, 3, 4], [0, 0, 0, 0])      # bad lengths
    assert same() and capi.device_error()[0] == 3 and new.tolist() == [1, -1, 1000, 1]
    new = run(lens, [-1, 41, 0, 0], [0, 1, 2, 3, 4], [0, 0, 0, 0])          # bad bases
    assert same() and capi.device_error()[0] == 3 and new.tolist() == [40, 40, 1, 1]
    new = run(lens, zero, [0, 5, 2, 3, 9], [0, 1, 2, 3])                    # bad slices: past the list, backwards
    assert capi.device_error()[0] == 7 and new.tolist() == [40, 40, 1, 40]
    before = [_bytes(t) for t in pairs[0]]
    new = run(lens, [3, 0, 0, 0], [0, 2, 4, 4, 4], [2, 40, 0, 0])           # below base, past the end, not ascending
    assert same() and capi.device_error()[0] == 7
    bad = bt.copy()
    bad[0, 0] = P
    new = run(lens, zero, [0, 1, 1, 1, 1], [20], table=bad)                 # a page out of range
    assert same() and capi.device_error() == (1, P)


def test_compact_captured_and_replayed(cuda_device):
    rng = np.random.default_rng(4)
    lens = [60, 90]
    bt, P = _sequences(rng, lens, 16)
    keep, ptr = _lists(rng, lens, [0, 0], 0.5)
    a, b = _pools(cuda_device, 2, P, 16, 2, 64, "bf16", seed=5), _pools(cuda_device, 2, P, 16, 2, 64, "bf16", seed=5)
    args = [_dev(x, cuda_device) for x in (bt, lens, ptr, keep)]
    pools = capi.make_pools(b)
    new = torch.zeros(2, dtype=torch.int32, device=cuda_device)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        capi.paged_kv_compact(pools, *args, new_seq_lens=new)
    graph.replay()
    capi.paged_kv_compact(a, *args)
    torch.cuda.synchronize()
    for x, y in zip(a, b):
        assert all(np.array_equal(_bytes(s), _bytes(t)) for s, t in zip(x, y))
    assert new.tolist() == np.diff(ptr).tolist()


def test_copy_captured_and_replayed(cuda_device):
    pairs = [tuple(torch.randn(12, 16, 2, 64, device=cuda_device).to(torch.bfloat16) for _ in range(2)) for _ in range(3)]
    pools = capi.make_pools(pairs)
    src = torch.tensor([0, 1, 2], dtype=torch.int32, device=cuda_device)
    dst = torch.tensor([6, 7, -1], dtype=torch.int32, device=cuda_device)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        capi.paged_kv_copy_pages(pools, src, dst)
    for s, d in (([0, 1, 2], [6, 7, -1]), ([3, 4, 5], [9, -1, 11])):   # the same graph serves other pairs
        before = [[x.clone() for x in p] for p in pairs]
        src.copy_(torch.tensor(s, dtype=torch.int32))
        dst.copy_(torch.tensor(d, dtype=torch.int32))
        graph.replay()
        torch.cuda.synchronize()
        for p, old in zip(pairs, before):
            for x, o in zip(p, old):
                want = o.clone()
                for a, b in zip(s, d):
                    if b >= 0:
                        want[b] = o[a]
                assert torch.equal(x.view(torch.int16), want.view(torch.int16))
    assert capi.device_error() == (0, 0)

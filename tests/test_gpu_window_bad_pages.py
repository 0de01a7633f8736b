"""Windowed calls whose block_table has entries out of range in visible places: the
entry is recorded, the keys of that page take no part (as on the CUDA-core path),
and every other row is bit for bit what it is with a good table."""
import numpy as np
import pytest
import torch

import oracle
from serving_slot_mapping_gb300 import build as build_mod
from serving_slot_mapping_gb300 import capi

from _parity import bits, to_f64
from _window import Case

pytestmark = pytest.mark.gpu

BAD = 1 << 29


@pytest.fixture(scope="module", autouse=True)
def _lib(cuda_device):
    build_mod.build()
    capi.lib()
    capi.device_error()  # clear


def _without(c, b, row, position, K, V, q):
    """One query row over its visible keys whose pages are in range: the output and
    the same over |V| (what the tolerance of _window.py is relative to)."""
    keys = [j for j in oracle.visible_keys(position, c.window, c.sinks) if 0 <= c.table[b, j // c.ps] < len(K)]
    y, A = np.zeros(q.shape[1:]), np.zeros(q.shape[1:])
    if keys:
        k = np.stack([K[c.table[b, j // c.ps], j % c.ps] for j in keys])
        v = np.stack([V[c.table[b, j // c.ps], j % c.ps] for j in keys])
        g = q.shape[1] // K.shape[2]
        for h in range(q.shape[1]):
            s = c.scale * (k[:, h // g] @ q[row, h])
            w = np.exp(s - s.max())
            y[h], A[h] = w @ v[:, h // g] / w.sum(), w @ np.abs(v[:, h // g]) / w.sum()
    return y, A


def _check(c, out, good, hurt):
    """`hurt`: the sequences with a bad entry."""
    if c.dtype == "e4m3":
        K = oracle.kv_fp8.dequantize(bits(c.kp), c.k_scale)
        V = oracle.kv_fp8.dequantize(bits(c.vp), c.v_scale)
    else:
        K, V = to_f64(bits(c.kp)), to_f64(bits(c.vp))
    q, got = to_f64(bits(c.q)), to_f64(bits(out))
    w = {"bf16": 2.0 ** -8, "e4m3": 2.0 ** -11, "f32": 0.0}[c.dtype]
    small = 2.0 ** -25 * int(c.lens.max()) * 4 if c.dtype == "e4m3" else 0.0
    start = 0
    for b, n in enumerate(c.n):
        rows = [b] if c.is_decode else range(start, start + int(n))
        start += int(n)
        for i, r in enumerate(rows):
            if b not in hurt:
                assert torch.equal(out[r].view(torch.uint8), good[r].view(torch.uint8)), f"row {r}"
                continue
            y, A = _without(c, b, r, int(c.lens[b]) - len(rows) + i, K, V, q)
            tol = 1e-5 * (1 + A) if c.dtype == "f32" else 2.0 ** -8 * np.abs(y) + (w + 2.0 ** -12) * A + small
            assert np.isfinite(got[r]).all()
            err = np.abs(got[r] - y)
            assert (err <= tol).all(), f"row {r}: error {err.max():.3e}, {(err / np.maximum(tol, 1e-30)).max():.2f} of the tolerance"


def _run(make, device, entries):
    """entries: {(sequence, page of the sequence): value}."""
    good = make().check(capi, device)
    c = make()
    for at, value in entries.items():
        c.table[at] = value
    out = c.run(capi, device)
    torch.cuda.synchronize()
    code, detail = capi.device_error()
    assert code == 1 and detail in entries.values()
    _check(c, out, good, {b for b, _ in entries})
    again = make().check(capi, device)
    assert torch.equal(again.view(torch.uint8), good.view(torch.uint8))


def _decode(**k):
    lens = np.array([300, 40, 700, 90, 1, 5])
    return Case(np.ones(6, dtype=int), lens - 1, 100, 4, **k)


def _pages(ps, *keys):
    return {(b, j // ps): v for b, j, v in keys}


# hq, hkv, d, ps: each number of heads on a KV head that has a form of its own, half blocks, large pages
@pytest.mark.parametrize("dtype,hq,hkv,d,ps", [
    ("bf16", 8, 2, 64, 16), ("bf16", 8, 2, 128, 8), ("bf16", 32, 2, 64, 16), ("bf16", 32, 1, 128, 8),
    ("bf16", 4, 4, 128, 64), ("e4m3", 8, 2, 128, 16), ("e4m3", 32, 1, 64, 8), ("e4m3", 16, 1, 128, 32),
    ("bf16", 4, 2, 64, 12), ("f32", 4, 2, 64, 16)])
def test_decode_skips_the_keys_of_bad_pages(cuda_device, dtype, hq, hkv, d, ps):
    make = lambda: _decode(hq=hq, hkv=hkv, d=d, ps=ps, dtype=dtype, seed=hq + d + ps)
    _run(make, cuda_device, _pages(ps, (0, 0, BAD)))                                 # the sinks' page
    _run(make, cuda_device, _pages(ps, (2, 660, -7), (0, 299, BAD)))                 # inside the window; the last page
    _run(make, cuda_device, _pages(ps, (4, 0, BAD), (5, 0, BAD)))                    # every key: the rows give 0
    _run(make, cuda_device, _pages(ps, *((2, j, BAD) for j in [0, *range(600, 700)])))


def test_decode_bad_pages_on_clusters_and_short_rings(cuda_device):
    lens = np.array([5000, 4000, 3])
    make = lambda: Case(np.ones(3, dtype=int), lens - 1, 2500, 20, hq=32, hkv=8, d=128, seed=10)
    _run(make, cuda_device, _pages(16, (0, 0, BAD), *((0, j, BAD) for j in range(3000, 3400)), (1, 3999, -1)))
    lens = np.random.default_rng(3).integers(1, 300, 420)  # over 608 CTAs
    make = lambda: Case(np.ones(420, dtype=int), lens - 1, 100, 4, hq=8, hkv=2, d=128, seed=12)
    _run(make, cuda_device, {(b, int(lens[b] - 1) // 16): BAD for b in range(0, 420, 7)})


NEW, CACHED = [60, 300, 20, 9, 130], [0, 200, 5, 900, 300]


# page sizes below, at and above a tile of 128 keys
@pytest.mark.parametrize("dtype,hq,hkv,d,ps", [
    ("bf16", 8, 2, 64, 16), ("bf16", 8, 2, 128, 8), ("bf16", 5, 1, 128, 64), ("bf16", 4, 2, 64, 128),
    ("bf16", 4, 2, 64, 256), ("e4m3", 8, 2, 64, 16), ("e4m3", 8, 2, 128, 8), ("e4m3", 4, 1, 128, 128),
    ("bf16", 4, 2, 64, 12)])
def test_prefill_skips_the_keys_of_bad_pages(cuda_device, dtype, hq, hkv, d, ps):
    make = lambda: Case(NEW, CACHED, 70, 4, hq=hq, hkv=hkv, d=d, ps=ps, dtype=dtype, seed=hq + d + ps)
    _run(make, cuda_device, _pages(ps, (1, 0, BAD)))                                 # the sinks' page
    _run(make, cuda_device, _pages(ps, (1, 333, -7), (0, 59, BAD), (4, 429, -1)))    # inside the window; the last pages
    _run(make, cuda_device, _pages(ps, *((2, j, BAD) for j in range(25))))           # every key: the rows give 0
    _run(make, cuda_device, _pages(ps, *((4, j, BAD) for j in [0, *range(250, 430, 8)])))


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
def test_prefill_bad_pages_on_clusters_and_many_items(cuda_device, dtype):
    make = lambda: Case([33, 1, 70], [900, 1500, 0], 1300, 40, hq=8, hkv=2, d=128, dtype=dtype, seed=51)
    _run(make, cuda_device, _pages(16, (0, 0, BAD), *((0, j, -3) for j in range(400, 700, 16)), (2, 69, BAD)))
    _run(make, cuda_device, _pages(16, *((0, j, BAD) for j in range(0, 933, 16))))   # every key of the first sequence
    make = lambda: Case(np.full(90, 25), np.full(90, 150), 100, 4, hq=16, hkv=4, d=128, dtype=dtype, seed=52)
    _run(make, cuda_device, {(b, m): BAD for b in range(0, 90, 5) for m in (0, 7, 10)})


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
def test_prefill_bad_pages_behind_an_items_last_key(cuda_device, dtype):
    """A page that only later rows of the sequence see, in the last key tile of the
    rows before them (64 tokens of 4 heads are one item)."""
    make = lambda: Case([300, 40], [0, 100], 70, 4, hq=8, hkv=2, d=128, dtype=dtype, seed=53)
    for j in (64, 80, 112, 130, 191, 256):
        _run(make, cuda_device, _pages(16, (0, j, BAD)))

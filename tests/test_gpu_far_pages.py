"""Pools whose far pages lie past 2^31 elements and 2^32 bytes: the windowed layer's
calls on those pages give what they give on small pools, bit for bit."""
import numpy as np
import pytest
import torch

from serving_slot_mapping_gb300 import build as build_mod
from serving_slot_mapping_gb300 import capi

from _window import Case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib(cuda_device):
    build_mod.build()
    capi.lib()
    capi.device_error()  # clear


@pytest.fixture(scope="module", params=["bf16", "e4m3"])
def far(request, cuda_device):
    """Two pools of 16 x 8 x 128 elements a page, 2.3e9 (e4m3: 4.7e9) elements each, and the page from which on a
    small pool is laid over them."""
    dtype = request.param
    n = 140_000 if dtype == "bf16" else 285_000
    t = torch.bfloat16 if dtype == "bf16" else torch.float8_e4m3fn
    pools = [torch.empty(n, 16, 8, 128, dtype=t, device=cuda_device) for _ in range(2)]
    yield dtype, pools, n - 2000
    del pools
    torch.cuda.empty_cache()


def _raw(t):
    return t.view(torch.uint8)


@pytest.mark.parametrize("new", [[1, 1, 1], [60, 1, 300]])
def test_attention(cuda_device, far, new):
    dtype, (kp, vp), base = far
    c = Case(new, [300, 1999, 40], 500, 20, hq=32, hkv=8, d=128, dtype=dtype, seed=91)
    good = c.check(capi, cuda_device)
    for pool, small in ((kp, c.kp), (vp, c.vp)):
        _raw(pool)[base:base + len(small)].copy_(_raw(small))
        _raw(pool)[:len(small)].fill_(0x55)          # where a truncated offset would land
    dev = lambda a: torch.from_numpy(np.ascontiguousarray(a)).to(cuda_device)
    table = dev(np.where((c.table >= 0) & (c.table < len(c.kp)), c.table + base, -1).astype(np.int32))
    kw = dict(max_seq_len=int(c.lens.max()), k_scale=c.k_scale, v_scale=c.v_scale)
    q = c.q.to(cuda_device)
    if c.is_decode:
        out = capi.paged_attention_decode_window(kp, vp, q, table, dev(c.lens), c.scale, 500, 20, **kw)
    else:
        out = capi.paged_attention_prefill_window(kp, vp, q, dev(c.qsl), table, dev(c.lens), c.scale, 300, 500, 20, **kw)
    torch.cuda.synchronize()
    assert capi.device_error() == (0, 0)
    assert torch.equal(out.view(torch.int16), good.view(torch.int16))


@pytest.mark.parametrize("tokens", [5, 700])
def test_append(cuda_device, far, tokens):
    dtype, (kp, vp), base = far
    g = torch.Generator(device=cuda_device).manual_seed(92)
    r = lambda h: torch.randn(tokens, h, 128, generator=g, device=cuda_device).bfloat16()
    q, k, v = r(32), r(8), r(8)
    cs = torch.randn(100, 128, generator=g, device=cuda_device)
    pos = torch.randint(0, 100, (tokens,), generator=g, device=cuda_device, dtype=torch.int32)
    slots = torch.randperm(50 * 16, generator=g, device=cuda_device)[:tokens]
    small = [torch.zeros(50, 16, 8, 128, device=cuda_device).to(kp.dtype) for _ in range(2)]
    want = capi.paged_qk_norm_rope_append(*small, q, k, v, slots, pos, cs, k_scale=0.02, v_scale=0.03)
    for pool in (kp, vp):
        _raw(pool)[base:base + 50].fill_(0)
        _raw(pool)[:50].fill_(0x55)
    got = capi.paged_qk_norm_rope_append(kp, vp, q, k, v, slots + base * 16, pos, cs, k_scale=0.02, v_scale=0.03)
    torch.cuda.synchronize()
    assert capi.device_error() == (0, 0)
    assert torch.equal(got, want)
    for pool, s in zip((kp, vp), small):
        assert torch.equal(_raw(pool)[base:base + 50], _raw(s))
        assert torch.all(_raw(pool)[:50] == 0x55)


def test_page_moves(cuda_device, far):
    _, (kp, vp), base = far
    g = torch.Generator(device=cuda_device).manual_seed(93)
    for pool in (kp, vp):
        _raw(pool)[base:base + 100].copy_(torch.randint(0, 256, _raw(pool)[base:base + 100].shape, generator=g,
                                                        device=cuda_device, dtype=torch.uint8))
        _raw(pool)[:100].fill_(0x55)
    small = [p[base:base + 100].clone() for p in (kp, vp)]
    i32 = lambda a: torch.as_tensor(a, device=cuda_device, dtype=torch.int32)
    src, dst = i32([3, 0, 41, 7]), i32([99, 60, 98, 61])
    capi.paged_kv_copy_pages([(kp, vp)], src + base, dst + base)
    capi.paged_kv_copy_pages([tuple(small)], src, dst)
    table, lens = torch.arange(40, device=cuda_device, dtype=torch.int32).view(2, 20), i32([300, 77])
    keep = [np.arange(3, 290, 2), np.arange(5, 77)]
    ptr, kk = i32([0, len(keep[0]), len(keep[0]) + len(keep[1])]), i32(np.concatenate(keep))
    a = capi.paged_kv_compact([(kp, vp)], table + base, lens, ptr, kk)
    b = capi.paged_kv_compact([tuple(small)], table, lens, ptr, kk)
    torch.cuda.synchronize()
    assert capi.device_error() == (0, 0)
    assert torch.equal(a, b)
    for pool, s in zip((kp, vp), small):
        assert torch.equal(_raw(pool)[base:base + 100], _raw(s))
        assert torch.all(_raw(pool)[:100] == 0x55)

"""Host-side checks of the int8 calls, the decode with attention weights and the
evictions: status codes of the C ABI and the binding's refusals.  No kernel is launched
(no GPU needed)."""
import ctypes
import os
import re

import pytest
import torch

from serving_slot_mapping_gb300 import build as build_mod
from serving_slot_mapping_gb300 import capi

FAKE = ctypes.c_void_p(0x40000)  # never dereferenced: every call below fails validation or does nothing
OUT = ctypes.c_void_p(0x8000000)
CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "serving_slot_mapping_gb300", "csrc")


@pytest.fixture(scope="module")
def L():
    build_mod.build()
    return capi.lib()


def _pool(dtype=capi.PA_DTYPE_INT8, hkv=8, d=128, ps=16, P=64, k=0x10000000, v=0x20000000, ks=1.0, vs=1.0):
    return capi.PaKvPool(k, v, P, ps, hkv, d, dtype, ks, vs)


def _scales(k=0x30000000, v=0x31000000, blk=16):
    return capi.PaKvScales(k, v, blk)


BAD_POOLS = [(dict(pool=_pool(dtype=capi.PA_DTYPE_BF16)), capi.PA_ERR_DTYPE),
             (dict(pool=_pool(dtype=capi.PA_DTYPE_FP8_E4M3)), capi.PA_ERR_DTYPE),
             (dict(pool=_pool(d=96)), capi.PA_ERR_UNSUPPORTED), (dict(pool=_pool(d=256)), capi.PA_ERR_UNSUPPORTED),
             (dict(pool=_pool(ps=48), scales=_scales(blk=16)), capi.PA_ERR_UNSUPPORTED),
             (dict(pool=_pool(ps=32), scales=_scales(blk=24)), capi.PA_ERR_UNSUPPORTED),
             (dict(scales=_scales(blk=8)), capi.PA_ERR_UNSUPPORTED), (dict(scales=_scales(blk=32)), capi.PA_ERR_SHAPE),
             (dict(scales=_scales(blk=0)), capi.PA_ERR_SHAPE), (dict(scales=_scales(k=0)), capi.PA_ERR_NULL),
             (dict(scales=_scales(v=0x31000008)), capi.PA_ERR_ALIGN), (dict(pool=_pool(k=0x10000008)), capi.PA_ERR_ALIGN),
             (dict(pool=_pool(P=1 << 27)), capi.PA_ERR_RANGE), (dict(pool=_pool(P=0)), capi.PA_ERR_SHAPE)]


def _append(L, pool=_pool(), scales=_scales(), key=FAKE, ks=1024, value=FAKE, vs=1024, slots=FAKE, T=4):
    return L.paged_kv_append_int8(ctypes.byref(pool), ctypes.byref(scales), key, ks, value, vs, slots, T, None)


def _decode(L, pool=_pool(), scales=_scales(), q=FAKE, out=OUT, batch=2, hq=32, bt=FAKE, mb=4, sl=FAKE, msl=64, scale=0.1,
            ws=FAKE, wsb=1 << 30):
    return L.paged_attention_decode_int8(ctypes.byref(pool), ctypes.byref(scales), q, out, batch, hq, bt, mb, sl, msl, scale,
                                         ws, wsb, None)


def _prefill(L, pool=_pool(), scales=_scales(), q=FAKE, out=OUT, batch=2, hq=32, qsl=FAKE, total=10, mql=5, bt=FAKE, mb=4,
             sl=FAKE, msl=64, scale=0.1):
    return L.paged_attention_prefill_int8(ctypes.byref(pool), ctypes.byref(scales), q, out, batch, hq, qsl, total, mql, bt,
                                          mb, sl, msl, scale, None)


def _mass(L, pool=_pool(), scales=_scales(), q=FAKE, out=OUT, batch=2, hq=32, bt=FAKE, mb=4, sl=FAKE, msl=64, scale=0.1,
          mass_in=None, decay=1.0, mass_out=ctypes.c_void_p(0x9000000), stride=64, ws=FAKE, wsb=1 << 30):
    return L.paged_attention_decode_mass(ctypes.byref(pool), None if scales is None else ctypes.byref(scales), q, out, batch,
                                         hq, bt, mb, sl, msl, scale, mass_in, decay, mass_out, stride, ws, wsb, None)


@pytest.mark.parametrize("call", [_append, _decode, _prefill, _mass])
@pytest.mark.parametrize("bad,status", BAD_POOLS)
def test_int8_pools(L, call, bad, status):
    if call is _mass and "pool" in bad and bad["pool"].dtype != capi.PA_DTYPE_INT8:
        return  # it takes those
    assert call(L, **bad) == status


def test_int8_pools_are_refused_elsewhere(L):
    p = _pool()
    assert L.paged_kv_append(ctypes.byref(p), FAKE, FAKE, FAKE, 4, None) == capi.PA_ERR_DTYPE
    assert L.paged_attention_decode(ctypes.byref(p), FAKE, OUT, 2, 32, FAKE, 4, FAKE, 64, 0.1, FAKE, 1 << 30, None) \
        == capi.PA_ERR_DTYPE
    assert L.paged_attention_prefill(ctypes.byref(p), FAKE, OUT, 2, 32, FAKE, 10, 5, FAKE, 4, FAKE, 64, 0.1, None) \
        == capi.PA_ERR_DTYPE
    assert L.paged_attention_decode_window(ctypes.byref(p), FAKE, OUT, 2, 32, FAKE, 4, FAKE, 64, 0.1, 8, 0, FAKE, 1, None) \
        == capi.PA_ERR_DTYPE
    pools = (capi.PaKvPool * 1)(p)
    assert L.paged_kv_compact(pools, 1, FAKE, 4, FAKE, 2, None, FAKE, FAKE, 5, OUT, None) == capi.PA_ERR_DTYPE
    assert L.paged_kv_copy_pages(pools, 1, FAKE, FAKE, 0, None) == capi.PA_OK      # taken


def test_append_validation(L):
    assert _append(L, T=0) == capi.PA_OK
    assert _append(L, T=-1) == capi.PA_ERR_SHAPE
    assert _append(L, T=1 << 32) == capi.PA_ERR_RANGE
    assert _append(L, ks=1016) == capi.PA_ERR_SHAPE
    assert _append(L, vs=-1024) == capi.PA_ERR_SHAPE
    assert _append(L, vs=1 << 40) == capi.PA_ERR_RANGE
    assert _append(L, ks=1028) == capi.PA_ERR_ALIGN
    for name in ("key", "value", "slots"):
        assert _append(L, **{name: None}) == capi.PA_ERR_NULL, name
        assert _append(L, **{name: ctypes.c_void_p(0x40004)}) == capi.PA_ERR_ALIGN, name


def test_attention_validation(L):
    for call in (_decode, _prefill, _mass):
        assert call(L, hq=12) == capi.PA_ERR_SHAPE
        assert call(L, pool=_pool(hkv=1), hq=64) == capi.PA_ERR_UNSUPPORTED
        assert call(L, msl=65, **(dict(stride=65) if call is _mass else {})) == capi.PA_ERR_SHAPE
        assert call(L, scale=float("nan")) == capi.PA_ERR_RANGE
        assert call(L, out=FAKE) == capi.PA_ERR_SHAPE
        assert call(L, out=ctypes.c_void_p(0x8000004)) == capi.PA_ERR_ALIGN
        assert call(L, batch=0) == capi.PA_OK
        for name in ("q", "out", "bt", "sl"):
            assert call(L, **{name: None}) == capi.PA_ERR_NULL, name
    assert _decode(L, wsb=16) == capi.PA_ERR_WORKSPACE
    assert _prefill(L, qsl=None) == capi.PA_ERR_NULL
    assert _prefill(L, q=ctypes.c_void_p(0x40008)) == capi.PA_ERR_ALIGN
    assert _prefill(L, total=0) == capi.PA_OK


def test_mass_validation(L):
    bf16 = dict(pool=_pool(dtype=capi.PA_DTYPE_BF16), scales=None)
    assert _mass(L, pool=_pool(dtype=capi.PA_DTYPE_F32), scales=None) == capi.PA_ERR_UNSUPPORTED
    assert _mass(L, pool=_pool(dtype=capi.PA_DTYPE_BF16, ps=4), scales=None, msl=16) == capi.PA_ERR_UNSUPPORTED
    assert _mass(L, scales=None) == capi.PA_ERR_NULL          # int8 pools need their scales
    assert _mass(L, stride=63, **bf16) == capi.PA_ERR_SHAPE
    assert _mass(L, stride=1 << 31, **bf16) == capi.PA_ERR_RANGE
    assert _mass(L, decay=float("inf"), **bf16) == capi.PA_ERR_RANGE
    assert _mass(L, batch=65536, **bf16) == capi.PA_ERR_RANGE
    assert _mass(L, mass_out=None, **bf16) == capi.PA_ERR_NULL
    assert _mass(L, mass_out=ctypes.c_void_p(0x9000002), **bf16) == capi.PA_ERR_ALIGN
    assert _mass(L, mass_in=ctypes.c_void_p(0x9000100), **bf16) == capi.PA_ERR_SHAPE       # rows one beside the other
    need = L.paged_attention_decode_mass_workspace_size(2, 32, 8, 128, capi.PA_DTYPE_BF16, 64)
    assert need >= L.paged_attention_decode_workspace_size(2, 32, 8, 128, capi.PA_DTYPE_BF16) + 2 * 32 * 65 * 4
    assert _mass(L, wsb=need - 1, **bf16) == capi.PA_ERR_WORKSPACE
    assert _mass(L, ws=None, **bf16) == capi.PA_ERR_WORKSPACE
    assert L.paged_attention_decode_mass_workspace_size(2, 32, 8, 128, capi.PA_DTYPE_F32, 64) == 0
    assert L.paged_attention_decode_mass_workspace_size(2, 32, 8, 128, capi.PA_DTYPE_BF16, -1) == 0


def test_evict_rows_validation(L):
    def call(mass=FAKE, ms=100, sl=OUT, B=2, width=100, budget=50, sinks=4, recent=8, ptr=ctypes.c_void_p(0x9000000),
             keep=ctypes.c_void_p(0x9100000), n=92, base=ctypes.c_void_p(0x9200000), new=ctypes.c_void_p(0x9300000), ns=100):
        return L.paged_kv_evict_rows(mass, ms, sl, B, width, budget, sinks, recent, ptr, keep, n, base, new, ns, None)
    assert call(B=0, n=0) == capi.PA_OK
    for bad in (dict(B=-1), dict(width=-1), dict(budget=-1, sinks=0, recent=0), dict(sinks=-1), dict(recent=-1), dict(ms=99),
                dict(ns=99), dict(budget=11), dict(sinks=2 ** 31 - 1, recent=2 ** 31 - 1), dict(n=91), dict(n=-1)):
        assert call(**bad) == capi.PA_ERR_SHAPE, bad
    assert call(ms=1 << 31) == capi.PA_ERR_RANGE
    assert call(B=1 << 27, n=1 << 40) == capi.PA_ERR_RANGE
    for name in ("mass", "sl", "ptr", "keep", "base", "new"):
        assert call(**{name: None}) == capi.PA_ERR_NULL, name
        assert call(**{name: ctypes.c_void_p(0x9000002)}) == capi.PA_ERR_ALIGN, name
    for bad in (dict(new=FAKE), dict(new=ctypes.c_void_p(0x40000 + 796)), dict(base=OUT), dict(keep=ctypes.c_void_p(0x9000008)),
                dict(ptr=ctypes.c_void_p(0x9300000))):
        assert call(**bad) == capi.PA_ERR_SHAPE, bad


def test_evict_pages_validation(L):
    def call(mass=FAKE, ms=100, bt=ctypes.c_void_p(0x9000000), mb=7, sl=OUT, B=2, width=100, ps=16, budget=5, sinks=4, recent=8,
             nbt=ctypes.c_void_p(0x9100000), nl=ctypes.c_void_p(0x9200000), new=ctypes.c_void_p(0x9300000), ns=100):
        return L.paged_kv_evict_pages(mass, ms, bt, mb, sl, B, width, ps, budget, sinks, recent, nbt, nl, new, ns, None)
    assert call(B=0) == capi.PA_OK
    # 4 sinks: a page; 8 recent rows: two at most
    for bad in (dict(B=-1), dict(mb=0), dict(ps=0), dict(budget=2), dict(ms=99), dict(ns=99), dict(sinks=-1), dict(recent=-1),
                dict(sinks=0, recent=0, budget=0)):
        assert call(**bad) == capi.PA_ERR_SHAPE, bad
    assert call(ps=12) == capi.PA_ERR_UNSUPPORTED
    assert call(ps=2048) == capi.PA_ERR_UNSUPPORTED
    assert call(mb=1 << 28) == capi.PA_ERR_RANGE
    assert call(ps=1, mb=400000, width=400000, ms=400000, ns=400000, budget=100) == capi.PA_ERR_RANGE
    for name in ("mass", "bt", "sl", "nbt", "nl", "new"):
        assert call(**{name: None}) == capi.PA_ERR_NULL, name
        assert call(**{name: ctypes.c_void_p(0x9000002)}) == capi.PA_ERR_ALIGN, name
    for bad in (dict(nbt=ctypes.c_void_p(0x9000000)), dict(nl=OUT), dict(new=FAKE), dict(nl=ctypes.c_void_p(0x9100004))):
        assert call(**bad) == capi.PA_ERR_SHAPE, bad


# ---- the binding -----------------------------------------------------------------

def _t(dtype=torch.int8, blocks=1):
    kp = torch.zeros(4, 16, 2, 64, dtype=dtype)
    return kp, torch.zeros_like(kp), torch.ones(4, blocks, 2), torch.ones(4, blocks, 2)


def test_binding_refuses_tensors_that_are_not_on_the_device():
    pools = _t()
    bf = _t(torch.bfloat16)
    q, k = torch.zeros(3, 4, 64, dtype=torch.bfloat16), torch.zeros(3, 2, 64, dtype=torch.bfloat16)
    bt, sl = torch.zeros(3, 2, dtype=torch.int32), torch.ones(3, dtype=torch.int32)
    qsl, m = torch.tensor([0, 1, 2, 3], dtype=torch.int32), torch.zeros(3, 32)
    for f in (lambda: capi.paged_kv_append_int8(*pools, k, k, torch.zeros(3, dtype=torch.int64)),
              lambda: capi.paged_attention_decode_int8(*pools, q, bt, sl, 0.1),
              lambda: capi.paged_attention_prefill_int8(*pools, q, qsl, bt, sl, 0.1, 1),
              lambda: capi.paged_attention_decode_mass(bf[0], bf[1], q, bt, sl, 0.1, m),
              lambda: capi.paged_kv_evict_rows(m, sl, 20, 1, 1),
              lambda: capi.paged_kv_evict_pages(m, bt, sl, 16, 3, 1, 1)):
        with pytest.raises(ValueError, match="CUDA tensor"):
            f()


def test_binding_checks_of_int8_calls():
    kp, vp, ks, vs = _t()
    q, k = torch.zeros(3, 4, 64, dtype=torch.bfloat16), torch.zeros(3, 2, 64, dtype=torch.bfloat16)
    bt, sl = torch.zeros(3, 2, dtype=torch.int32), torch.ones(3, dtype=torch.int32)
    slots = torch.zeros(3, dtype=torch.int64)
    app = lambda kp=kp, vp=vp, ks=ks, vs=vs, k=k, v=k, slots=slots: capi.paged_kv_append_int8(kp, vp, ks, vs, k, v, slots)
    for bad in (dict(kp=kp.bfloat16(), vp=vp.bfloat16()), dict(vp=vp[:3]), dict(ks=ks[:3]), dict(ks=ks.double()),
                dict(ks=torch.ones(4, 3, 2), vs=torch.ones(4, 3, 2)), dict(ks=ks[:, 0]), dict(k=k.float()), dict(v=k[:2]),
                dict(k=k.transpose(1, 2).contiguous().transpose(1, 2)), dict(ks=torch.ones(4, 2, 1).transpose(1, 2))):
        with pytest.raises(ValueError):
            app(**bad)
    with pytest.raises(TypeError):
        app(slots=slots.int())
    dec = lambda q=q, bt=bt, sl=sl, **kw: capi.paged_attention_decode_int8(kp, vp, ks, vs, q, bt, sl, 0.1, **kw)
    for bad in (dict(q=q.float()), dict(bt=bt[:2]), dict(sl=sl[:2]), dict(out=torch.zeros(3, 4, 64)),
                dict(max_seq_len=1 << 40)):
        with pytest.raises(ValueError):
            dec(**bad)
    with pytest.raises(TypeError):
        dec(bt=bt.long())
    with pytest.raises(ValueError, match="query_start_loc"):
        capi.paged_attention_prefill_int8(kp, vp, ks, vs, q, torch.zeros(3, dtype=torch.int32), bt, sl, 0.1, 1)


def test_binding_checks_of_masses():
    kp, vp, ks, vs = _t()
    q = torch.zeros(3, 4, 64, dtype=torch.bfloat16)
    bt, sl, m = torch.zeros(3, 2, dtype=torch.int32), torch.ones(3, dtype=torch.int32), torch.zeros(3, 32)
    call = lambda m=m, ks=ks, vs=vs, **kw: capi.paged_attention_decode_mass(kp, vp, q, bt, sl, 0.1, m, key_scales=ks,
                                                                            value_scales=vs, **kw)
    for bad in (dict(ks=None), dict(ks=None, vs=None), dict(m=m[:2]), dict(m=m[:, :31]), dict(m=m.double()),
                dict(m=torch.zeros(32, 3).t()), dict(mass_in=torch.zeros(3, 40)), dict(mass_in=m.half())):
        with pytest.raises(ValueError):
            call(**bad)
    rows = lambda m=m, sl=sl, **kw: capi.paged_kv_evict_rows(m, sl, 20, 1, 1, **kw)
    for bad in (dict(m=m[0]), dict(m=m.double()), dict(sl=sl[:2]), dict(base=sl[:2]), dict(keep_indptr=sl)):
        with pytest.raises(ValueError):
            rows(**bad)
    with pytest.raises(TypeError):
        rows(sl=sl.long())
    with pytest.raises(ValueError):
        capi.paged_kv_evict_rows(m, sl, 1 << 40)
    for bad in (dict(new_block_table=bt[:2]), dict(new_seq_lens=sl[:2])):
        with pytest.raises(ValueError):
            capi.paged_kv_evict_pages(m, bt, sl, 16, 3, 1, 1, **bad)


@pytest.mark.parametrize("name", ["append_int8.cu", "decode_mass.cu", "evict.cu"])
def test_kernels_wait_ahead_of_ordinary_reads(name):
    """They may start before the kernel ahead of them has ended: no load that promises
    data that nobody writes, and none ahead of the wait."""
    src = re.sub(r"//[^\n]*", "", open(os.path.join(CSRC, name)).read())
    assert not re.search(r"__ldg|__ldc[sagv]|__ldlu|\.nc\b|__restrict__|\b(seq_keys|page_list_start)\b", src)
    for m in re.finditer(r"__global__ void", src):
        body = src[m.start():]
        assert not re.search(r"ld_input\(|ld_stream\(|ld_seq_len\(|ld_float\(", body[:body.index("griddep_wait()")])

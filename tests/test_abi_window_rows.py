"""Host-side checks of the sliding-window calls, the norm-rotate-append call and
the page moves: status codes of the C ABI and the binding's refusals.  No kernel
is launched (no GPU needed)."""
import ctypes

import pytest
import torch

from serving_slot_mapping_gb300 import build as build_mod
from serving_slot_mapping_gb300 import capi

FAKE = ctypes.c_void_p(0x40000)  # never dereferenced: every call below fails validation or does nothing
OUT = ctypes.c_void_p(0x8000000)


@pytest.fixture(scope="module")
def L():
    build_mod.build()
    return capi.lib()


def _pool(dtype=capi.PA_DTYPE_BF16, hkv=8, d=128, ps=16, P=64, k=0x10000000, v=0x20000000, ks=1.0, vs=1.0):
    return capi.PaKvPool(k, v, P, ps, hkv, d, dtype, ks, vs)


def test_decode_window_validation(L):
    def call(pool=None, window=10, sinks=4, msl=64, q=FAKE, out=OUT, hq=32, batch=2, ws=FAKE, wsb=1 << 30):
        pool = pool or _pool()
        return L.paged_attention_decode_window(ctypes.byref(pool), q, out, batch, hq, FAKE, 4, FAKE, msl, 0.1, window,
                                               sinks, ws, wsb, None)
    assert call(window=0) == capi.PA_ERR_SHAPE
    assert call(window=-3) == capi.PA_ERR_SHAPE
    assert call(sinks=-1) == capi.PA_ERR_SHAPE
    assert call(batch=0) == capi.PA_OK
    assert call(hq=12) == capi.PA_ERR_SHAPE
    assert call(q=None) == capi.PA_ERR_NULL
    assert call(out=FAKE) == capi.PA_ERR_SHAPE
    assert call(msl=65) == capi.PA_ERR_SHAPE
    assert call(pool=_pool(d=96)) == capi.PA_ERR_UNSUPPORTED
    assert call(out=ctypes.c_void_p(0x8000004)) == capi.PA_ERR_ALIGN
    assert call(ws=None, wsb=0) == capi.PA_ERR_WORKSPACE
    assert L.paged_attention_decode_window(None, FAKE, OUT, 2, 32, FAKE, 4, FAKE, 64, 0.1, 8, 0, FAKE, 1, None) \
        == capi.PA_ERR_NULL


def test_prefill_window_validation(L):
    def call(window=10, sinks=4, total=10, mql=5, q=FAKE, out=OUT, p=_pool()):
        return L.paged_attention_prefill_window(ctypes.byref(p), q, out, 2, 32, FAKE, total, mql, FAKE, 4, FAKE, 64,
                                                0.1, window, sinks, None)
    assert call(window=0) == capi.PA_ERR_SHAPE
    assert call(sinks=-1) == capi.PA_ERR_SHAPE
    assert call(total=0) == capi.PA_OK
    assert call(mql=0) == capi.PA_ERR_SHAPE
    assert call(q=None) == capi.PA_ERR_NULL
    assert call(q=ctypes.c_void_p(0x40008)) == capi.PA_ERR_ALIGN
    assert call(out=ctypes.c_void_p(0x8000008)) == capi.PA_ERR_ALIGN
    assert call(p=_pool(P=1 << 27)) == capi.PA_ERR_RANGE             # 2^31 slots


def test_norm_rope_append_validation(L):
    def call(pool=None, q=FAKE, qs=4096, key=FAKE, kstr=1024, value=FAKE, vstr=1024, out=OUT, hq=32, qw=FAKE, kw=FAKE,
             eps=1e-6, pos=FAKE, cs=FAKE, max_pos=100, rot=128, inter=0, slots=FAKE, T=4):
        pool = pool or _pool()
        return L.paged_qk_norm_rope_append(ctypes.byref(pool), q, qs, key, kstr, value, vstr, out, hq, qw, kw, eps, pos,
                                           cs, max_pos, rot, inter, slots, T, None)
    assert call(T=0) == capi.PA_OK
    assert call(T=-1) == capi.PA_ERR_SHAPE
    assert call(hq=0) == capi.PA_ERR_SHAPE
    assert call(rot=136) == capi.PA_ERR_SHAPE                       # more than head_dim
    assert call(rot=-8) == capi.PA_ERR_SHAPE
    assert call(rot=20) == capi.PA_ERR_UNSUPPORTED                  # not a multiple of 8
    assert call(inter=2) == capi.PA_ERR_SHAPE
    assert call(pool=_pool(d=100), rot=64) == capi.PA_ERR_UNSUPPORTED
    assert call(pool=_pool(d=264), qs=9000) == capi.PA_ERR_UNSUPPORTED
    assert call(max_pos=0) == capi.PA_ERR_SHAPE
    assert call(eps=-1.0) == capi.PA_ERR_RANGE
    assert call(eps=float("nan")) == capi.PA_ERR_RANGE
    assert call(qs=4095) == capi.PA_ERR_SHAPE                       # rows overlap
    assert call(kstr=1000) == capi.PA_ERR_SHAPE
    assert call(vstr=-1024) == capi.PA_ERR_SHAPE
    for name in ("q", "key", "value", "out", "slots", "pos", "cs"):
        assert call(**{name: None}) == capi.PA_ERR_NULL, name
    odd = ctypes.c_void_p(0x40001)
    for name in ("q", "key", "value", "out", "qw", "kw", "slots", "pos", "cs"):
        assert call(**{name: odd}) == capi.PA_ERR_ALIGN, name
    assert call(slots=ctypes.c_void_p(0x40004)) == capi.PA_ERR_ALIGN
    # q_out over q: only row for row
    assert call(out=ctypes.c_void_p(0x40010)) == capi.PA_ERR_SHAPE
    assert call(out=ctypes.c_void_p(0x40000 - 16)) == capi.PA_ERR_SHAPE
    assert call(out=FAKE, qs=6144) == capi.PA_ERR_SHAPE             # strided q cannot be written in place
    assert call(out=ctypes.c_void_p(0x40000), q=ctypes.c_void_p(0x90000)) == capi.PA_ERR_SHAPE    # over key and value
    assert call(T=1 << 32) == capi.PA_ERR_RANGE
    assert call(vstr=1 << 40) == capi.PA_ERR_RANGE
    assert call(pool=_pool(dtype=capi.PA_DTYPE_FP8_E4M3, ks=0.0)) == capi.PA_ERR_RANGE


def _pools(*ps):
    return (capi.PaKvPool * len(ps))(*ps)


def test_copy_pages_validation(L):
    two = lambda **k: _pools(_pool(), _pool(k=0x30000000, v=0x50000000, **k))
    call = lambda pools, n=2, src=FAKE, dst=FAKE, copies=3: L.paged_kv_copy_pages(pools, n, src, dst, copies, None)
    assert call(two(), copies=0) == capi.PA_OK
    assert call(None, n=0) == capi.PA_OK
    assert call(None) == capi.PA_ERR_NULL
    assert call(two(), n=-1) == capi.PA_ERR_SHAPE
    assert call(two(), n=1025) == capi.PA_ERR_RANGE
    assert call(two(), copies=-1) == capi.PA_ERR_SHAPE
    assert call(two(), copies=1 << 31) == capi.PA_ERR_RANGE
    assert call(two(), src=None) == capi.PA_ERR_NULL
    assert call(two(), dst=None) == capi.PA_ERR_NULL
    assert call(two(), src=ctypes.c_void_p(0x40002)) == capi.PA_ERR_ALIGN
    for other in (dict(P=65), dict(ps=8), dict(hkv=4), dict(d=64), dict(dtype=capi.PA_DTYPE_F32)):
        assert call(two(**other)) == capi.PA_ERR_SHAPE              # another geometry or type
    assert call(_pools(_pool(), _pool())) == capi.PA_ERR_SHAPE      # the same pool twice
    assert call(_pools(_pool(v=0x10000000)), n=1) == capi.PA_ERR_SHAPE          # K and V in one tensor
    size = 64 * 16 * 8 * 128 * 2
    assert call(_pools(_pool(), _pool(k=0x10000000 + size - 256, v=0x50000000))) == capi.PA_ERR_SHAPE  # overlapping
    assert call(_pools(_pool(k=0)), n=1) == capi.PA_ERR_NULL


def test_compact_validation(L):
    def call(pools=None, n=1, bt=FAKE, mb=4, sl=FAKE, B=2, base=None, ptr=FAKE, keep=FAKE, nk=5, new=OUT):
        return L.paged_kv_compact(pools if pools is not None else _pools(_pool()), n, bt, mb, sl, B, base, ptr, keep,
                                  nk, new, None)
    assert call(B=0) == capi.PA_OK
    assert call(n=0) == capi.PA_ERR_SHAPE
    assert call(B=-1) == capi.PA_ERR_SHAPE
    assert call(B=65536) == capi.PA_ERR_RANGE
    assert call(nk=-1) == capi.PA_ERR_SHAPE
    assert call(mb=0) == capi.PA_ERR_SHAPE
    assert call(mb=1 << 28) == capi.PA_ERR_RANGE
    for name in ("bt", "sl", "ptr", "keep"):
        assert call(**{name: None}) == capi.PA_ERR_NULL, name
    assert call(base=ctypes.c_void_p(0x40002)) == capi.PA_ERR_ALIGN
    assert call(new=FAKE) == capi.PA_ERR_SHAPE                      # new lengths over the inputs
    assert call(new=ctypes.c_void_p(0x40004)) == capi.PA_ERR_SHAPE
    assert call(pools=_pools(_pool(), _pool()), n=2) == capi.PA_ERR_SHAPE


# ---- the binding -----------------------------------------------------------------

def _t(dtype=torch.bfloat16):
    kp = torch.zeros(4, 16, 2, 64, dtype=dtype)
    return kp, torch.zeros_like(kp)


def test_binding_refuses_tensors_that_are_not_on_the_device():
    kp, vp = _t()
    q = torch.zeros(3, 4, 64, dtype=torch.bfloat16)
    k = torch.zeros(3, 2, 64, dtype=torch.bfloat16)
    bt, sl = torch.zeros(3, 2, dtype=torch.int32), torch.ones(3, dtype=torch.int32)
    qsl = torch.tensor([0, 1, 2, 3], dtype=torch.int32)
    for f in (lambda: capi.paged_attention_decode_window(kp, vp, q, bt, sl, 0.1, 8),
              lambda: capi.paged_attention_prefill_window(kp, vp, q, qsl, bt, sl, 0.1, 1, 8),
              lambda: capi.paged_qk_norm_rope_append(kp, vp, q, k, k, torch.zeros(3, dtype=torch.int64)),
              lambda: capi.paged_kv_copy_pages([(kp, vp)], sl, sl),
              lambda: capi.paged_kv_compact([(kp, vp)], bt, sl, qsl, sl)):
        with pytest.raises(ValueError, match="CUDA tensor"):
            f()


def test_binding_checks_window_tables():
    kp, vp = _t()
    q = torch.zeros(3, 4, 64, dtype=torch.bfloat16)
    bt, sl = torch.zeros(3, 2, dtype=torch.int32), torch.ones(3, dtype=torch.int32)
    with pytest.raises(ValueError, match="q must be"):
        capi.paged_attention_decode_window(kp, vp, q.float(), bt, sl, 0.1, 8)
    with pytest.raises(ValueError, match="block_table"):
        capi.paged_attention_decode_window(kp, vp, q, bt[:2], sl, 0.1, 8)
    with pytest.raises(ValueError, match="seq_lens"):
        capi.paged_attention_decode_window(kp, vp, q, bt, sl[:2], 0.1, 8)
    with pytest.raises(TypeError, match="int32"):
        capi.paged_attention_decode_window(kp, vp, q, bt.long(), sl, 0.1, 8)
    with pytest.raises(ValueError, match="contiguous"):
        capi.paged_attention_decode_window(kp, vp, q, bt.t().contiguous().t(), sl, 0.1, 8)
    with pytest.raises(ValueError, match="query_start_loc"):
        capi.paged_attention_prefill_window(kp, vp, q, torch.zeros(3, dtype=torch.int32), bt, sl, 0.1, 1, 8)


def test_binding_checks_rows_and_tables_of_the_append():
    kp, vp = _t()
    q, k = torch.zeros(3, 4, 64, dtype=torch.bfloat16), torch.zeros(3, 2, 64, dtype=torch.bfloat16)
    slots, pos = torch.zeros(3, dtype=torch.int64), torch.zeros(3, dtype=torch.int32)
    cs = torch.zeros(10, 64)
    f = lambda q=q, key=k, value=k, slots=slots, pos=pos, cs=cs, **kw: capi.paged_qk_norm_rope_append(
        kp, vp, q, key, value, slots, pos, cs, **kw)
    for bad in (dict(q=q.float()), dict(key=k[:2]), dict(value=torch.zeros(3, 2, 32, dtype=torch.bfloat16)),
                dict(q=q.transpose(0, 1).contiguous().transpose(0, 1)), dict(key=k[..., ::2]), dict(slots=slots[:2]),
                dict(pos=None), dict(pos=pos[:2]), dict(cs=cs[0]), dict(cs=cs.double()),
                dict(q_weight=torch.ones(64)), dict(k_weight=torch.ones(32, dtype=torch.bfloat16)),
                dict(out=torch.zeros(3, 4, 64))):
        with pytest.raises(ValueError):
            f(**bad)
    for bad in (dict(slots=slots.int()), dict(pos=pos.long())):
        with pytest.raises(TypeError):
            f(**bad)


def test_binding_checks_page_lists():
    pairs = [_t(), _t()]
    i = torch.zeros(3, dtype=torch.int32)
    bt = torch.zeros(3, 2, dtype=torch.int32)
    with pytest.raises(TypeError):
        capi.paged_kv_copy_pages(pairs, i.long(), i)
    with pytest.raises(ValueError, match="same length"):
        capi.paged_kv_copy_pages(pairs, i, i[:2])
    with pytest.raises(ValueError, match="keep_indptr"):
        capi.paged_kv_compact(pairs, bt, i, i, i)
    with pytest.raises(ValueError, match="base"):
        capi.paged_kv_compact(pairs, bt, i, torch.zeros(4, dtype=torch.int32), i, base=i[:2])
    with pytest.raises(ValueError, match="match in shape"):
        capi.make_pools([(pairs[0][0], pairs[0][1][:3])])

"""The calls on an int8 cache, of attention weights and of eviction behind a kernel that
lets its successor start early while it still writes their inputs; and the outputs and
workspaces that they make for a stream other than the current one."""
import numpy as np
import pytest
import torch

from serving_slot_mapping_gb300 import build as build_mod
from serving_slot_mapping_gb300 import capi

from _int8 import Case
from test_gpu_early_trigger import _check, late_copy  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib(cuda_device):
    build_mod.build()
    capi.lib()
    capi.device_error()  # clear


def _inputs(device, new, dtype="int8", seed=71):
    """(case, inputs, other inputs that are as valid) of an attention."""
    c = Case(new, [300, 90, 700, 40], hq=8, hkv=2, d=128, dtype=dtype, seed=seed)
    kp, vp, ks, vs, q, bt, L, qsl = c.tensors(device)
    bt = bt.clamp(0, kp.shape[0] - 1)
    clean = lambda t: torch.nan_to_num(t.float(), 1.0).clamp(-3, 3).to(t.dtype) if t.dtype != torch.int8 else t
    inputs = [clean(kp), clean(vp), q, bt, L] + ([] if ks is None else [ks.nan_to_num(1.0).clamp(0.01, 1), vs.nan_to_num(1.0).clamp(0.01, 1)])
    others = [t.flip(0).contiguous() for t in inputs]
    others[4] = torch.ones_like(L)
    return c, inputs, others, qsl


@pytest.mark.parametrize("dtype", ["bf16", "e4m3", "int8"])
def test_decode_with_weights(cuda_device, late_copy, dtype):  # noqa: F811
    c, inputs, others, _ = _inputs(cuda_device, [1, 1, 1, 1], dtype)
    msl = c.table.shape[1] * c.ps
    inputs.append(torch.rand(4, msl, device=cuda_device))
    others.append(torch.zeros(4, msl, device=cuda_device))
    m = torch.zeros(4, msl, device=cuda_device)

    def call(kp, vp, q, bt, L, *rest):
        m.zero_()
        ks, vs = rest[:2] if dtype == "int8" else (None, None)
        return capi.paged_attention_decode_mass(kp, vp, q, bt, L, c.scale, m, mass_in=rest[-1], k_scale=c.k_scale,
                                                v_scale=c.v_scale, key_scales=ks, value_scales=vs)
    ws = capi.decode_mass_workspace(4, 8, inputs[0], msl)  # noqa: F841  (the allocator's pages are there)
    bufs = [t.clone() for t in inputs]
    want = [call(*bufs).clone(), m.clone()]
    torch.cuda.synchronize()
    out, w = torch.empty_like(want[0]), capi.decode_mass_workspace(4, 8, inputs[0], msl)
    for _ in range(3):
        for b, o in zip(bufs, others):
            b.copy_(o)
        m.zero_()
        torch.cuda.synchronize()
        late_copy(list(zip(bufs, inputs)))
        ks, vs = bufs[5:7] if dtype == "int8" else (None, None)
        capi.paged_attention_decode_mass(*bufs[:5], c.scale, m, mass_in=bufs[-1], k_scale=c.k_scale, v_scale=c.v_scale,
                                         key_scales=ks, value_scales=vs, out=out, workspace=w)
        torch.cuda.synchronize()
        assert torch.equal(out, want[0]) and torch.equal(m, want[1])
    assert capi.device_error() == (0, 0)


def test_decode(cuda_device, late_copy):  # noqa: F811
    c, inputs, others, _ = _inputs(cuda_device, [1, 1, 1, 1])
    call = lambda kp, vp, q, bt, L, ks, vs: capi.paged_attention_decode_int8(kp, vp, ks, vs, q, bt, L, c.scale)
    _check(late_copy, inputs, others, call, lambda out, bufs: [out])


@pytest.mark.parametrize("new", [[20, 1, 33, 7], [500, 260, 300, 400]])
def test_prefill(cuda_device, late_copy, new):  # noqa: F811
    c, inputs, others, qsl = _inputs(cuda_device, new)
    inputs.append(qsl)
    others.append(torch.zeros_like(qsl))
    call = lambda kp, vp, q, bt, L, ks, vs, qsl: capi.paged_attention_prefill_int8(
        kp, vp, ks, vs, q, qsl, bt, L, c.scale, int(c.n.max()), out=torch.zeros_like(q))
    _check(late_copy, inputs, others, call, lambda out, bufs: [out])


@pytest.mark.parametrize("tokens", [3, 2000])
def test_append(cuda_device, late_copy, tokens):  # noqa: F811
    g = torch.Generator(device=cuda_device).manual_seed(72)
    r = lambda *s: torch.randn(*s, generator=g, device=cuda_device).bfloat16()
    codes = lambda: torch.randint(-127, 128, (200, 16, 2, 64), generator=g, device=cuda_device, dtype=torch.int8)
    scales = lambda: torch.rand(200, 1, 2, generator=g, device=cuda_device) * 0.02
    page = torch.randperm(200, generator=g, device=cuda_device)
    slots = (page[:, None] * 16 + torch.arange(16, device=cuda_device)).flatten()[5:5 + tokens]
    inputs = [codes(), codes(), scales(), scales(), r(tokens, 2, 64), r(tokens, 2, 64), slots]
    others = [t.flip(0).contiguous() for t in inputs[:6]] + [torch.full_like(slots, -1)]
    call = lambda kp, vp, ks, vs, k, v, sl: capi.paged_kv_append_int8(kp, vp, ks, vs, k, v, sl)
    _check(late_copy, inputs, others, call, lambda out, bufs: bufs[:4])


@pytest.mark.parametrize("width", [320, 20000])
def test_evict(cuda_device, late_copy, width):  # noqa: F811
    g = torch.Generator(device=cuda_device).manual_seed(73)
    m = torch.rand(2, width, generator=g, device=cuda_device)
    L = torch.tensor([width, width // 2 + 3], dtype=torch.int32, device=cuda_device)
    bt = torch.randperm(2 * width // 16, generator=g, device=cuda_device).to(torch.int32).view(2, -1)
    def rows(m, L):
        keep = torch.zeros(2 * 96, dtype=torch.int32, device=cuda_device)
        return capi.paged_kv_evict_rows(m, L, 100, 4, 20, keep=keep)
    _check(late_copy, [m, L], [m.flip(0).contiguous(), torch.full_like(L, 50)], rows, lambda out, bufs: list(out))
    _check(late_copy, [m, bt, L], [m.flip(0).contiguous(), bt.flip(0).contiguous(), torch.full_like(L, 50)],
           lambda m, bt, L: capi.paged_kv_evict_pages(m, bt, L, 16, 9, 4, 20), lambda out, bufs: list(out))


def test_made_tensors_belong_to_the_stream_of_the_call(cuda_device):
    c = Case([1] * 4, [300, 90, 700, 40], hq=8, hkv=2, d=64, seed=3)
    kp, vp, ks, vs, q, bt, L, qsl = c.tensors(cuda_device)
    m = torch.rand(4, c.table.shape[1] * c.ps, device=cuda_device)
    w = torch.zeros_like(m)
    calls = {
        "decode": lambda s: [capi.paged_attention_decode_int8(kp, vp, ks, vs, q, bt, L, c.scale, stream=s)],
        "prefill": lambda s: [capi.paged_attention_prefill_int8(kp, vp, ks, vs, q, qsl, bt, L, c.scale, 1, stream=s)],
        "mass": lambda s: [capi.paged_attention_decode_mass(kp, vp, q, bt, L, c.scale, w, key_scales=ks, value_scales=vs, stream=s)],
        "rows": lambda s: list(capi.paged_kv_evict_rows(m, L, 50, 4, 8, stream=s)),
        "pages": lambda s: list(capi.paged_kv_evict_pages(m, bt, L, c.ps, 5, 4, 8, stream=s)),
    }
    side = torch.cuda.Stream()
    for name, call in calls.items():
        want = [t.clone() for t in call(None)]
        n = int(want[0][-1]) if name == "rows" else None
        torch.cuda.synchronize()
        gone = [torch.empty_like(t) for t in want]      # memory that the current stream frees
        at = {t.data_ptr() for t in gone}
        del gone
        for stream in (side, side.cuda_stream):
            out = call(stream)
            assert not at & {t.data_ptr() for t in out}, name
            side.synchronize()
            for i, (x, y) in enumerate(zip(out, want)):
                cut = n if name == "rows" and i == 1 else None
                assert torch.equal(x[:cut], y[:cut]), name
    assert capi.device_error() == (0, 0)

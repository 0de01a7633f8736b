"""Inputs that a kernel writes which lets the next kernel on the stream start early
(programmatic dependent launch): the windowed layer's calls read them only once it
is done.  The writer here triggers at once, waits 200 us and then copies every
input into place; before that the buffers hold other, equally valid inputs."""
import ctypes
import subprocess

import numpy as np
import pytest
import torch

from serving_slot_mapping_gb300 import build as build_mod
from serving_slot_mapping_gb300 import capi

from _window import Case

pytestmark = pytest.mark.gpu

WRITER = r"""
#include <cuda_runtime.h>
#include <stdint.h>
struct Copies { const unsigned char* src[16]; unsigned char* dst[16]; long long bytes[16]; int n; };
__global__ void late(Copies c) {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  unsigned long long t0, t;
  asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t0));
  for (int i = 0; i < 1000000; ++i) {  // bounded whatever the timer does
    asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t));
    if (t - t0 > 200000) break;
  }
  for (int k = 0; k < c.n; ++k)
    for (long long i = threadIdx.x; i < c.bytes[k]; i += blockDim.x) c.dst[k][i] = c.src[k][i];
}
extern "C" int late_copy(const Copies* c, void* stream) {
  late<<<1, 256, 0, (cudaStream_t)stream>>>(*c);
  return (int)cudaGetLastError();
}
"""


class _Copies(ctypes.Structure):
    _fields_ = [("src", ctypes.c_void_p * 16), ("dst", ctypes.c_void_p * 16), ("bytes", ctypes.c_longlong * 16),
                ("n", ctypes.c_int)]


@pytest.fixture(scope="module")
def late_copy(cuda_device, tmp_path_factory):
    build_mod.build()
    capi.lib()
    capi.device_error()  # clear
    d = tmp_path_factory.mktemp("writer")
    (d / "writer.cu").write_text(WRITER)
    subprocess.run([build_mod.nvcc_path(), *build_mod.ARCH, "-O2", "-shared", "-Xcompiler", "-fPIC", "-o",
                    str(d / "writer.so"), str(d / "writer.cu")], check=True)
    f = ctypes.CDLL(str(d / "writer.so")).late_copy
    f.argtypes = [ctypes.POINTER(_Copies), ctypes.c_void_p]

    def copy(pairs):
        c = _Copies()
        c.n = len(pairs)
        for i, (dst, src) in enumerate(pairs):
            assert dst.numel() * dst.element_size() == src.numel() * src.element_size()
            c.src[i], c.dst[i], c.bytes[i] = src.data_ptr(), dst.data_ptr(), src.numel() * src.element_size()
        assert f(ctypes.byref(c), torch.cuda.current_stream().cuda_stream) == 0

    return copy


def _check(late_copy, inputs, others, call, results):
    """`call(*inputs)` and the tensors it leaves, with `inputs` in place and with
    `others` in place until the writer's copies land."""
    bufs = [t.clone() for t in inputs]
    expected = [t.clone() for t in results(call(*bufs), bufs)]
    torch.cuda.synchronize()
    for _ in range(3):
        for b, o in zip(bufs, others):
            b.copy_(o)
        torch.cuda.synchronize()
        late_copy(list(zip(bufs, inputs)))
        got = results(call(*bufs), bufs)
        torch.cuda.synchronize()
        for g, e in zip(got, expected):
            assert torch.equal(g.view(torch.uint8), e.view(torch.uint8))
    assert capi.device_error() == (0, 0)


def _attention(device, new, dtype, seed):
    c = Case(new, [300, 90, 700, 40], 100, 4, hq=8, hkv=2, d=128, dtype=dtype, seed=seed)
    c.table = np.where(c.table < 0, 0, np.minimum(c.table, len(c.kp) - 1))  # valid in the other order too
    dev = lambda a: torch.from_numpy(np.ascontiguousarray(a)).to(device)
    nan = lambda t: torch.nan_to_num(t.float(), 1.0).to(t.dtype)           # either table may see any slot
    inputs = [nan(c.kp).to(device), nan(c.vp).to(device), c.q.to(device), dev(c.table), dev(c.lens), dev(c.qsl)]
    others = [t.flip(0) for t in inputs[:4]] + [torch.ones_like(inputs[4]), inputs[5].clone()]
    return c, inputs, others


@pytest.mark.parametrize("dtype", ["bf16", "e4m3", "f32"])
def test_windowed_decode(cuda_device, late_copy, dtype):
    c, inputs, others = _attention(cuda_device, [1, 1, 1, 1], dtype, 61)
    call = lambda kp, vp, q, bt, lens, qsl: capi.paged_attention_decode_window(
        kp, vp, q, bt, lens, c.scale, 100, 4, max_seq_len=c.table.shape[1] * 16)
    _check(late_copy, inputs, others, call, lambda out, bufs: [out])


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("new", [[20, 1, 33, 7], [500, 260, 300, 400]])  # clusters; items in turn
def test_windowed_prefill(cuda_device, late_copy, dtype, new):
    c, inputs, others = _attention(cuda_device, new, dtype, 62)
    others[5] = torch.zeros_like(inputs[5])
    call = lambda kp, vp, q, bt, lens, qsl: capi.paged_attention_prefill_window(
        kp, vp, q, qsl, bt, lens, c.scale, int(c.n.max()), 100, 4, max_seq_len=c.table.shape[1] * 16,
        out=torch.zeros_like(q))
    _check(late_copy, inputs, others, call, lambda out, bufs: [out])


@pytest.mark.parametrize("tokens", [3, 3000])  # registers; the ring
def test_norm_rope_append(cuda_device, late_copy, tokens):
    g = torch.Generator(device=cuda_device).manual_seed(63)
    r = lambda *s: torch.randn(*s, generator=g, device=cuda_device).bfloat16()
    slots = torch.randperm(200 * 16, generator=g, device=cuda_device)[:tokens]
    pos = torch.randint(0, 64, (tokens,), generator=g, device=cuda_device, dtype=torch.int32)
    cs = torch.randn(64, 64, generator=g, device=cuda_device)
    inputs = [r(200, 16, 2, 64), r(200, 16, 2, 64), r(tokens, 8, 64), r(tokens, 2, 64), r(tokens, 2, 64), slots, pos, cs,
              r(64), r(64)]
    others = [t.flip(0) for t in inputs[:7]] + [t * 2 for t in inputs[7:]]
    others[5] = torch.full_like(slots, -1)
    call = lambda kp, vp, q, k, v, sl, ps, cs, qw, kw: capi.paged_qk_norm_rope_append(kp, vp, q, k, v, sl, ps, cs, qw, kw)
    _check(late_copy, inputs, others, call, lambda out, bufs: [out, bufs[0], bufs[1]])


def test_page_moves(cuda_device, late_copy):
    g = torch.Generator(device=cuda_device).manual_seed(64)
    r = lambda: torch.randn(40, 16, 2, 64, generator=g, device=cuda_device).bfloat16()
    i32 = lambda *a: torch.tensor(a, device=cuda_device, dtype=torch.int32)
    inputs = [r(), r(), i32(0, 1, 2), i32(30, 31, 32)]
    others = [inputs[1], inputs[0], i32(-1, -1, -1), i32(5, 6, 7)]
    call = lambda kp, vp, src, dst: capi.paged_kv_copy_pages([(kp, vp)], src, dst)
    _check(late_copy, inputs, others, call, lambda out, bufs: bufs[:2])
    keep = i32(*range(5, 60, 3), *range(0, 30, 2))
    inputs = [r(), r(), i32(*range(20)).view(2, 10), i32(100, 30), i32(0, 19, 34), keep]
    others = [inputs[1], inputs[0], inputs[2].flip(0), i32(1, 1), i32(0, 0, 0), torch.zeros_like(keep)]
    call = lambda kp, vp, bt, lens, ptr, keep: capi.paged_kv_compact([(kp, vp)], bt, lens, ptr, keep)
    _check(late_copy, inputs, others, call, lambda out, bufs: [out, bufs[0], bufs[1]])

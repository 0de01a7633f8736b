"""Outputs and workspaces that the windowed layer's calls make themselves, for a
stream other than the current one: their memory is never one that kernels queued on
the current stream still use."""
import pytest
import torch

from serving_slot_mapping_gb300 import build as build_mod
from serving_slot_mapping_gb300 import capi

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib(cuda_device):
    build_mod.build()
    capi.lib()
    capi.device_error()  # clear


def _calls(dev):
    """name: (call(stream) -> the tensor it makes, a tensor of that size and type)."""
    kp = torch.randn(64, 16, 2, 64, device=dev).bfloat16()
    vp, q = torch.randn_like(kp), torch.randn(300, 8, 64, device=dev).bfloat16()
    k = torch.randn(300, 2, 64, device=dev).bfloat16()
    bt = torch.arange(300, device=dev, dtype=torch.int32).remainder(64).view(300, 1).contiguous()
    one = torch.full((300,), 9, device=dev, dtype=torch.int32)
    qsl = torch.arange(301, device=dev, dtype=torch.int32)
    slots = torch.arange(300, device=dev)
    ptr = torch.zeros(301, device=dev, dtype=torch.int32)
    keep = torch.zeros(0, device=dev, dtype=torch.int32)
    ws = capi.decode_workspace(300, 8, kp)
    pools = capi.make_pools([(kp.clone(), vp.clone())])
    return {
        "decode": (lambda s: capi.paged_attention_decode_window(kp, vp, q, bt, one, 0.1, 4, workspace=ws, stream=s), q),
        "prefill": (lambda s: capi.paged_attention_prefill_window(kp, vp, q, qsl, bt, one, 0.1, 1, 4, stream=s), q),
        "append": (lambda s: capi.paged_qk_norm_rope_append(kp, vp, q, k, k, slots, stream=s), q),
        "compact": (lambda s: capi.paged_kv_compact(pools, bt, one, ptr, keep, base=one, stream=s), one),
    }


@pytest.mark.parametrize("name", ["decode", "prefill", "append", "compact"])
def test_made_tensors_belong_to_the_stream_of_the_call(cuda_device, name):
    call, like = _calls(cuda_device)[name]
    side = torch.cuda.Stream()
    expected = call(None).clone()
    torch.cuda.synchronize()
    other = torch.empty_like(like)      # memory that the current stream frees ...
    at = other.data_ptr()
    del other
    for stream in (side, side.cuda_stream):
        out = call(stream)              # ... is not the call's on the other stream
        assert out.data_ptr() != at
        side.synchronize()
        assert torch.equal(out, expected)
    # an output that the current stream still reads is not handed out again
    out = call(side)
    torch.cuda.current_stream().wait_stream(side)
    at = out.data_ptr()
    torch.cuda._sleep(1 << 29)
    copy = out.clone()
    del out
    again = call(side)
    assert again.data_ptr() != at
    torch.cuda.synchronize()
    assert torch.equal(copy, expected) and torch.equal(again, expected)
    assert capi.device_error() == (0, 0)


def test_a_made_workspace_belongs_to_the_stream_of_the_call(cuda_device, monkeypatch):
    """The plain kernels that a wide window runs on use it."""
    kp = torch.randn(64, 16, 2, 64, device=cuda_device).bfloat16()
    vp, q = torch.randn_like(kp), torch.randn(3, 8, 64, device=cuda_device).bfloat16()
    bt = torch.arange(60, device=cuda_device, dtype=torch.int32).view(3, 20)
    lens = torch.full((3,), 300, device=cuda_device, dtype=torch.int32)
    made, real = [], capi.decode_workspace
    monkeypatch.setattr(capi, "decode_workspace", lambda *a, **k: (made.append(torch.cuda.current_stream().cuda_stream),
                                                                   real(*a, **k))[1])
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    out = capi.paged_attention_decode_window(kp, vp, q, bt, lens, 0.1, 1000, stream=side)
    torch.cuda.synchronize()
    assert made == [side.cuda_stream]
    assert torch.equal(out, capi.paged_attention_decode(kp, vp, q, bt, lens, 0.1))

"""e4m3 codes of keys under scales near 2^-100, where x - q scale is no longer a
multiple of fp32's smallest step: the code is still that of the IEEE quotient."""
import numpy as np
import pytest
import torch

from serving_slot_mapping_gb300 import build as build_mod
from serving_slot_mapping_gb300 import capi

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("scale,key", [
    # the quotient is one fp32 step above 2^-10, half the smallest code's value: code 1, not 0
    ("0x1.ffffdep-100", "0x1.ffffep-110"), ("0x1.ffffc2p-100", "0x1.ffffc4p-110"),
    # around the change of method, and scales at which it was right
    ("0x1.ffff7ap-101", "0x1.ffff7cp-111"), ("0x1.ffffdep-90", "0x1.ffffep-100"), ("0x1.ffffdep-91", "0x1.ffffep-101"),
    ("0x1.3p-92", "0x1.3p-102"), ("0x1.ffffdep-40", "0x1.ffffep-50")])
def test_codes_of_keys_are_those_of_the_quotient(cuda_device, scale, key, interleaved):
    build_mod.build()
    scale, key = np.float32(float.fromhex(scale)), np.float32(float.fromhex(key))
    near = [key, *(np.nextafter(key, np.float32(k)) for k in (0, 1)), key * 2, key * 3, key * 5, key * 1000, -key]
    x = torch.tensor(np.array(near, dtype=np.float32))
    T = len(near)
    cos_sin = torch.zeros(T, 64)
    cos_sin[:, :32] = x[:, None]        # 1 turned by "cosine" x and sine 0 is x, exactly
    one = torch.ones(T, 1, 64, dtype=torch.bfloat16, device=cuda_device)
    kp, vp = (torch.zeros(1, 16, 1, 64, device=cuda_device).to(torch.float8_e4m3fn) for _ in range(2))
    q = capi.paged_qk_norm_rope_append(kp, vp, one, one, one, torch.arange(T, device=cuda_device),
                                       torch.arange(T, dtype=torch.int32, device=cuda_device), cos_sin.to(cuda_device),
                                       interleaved=interleaved, k_scale=float(scale))
    torch.cuda.synchronize()
    assert capi.device_error() == (0, 0)
    assert torch.equal(q.cpu(), x.bfloat16()[:, None, None].expand(T, 1, 64))
    codes = (x / torch.tensor(scale)).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    got = kp.view(torch.uint8).view(16, 64)[:T].cpu()
    assert torch.equal(got, codes[:, None].expand(T, 64))

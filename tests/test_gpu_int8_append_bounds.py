"""The append into int8 pools at the ends of its range, and its quotients: every one that
a new block can meet, and a sample of those of blocks in use, against the oracle's fp32
division."""
import numpy as np
import pytest
import torch

from serving_slot_mapping_gb300 import build as build_mod
from serving_slot_mapping_gb300 import capi

from test_gpu_int8_append import State

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib(cuda_device):
    build_mod.build()
    capi.lib()
    capi.device_error()  # clear


def _bf16(bits):
    return torch.tensor(bits, dtype=torch.int32).to(torch.int16).view(torch.bfloat16)


# 127.5 times the largest scale, 2^40, is a bf16 value, and its quotient a tie
LARGEST = int(torch.tensor(127.5 * 2.0 ** 40).to(torch.bfloat16).view(torch.int16))


@pytest.mark.parametrize("step", [-2, -1, 0, 1, 2])
@pytest.mark.parametrize("slot", [16, 21], ids=["new", "used"])
@pytest.mark.parametrize("d", [64, 128])
def test_values_next_to_the_largest_scale(cuda_device, step, slot, d):
    """Magnitudes around 127.5 times 2^40, of both signs: codes of at most 127."""
    x = _bf16([LARGEST + step])
    s = State(P=4, d=d)
    k, v = s.rows(2), s.rows(2)
    k[0, 0, 3], k[0, 1, 5], v[1, 1, 7], v[1, 0, 0] = x, -x, x, -x
    s.check(cuda_device, [slot, slot + 1], key=k, value=v)
    assert s.codes[0].min() >= -127 and abs(int(s.codes[0][1, slot % 16, 0, 3])) in (126, 127)


def test_every_quotient_of_a_new_block(cuda_device):
    """A new block's scale is a / 127 for a bf16 a: with each of the 128 significands of a,
    every bf16 value of the nine binades up to a (below them the code is 0 or 1 / 2 of one)."""
    rows, slots = [], []
    for m in range(128):
        a = (130 << 7) | m                                     # a bf16 in [8, 16)
        x = _bf16(list(range(a - 9 * 128, a + 1)))             # up to a itself
        x = torch.cat([x, x[-1:].expand(-len(x) % 64)])
        rows.append(torch.cat([x[-1:].expand(64)[None], x.view(-1, 64)]))
        n = len(rows[-1])
        assert n <= 32
        slots += [32 * m + i for i in range(n)]
    rows = torch.cat(rows)[:, None]
    s = State(P=128, ps=32, blk=32, hkv=1)
    s.check(cuda_device, slots, key=rows, value=-rows)


def test_quotients_of_blocks_in_use(cuda_device):
    """Scales of every fp32 significand (a random sample) that stay as they are."""
    P = 512
    s = State(P=P, hkv=2)
    rng = np.random.default_rng(1)
    for t in range(2):
        s.scales[t] = rng.integers(0x3c000000, 0x3d000000, size=s.scales[t].shape, dtype=np.int32).view(np.float32)
    slots = [16 * p + i for p in range(P) for i in range(1, 16)]
    top = [np.repeat(sc[:, 0], 15, axis=0)[:, :, None] * np.float32(126.5) for sc in s.scales]
    k, v = (torch.from_numpy((rng.uniform(-1, 1, size=t.shape[:2] + (64,)) * t).astype(np.float32)).to(torch.bfloat16)
            for t in top)
    before = [sc.copy() for sc in s.scales]
    s.check(cuda_device, slots, key=k, value=v)
    assert all(np.array_equal(x, y) for x, y in zip(before, s.scales))

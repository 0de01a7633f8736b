"""The append into int8 pools: codes and scales bit for bit those of the oracle."""
import numpy as np
import pytest
import torch

import oracle
from serving_slot_mapping_gb300 import build as build_mod
from serving_slot_mapping_gb300 import capi

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib(cuda_device):
    build_mod.build()
    capi.lib()
    capi.device_error()  # clear


class State:
    def __init__(self, P=12, ps=16, blk=16, hkv=2, d=64, seed=0):
        rng = np.random.default_rng(seed)
        self.shape = (P, ps, hkv, d)
        self.codes = [rng.integers(-127, 128, size=self.shape, dtype=np.int8) for _ in range(2)]
        self.scales = [rng.uniform(0.005, 0.03, size=(P, ps // blk, hkv)).astype(np.float32) for _ in range(2)]
        self.rng = rng

    def rows(self, T, sigma=1.0):
        x = torch.from_numpy(self.rng.standard_normal((T,) + self.shape[2:]).astype(np.float32) * sigma)
        return x.to(torch.bfloat16)

    def check(self, device, slots, key=None, value=None, strided=False, error=(0, 0), **k):
        T = len(slots)
        key = self.rows(T) if key is None else key
        value = self.rows(T) if value is None else value
        dev = [torch.from_numpy(a.copy()).to(device) for a in self.codes + self.scales]
        kd, vd = key.to(device), value.to(device)
        if strided:
            both = torch.cat([torch.zeros_like(kd), kd, vd], 1).contiguous()
            n = key.shape[1]
            kd, vd = both[:, n:2 * n], both[:, 2 * n:]
        capi.paged_kv_append_int8(dev[0], dev[1], dev[2], dev[3], kd, vd, torch.tensor(slots, dtype=torch.int64, device=device), **k)
        torch.cuda.synchronize()
        assert capi.device_error() == error
        ok = [s if s < self.shape[0] * self.shape[1] else -1 for s in slots]
        for i, x in enumerate((key, value)):
            codes, scales = oracle.kv_int8.append_int8(self.codes[i], self.scales[i], x.float().numpy(), ok)
            assert np.array_equal(dev[2 + i].cpu().numpy(), scales)
            assert np.array_equal(dev[i].cpu().numpy(), codes)
            self.codes[i], self.scales[i] = codes, scales


@pytest.mark.parametrize("hkv,d", [(1, 64), (2, 64), (8, 128), (3, 128)])
@pytest.mark.parametrize("ps,blk", [(16, 16), (64, 16), (32, 32), (256, 256), (128, 64)])
def test_runs_and_single_tokens(cuda_device, hkv, d, ps, blk):
    s = State(P=6, ps=ps, blk=blk, hkv=hkv, d=d)
    # a sequence over pages 3, 1, 4 from the middle of a block on, then another from the start of one
    first = [3 * ps + i for i in range(5, ps)] + [ps + i for i in range(ps)] + [4 * ps + i for i in range(3)]
    s.check(cuda_device, first + [i for i in range(ps - 1)], strided=True)
    for i in range(3, 3 + 4):     # then token by token, growing and not
        s.check(cuda_device, [4 * ps + i, ps - 1 if i == 3 else -1], key=s.rows(2, 2.0 ** (i - 4)))


def test_padding_and_order(cuda_device):
    s = State(ps=32, blk=16)
    s.check(cuda_device, [-1, 5, -1, -1, 40, 42, 41, -5, 70, 100, 96, -1])
    s.check(cuda_device, [-1, -2, -3])
    s.check(cuda_device, list(range(20, 14, -1)))    # a block's slots in any order


def test_a_new_block_forgets_its_scale(cuda_device):
    s = State()
    s.scales[0][2] = 1e30
    s.check(cuda_device, [32, 33, 34])
    assert (s.scales[0][2] < 1).all()


def test_growing_scales_encode_the_block_anew(cuda_device):
    s = State(hkv=4, d=128)
    before = [c.copy() for c in s.codes]
    s.check(cuda_device, [20], key=s.rows(1, 100.0), value=s.rows(1, 0.001))
    assert (s.codes[0][1, :4] != before[0][1, :4]).any() and (s.codes[1][1, :4] == before[1][1, :4]).all()


@pytest.mark.parametrize("value", [0.0, float("nan"), float("inf"), -float("inf"), 3e38, 1e-30, 1e-38])
@pytest.mark.parametrize("slot", [16, 21])
def test_odd_values(cuda_device, value, slot):
    s = State(P=4)
    k, v = s.rows(2), s.rows(2)
    k[0, 0, 3], v[1, 1] = value, value
    s.check(cuda_device, [slot, slot + 1], key=k, value=v)


@pytest.mark.parametrize("old", [0.0, float("nan"), float("inf"), -1.0, 1e-30])
def test_odd_scales_of_a_block_in_use(cuda_device, old):
    s = State(P=4)
    s.scales[0][1], s.scales[1][1] = old, old
    s.check(cuda_device, [20])


def test_rounding_is_to_nearest_even_of_the_fp32_quotient(cuda_device):
    """Quotients on and next to ties: every bf16 of a few binades against scales of the
    form a / 127."""
    x = torch.arange(0x3c00, 0x4480, dtype=torch.int32).to(torch.int16).view(torch.bfloat16)
    n = x.numel() // 64
    x = x[:n * 64].view(n, 1, 64)
    for top in (381.0, 127.0, 1016.0, 890.0):
        s = State(P=n // 16 + 2, hkv=1)
        rows = torch.cat([torch.full((1, 1, 64), top, dtype=torch.bfloat16), x])
        for t in range(0, n, 15):        # every block begins with the row that sets its scale
            part = torch.cat([rows[:1], rows[1 + t:1 + t + 15]])
            s.check(cuda_device, [16 * (t // 15) + i for i in range(part.shape[0])], key=part, value=-part) if t % 45 == 0 else None


def test_slots_out_of_range_are_skipped(cuda_device):
    s = State(P=3)
    s.check(cuda_device, [4, 5, 48, 6, 7], error=(2, 48))


@pytest.mark.parametrize("gap", [1, 2, 30, 31])
def test_padding_inside_a_block(cuda_device, gap):
    s = State(P=4, blk=32, ps=32)
    pads = [-1] * gap
    s.check(cuda_device, [35] + pads + [36, 37] + pads + [32] + pads + [70])
    s.check(cuda_device, pads + [40] + pads + [41] + pads + [99, 98] + pads)


def test_many_tokens(cuda_device):
    s = State(P=300, ps=16, hkv=8, d=128)
    perm = s.rng.permutation(300)
    slots = [int(p) * 16 + i for p in perm[:280] for i in range(16)]
    s.check(cuda_device, slots[5:-3] + [-1] * 9, strided=True)
    # a decode step: one token in each of many blocks
    s.check(cuda_device, [int(p) * 16 + int(s.rng.integers(0, 16)) for p in perm])


def test_captured_and_replayed(cuda_device):
    s = State(P=8, hkv=2)
    dev = [torch.from_numpy(a.copy()).to(cuda_device) for a in s.codes + s.scales]
    key, value = s.rows(4).to(cuda_device), s.rows(4).to(cuda_device)
    slots = torch.tensor([3, 17, 33, 50], device=cuda_device)
    call = lambda: capi.paged_kv_append_int8(*dev, key, value, slots)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    for step in range(3):
        key.copy_(s.rows(4, 1.0 + step))
        value.copy_(s.rows(4, 3.0 - step))
        slots.copy_(torch.tensor([4 + step, 18 + step, 34 + step, 51 + step]))
        g.replay()
        torch.cuda.synchronize()
        for i, x in enumerate((key, value)):
            s.codes[i], s.scales[i] = oracle.kv_int8.append_int8(s.codes[i], s.scales[i], x.float().cpu().numpy(), slots.tolist())
            assert np.array_equal(dev[i].cpu().numpy(), s.codes[i]) and np.array_equal(dev[2 + i].cpu().numpy(), s.scales[i])
    assert capi.device_error() == (0, 0)

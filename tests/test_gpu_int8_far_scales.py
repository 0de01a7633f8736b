"""Attention over int8 pools whose blocks' scales lie far apart, row by row: what a row
does not see, or hardly weighs, takes nothing from what it does."""
import numpy as np
import pytest
import torch

from serving_slot_mapping_gb300 import build as build_mod
from serving_slot_mapping_gb300 import capi

from _int8_rows import RowCase

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib(cuda_device):
    build_mod.build()
    capi.lib()
    capi.device_error()  # clear


def last_blocks(c, scales, power):
    """The scale of the last block of every sequence, 2^power times as large."""
    for b, L in enumerate(c.lens.tolist()):
        if L > 0:
            j = L - 1
            scales[c.seen[b, j // c.ps], j % c.ps // c.blk] *= 2.0 ** power


def spread(c, scales, sigma, seed=3):
    rng = np.random.default_rng(seed)
    scales *= torch.from_numpy(np.exp(sigma * rng.standard_normal(tuple(scales.shape))).astype(np.float32))


PREFILLS = [([130, 20, 33], [300, 40, 0]), ([257], [0]), ([60, 1], [1500, 100])]


@pytest.mark.parametrize("power", [16, 20, 26, 38])
@pytest.mark.parametrize("new,cached", PREFILLS)
@pytest.mark.parametrize("d", [64, 128])
def test_rows_before_a_block_of_large_values(cuda_device, power, new, cached, d):
    """A later block's V scale is 2^power times the others': rows before it see none of it."""
    c = RowCase(new, cached, hq=4, hkv=2, d=d, seed=power)
    last_blocks(c, c.vs, power)
    c.check(capi, cuda_device)


@pytest.mark.parametrize("power", [8, 20, 30])
@pytest.mark.parametrize("new,cached", PREFILLS[:2])
def test_rows_before_a_block_of_large_keys(cuda_device, power, new, cached):
    c = RowCase(new, cached, hq=4, hkv=2, d=64, seed=power)
    last_blocks(c, c.ks, power)
    exp = c.rows()
    out = c.run(capi, cuda_device)
    c.compare(out, exp, judged=0.5)


@pytest.mark.parametrize("sigma", [3.0, 7.0])
@pytest.mark.parametrize("ps,blk,d", [(16, 16, 128), (32, 32, 64), (128, 64, 64), (256, 256, 128)])
def test_prefill_of_values_far_apart(cuda_device, sigma, ps, blk, d):
    c = RowCase([100, 20], [400, 40], hq=4, hkv=2, d=d, ps=ps, blk=blk, seed=5)
    spread(c, c.vs, sigma)
    c.check(capi, cuda_device)


@pytest.mark.parametrize("sigma", [2.0, 4.0])
def test_prefill_of_keys_far_apart(cuda_device, sigma):
    """K scales over many powers of two, the scores of ordinary size."""
    c = RowCase([100, 20], [400, 40], hq=4, hkv=2, d=64, seed=6)
    spread(c, c.ks, sigma)
    K, _ = c.values()
    c.scale = 6.0 / (np.linalg.norm(K, axis=-1).max() * 8.0)
    c.check(capi, cuda_device)


def test_prefill_of_long_items_far_apart(cuda_device):
    """Many key tiles a sequence, shared by clusters and in turn."""
    c = RowCase([40, 3, 70], [1000, 2500, 100], hq=2, hkv=1, d=64, ps=32, blk=32, seed=7)
    spread(c, c.vs, 4.0)
    last_blocks(c, c.vs, 20)
    c.check(capi, cuda_device)


@pytest.mark.parametrize("d", [64, 128])
def test_prefill_of_many_items_far_apart(cuda_device, d):
    """More items than SMs, in turn on persistent CTAs, some sequences without a new row."""
    rng = np.random.default_rng(2)
    c = RowCase(rng.integers(0, 120, size=60), rng.integers(0, 400, size=60), hq=8, hkv=4, d=d, seed=4)
    spread(c, c.vs, 4.0)
    last_blocks(c, c.vs, 20)
    c.check(capi, cuda_device)


@pytest.mark.parametrize("scale", [0.0, -0.2])
def test_prefill_scales_of_the_softmax_far_apart(cuda_device, scale):
    c = RowCase([50], [90], hq=4, hkv=2, d=64, scale=scale, seed=8)
    spread(c, c.vs, 4.0)
    last_blocks(c, c.vs, 24)
    c.check(capi, cuda_device)


@pytest.mark.parametrize("room", [0, 2400], ids=["clusters", "cut"])
@pytest.mark.parametrize("sigma", [3.0, 7.0])
@pytest.mark.parametrize("hq,hkv,d", [(8, 2, 64), (16, 1, 128)])
def test_decode_of_values_far_apart(cuda_device, room, sigma, hq, hkv, d):
    lens = np.asarray([300, 40, 1000, 17])
    c = RowCase(np.ones_like(lens), lens - 1, hq=hq, hkv=hkv, d=d, seed=5, room=room)
    spread(c, c.vs, sigma)
    c.check(capi, cuda_device)


def test_a_later_token_leaves_earlier_rows_as_they_are(cuda_device):
    """The same chunk with and without large values in its last block: the same bits in the
    rows before it."""
    c = RowCase([96], [64], hq=4, hkv=2, d=64, seed=9)
    a = c.run(capi, cuda_device)
    last_blocks(c, c.vs, 24)
    b = c.run(capi, cuda_device)
    assert not (a[:80] != b[:80]).any()     # the last block's 16 rows aside
    c.compare(b, judged=0.9)

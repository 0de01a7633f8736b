"""Attention weights over bf16 and e4m3 pools with block-table entries out of range: the
keys of such pages take no part and have weight 0, whatever the shared memory that they
would have come to holds."""
import numpy as np
import pytest
import torch

import oracle
from serving_slot_mapping_gb300 import build as build_mod
from serving_slot_mapping_gb300 import capi

from _int8 import Case
from _parity import bits, to_f64

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib(cuda_device):
    build_mod.build()
    capi.lib()
    capi.device_error()  # clear


def decode(lens, **k):
    lens = np.asarray(lens)
    return Case(np.ones_like(lens), lens - 1, **k)


def run(c, device, before=None, decay=1.0):
    kp, vp, ks, vs, q, bt, L, _ = c.tensors(device)
    m = torch.full((len(c.lens), c.max_len + 3), -7.0, device=device)
    # a decode of NaN keys and values first: what the stages of shared memory may hold
    nan = torch.full_like(kp.float(), float("nan")).to(kp.dtype)
    good = torch.zeros_like(bt)
    capi.paged_attention_decode_mass(nan, nan, q, good, L, c.scale, m.clone(), max_seq_len=c.max_len)
    out = capi.paged_attention_decode_mass(kp, vp, q, bt, L, c.scale, m, mass_in=before, decay=decay, max_seq_len=c.max_len,
                                           k_scale=c.k_scale, v_scale=c.v_scale, key_scales=ks, value_scales=vs,
                                           out=torch.full_like(q, float("nan")))
    torch.cuda.synchronize()
    assert capi.device_error()[0] == 1
    return out, m.cpu().numpy()


def gone(c, b):
    """Positions of sequence b whose page is out of range."""
    return np.concatenate([np.arange(m * c.ps, min((m + 1) * c.ps, int(c.lens[b]))) for bb, m in c.bad if bb == b] or
                          [np.zeros(0, dtype=int)]).astype(int)


def check(c, device, before=None, decay=1.0):
    """Tolerance of a weight: its score's error, from fp32 sums of d products (at most (d + 4)
    2^-24 sum_d |q_d K_d| scale, on the weight and on its row's sum), the exponential's and
    the sums' (2^-20), relative to the weight; the masses before add 2^-22 of the result."""
    out, m = run(c, device, None if before is None else torch.from_numpy(before).to(device), decay)
    c.compare(out)
    K, _ = c.values()
    q = to_f64(bits(c.q))
    table, lens = c._compact(None)
    want = oracle.evict.key_weights(K, q, table, lens, c.scale)
    for b, L in enumerate(c.lens.tolist()):
        w = np.zeros(L)
        w[np.setdiff1d(np.arange(L), gone(c, b))] = want[b]
        e = 2 * (c.d + 4) * 2.0 ** -24 * abs(c.scale) * np.abs(q[b]).sum(-1).max() * np.abs(K).max() + 2.0 ** -20
        all_ = w + (0.0 if before is None else decay * before[b, :L].astype(np.float64))
        assert (np.abs(m[b, :L] - all_) <= e * w + 2.0 ** -22 * np.abs(all_)).all()
        if before is None:
            assert (m[b, gone(c, b)] == 0).all()
        assert (m[b, L:] == -7.0).all()


BAD = [[(0, 0)], [(0, 2)], [(1, 0), (1, 1), (0, 3)], [(0, 0), (1, 2), (2, 1)]]


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("ps", [8, 16, 32])
@pytest.mark.parametrize("bad", BAD)
def test_pages(cuda_device, dtype, ps, bad):
    check(decode([6 * ps + 3, 5 * ps, 300], ps=ps, blk=ps, hq=8, hkv=2, d=64, dtype=dtype, bad=bad, seed=ps), cuda_device)


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("hq,hkv,d", [(32, 8, 128), (1, 1, 64), (32, 1, 128), (64, 2, 64), (12, 3, 128), (16, 16, 64)])
@pytest.mark.parametrize("ps", [8, 16])
def test_head_layouts(cuda_device, dtype, hq, hkv, d, ps):
    check(decode([100, 700, 64, 41], ps=ps, blk=ps, hq=hq, hkv=hkv, d=d, dtype=dtype, bad=[(0, 1), (1, 0), (1, 3), (2, 2)],
                 seed=hq), cuda_device)


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("ps", [8, 16, 64])
def test_long_sequences(cuda_device, dtype, ps):
    """Parts of a sequence on many CTAs, some of them with nothing but bad pages."""
    bad = [(0, m) for m in range(3, 3 + 640 // ps)] + [(1, 2)]
    check(decode([6000, 333], ps=ps, blk=ps, hq=32, hkv=8, d=128, dtype=dtype, bad=bad, seed=3), cuda_device)


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
def test_masses_before_are_kept(cuda_device, dtype):
    c = decode([96, 100], hq=8, hkv=2, d=64, dtype=dtype, bad=[(0, 1), (1, 0)])
    before = np.random.default_rng(0).random((2, c.max_len + 3)).astype(np.float32)
    check(c, cuda_device, before=before, decay=0.5)


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("ps", [8, 16])
def test_a_sequence_without_a_page_in_range(cuda_device, dtype, ps):
    c = decode([2 * ps, 50, ps], ps=ps, blk=ps, hq=8, hkv=2, d=64, dtype=dtype, bad=[(0, 0), (0, 1), (2, 0)])
    out, m = run(c, cuda_device)
    assert (out[0] == 0).all() and (out[2] == 0).all() and torch.isfinite(out).all()
    assert (m[0, :2 * ps] == 0).all() and (m[2, :ps] == 0).all() and abs(m[1, :50].sum() - 8) < 1e-3

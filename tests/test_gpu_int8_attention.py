"""Attention over int8 pools with a scale for each block of tokens and KV head,
against the oracle on the values that the codes stand for."""
import numpy as np
import pytest
import torch

from serving_slot_mapping_gb300 import build as build_mod
from serving_slot_mapping_gb300 import capi

from _int8 import Case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib(cuda_device):
    build_mod.build()
    capi.lib()
    capi.device_error()  # clear


def decode(room, lens, **k):
    lens = np.asarray(lens)
    return Case(np.ones_like(lens), lens - 1, room=room // (k.get("ps", 16) // 16), **k)


# both kernels: short parts on clusters; the cut that all CTAs share
both = pytest.mark.parametrize("room", [0, 2400], ids=["clusters", "cut"])
RAGGED = [1, 15, 16, 17, 0, 33, 64, 129, 500, 31]


@both
@pytest.mark.parametrize("hq,hkv", [(1, 1), (8, 8), (8, 2), (12, 3), (16, 4), (32, 8), (16, 1), (32, 1), (64, 2), (128, 4)])
@pytest.mark.parametrize("d", [64, 128])
def test_decode_head_layouts(cuda_device, room, hq, hkv, d):
    decode(room, RAGGED, hq=hq, hkv=hkv, d=d, seed=hq + d).check(capi, cuda_device)


@both
@pytest.mark.parametrize("ps,blk", [(16, 16), (32, 16), (32, 32), (64, 16), (128, 64), (256, 256), (1024, 32)])
def test_decode_pages_and_blocks(cuda_device, room, ps, blk):
    decode(room, RAGGED + [1500], ps=ps, blk=blk, hkv=4, seed=ps + blk).check(capi, cuda_device)


@both
@pytest.mark.parametrize("lens", [[1], [16], [4096], [0, 0, 0], [1] * 40, list(range(1, 400, 7)), [5000, 3, 700]])
def test_decode_batches(cuda_device, room, lens):
    decode(room, lens, hq=32, hkv=8, d=128, seed=len(lens)).check(capi, cuda_device)


@both
def test_decode_many_short_sequences(cuda_device, room):
    decode(room, np.random.default_rng(3).integers(0, 60, size=600), hq=16, hkv=2, d=64).check(capi, cuda_device)


@both
@pytest.mark.parametrize("scale", [0.0, -0.2, 1.0])
def test_decode_scale(cuda_device, room, scale):
    decode(room, RAGGED, scale=scale).check(capi, cuda_device)


@both
@pytest.mark.parametrize("spread", [0.0, 3.0, 7.0])
def test_decode_scales_far_apart(cuda_device, room, spread):
    """Blocks whose scales differ by many powers of two, in K and in V."""
    decode(room, [300, 40, 1000], spread=spread, seed=5, scale=0.02).check(capi, cuda_device)


@both
def test_decode_first_block_with_tiny_values(cuda_device, room):
    """Most of the weight on a block whose V is almost 0 (a first token): the others'
    weights keep their precision and the row's sum its size."""
    c = decode(room, [200], hq=4, hkv=1, d=64, seed=9)
    p = c.table[0, 0]
    c.vs[p] *= 2.0 ** -20
    c.kp[p, 0] = torch.sign(c.q[0, :1].float()).mul(127).to(torch.int8)
    c.ks[p] = 0.1
    c.check(capi, cuda_device)


@both
@pytest.mark.parametrize("value", [0.0, -3.0, float("nan"), 2.0 ** -60, 2.0 ** 60, float("inf")])
def test_decode_scales_are_clamped(cuda_device, room, value):
    c = decode(room, [40, 70], hq=4, hkv=2, seed=2)
    c.vs[c.table[1, 1]] = value
    if not value > 1:
        c.ks[c.table[0, 1]] = value
    c.check(capi, cuda_device)


@both
@pytest.mark.parametrize("bad", [[(0, 0)], [(0, 3)], [(1, 1), (1, 2)], [(0, 0), (1, 0)]])
@pytest.mark.parametrize("hkv", [2, 8])
def test_decode_keys_of_bad_pages_take_no_part(cuda_device, room, bad, hkv):
    c = decode(room, [100, 75, 16], hq=16, hkv=hkv, d=128 if hkv == 8 else 64, bad=bad)
    c.check(capi, cuda_device, error=(1, None))


@both
def test_decode_of_nothing_but_a_bad_page_gives_zeros(cuda_device, room):
    c = decode(room, [16, 20], bad=[(0, 0)])
    out = c.run(capi, cuda_device)
    torch.cuda.synchronize()
    assert capi.device_error()[0] == 1
    assert (out[0] == 0).all() and torch.isfinite(out).all()


PREFILLS = [([5], [0]), ([1, 1, 2], [0, 300, 7]), ([300, 17, 130], [0, 1000, 128]), ([64, 1, 0, 33], [0, 0, 5, 63]),
            ([257], [1]), ([700, 40], [300, 2000])]


@pytest.mark.parametrize("new,cached", PREFILLS)
@pytest.mark.parametrize("d", [64, 128])
def test_prefill_batches(cuda_device, new, cached, d):
    Case(new, cached, hq=8, hkv=2, d=d, seed=sum(new)).check(capi, cuda_device)


@pytest.mark.parametrize("hq,hkv", [(1, 1), (4, 4), (12, 3), (32, 8), (16, 1), (32, 1)])
def test_prefill_head_layouts(cuda_device, hq, hkv):
    Case([70, 9], [50, 0], hq=hq, hkv=hkv, d=128, seed=hq).check(capi, cuda_device)


@pytest.mark.parametrize("ps,blk", [(16, 16), (32, 16), (32, 32), (64, 64), (128, 16), (256, 256), (512, 128)])
def test_prefill_pages_and_blocks(cuda_device, ps, blk):
    Case([150, 3], [600, 129], ps=ps, blk=blk, seed=ps).check(capi, cuda_device)


def test_prefill_many_items(cuda_device):
    """More items than SMs: the persistent loop, its rings and both sizes of tiles."""
    rng = np.random.default_rng(1)
    Case(rng.integers(0, 300, size=40), rng.integers(0, 200, size=40), hq=16, hkv=4, d=64, seed=4).check(capi, cuda_device)


@pytest.mark.parametrize("scale", [0.0, -0.2, 0.5])
def test_prefill_scale(cuda_device, scale):
    Case([100], [60], scale=scale).check(capi, cuda_device)


@pytest.mark.parametrize("spread", [3.0, 7.0])
def test_prefill_scales_far_apart(cuda_device, spread):
    Case([130, 20], [300, 40], spread=spread, seed=5, scale=0.02).check(capi, cuda_device)


def test_prefill_rows_without_a_key_are_zeros(cuda_device):
    c = Case([20, 5], [-8, 3], seed=6)
    out = c.check(capi, cuda_device)
    assert (out[:8] == 0).all()


@pytest.mark.parametrize("new,cached,bad", [([40], [100], [(0, 1)]), ([300], [700], [(0, 0), (0, 20)]),
                                            ([300, 2000, 40, 900], [500, 0, 60, 400], [(0, 3)])])
def test_prefill_keys_of_bad_pages_take_no_part(cuda_device, new, cached, bad):
    """Compared with a sequence that never had those pages' keys, row by row (rows that
    lie before the page see none of it)."""
    c = Case(new, cached, bad=bad, seed=8)
    out = c.run(capi, cuda_device)
    torch.cuda.synchronize()
    assert capi.device_error()[0] == 1
    gone = {m for _, m in bad}
    keep = [m for m in range(-(-int(c.lens[0]) // c.ps)) if m not in gone]
    c.seen[0, :len(keep)] = c.seen[0, keep]
    c.lens[0] -= c.ps * len(gone)
    c.bad = []
    c.compare(out)


@pytest.mark.parametrize("msl", [300, 40000], ids=["clusters", "cut"])
def test_replays_on_other_inputs_and_two_calls_at_once(cuda_device, msl):
    """A captured decode and prefill replayed on other lengths, tables, codes and scales;
    two calls in flight with workspaces of their own give the same bits."""
    a = decode(0, [100, 7, 300], hq=32, hkv=8, d=128, seed=1)
    b = decode(0, [250, 300, 1], hq=32, hkv=8, d=128, seed=2)
    width = max(a.table.shape[1], b.table.shape[1], msl // 16)
    pages = max(a.kp.shape[0], b.kp.shape[0])
    def padded(c):
        grow = lambda t, n, v: torch.cat([t, torch.full((n - t.shape[0],) + t.shape[1:], v, dtype=t.dtype)]) if t is not None else None
        t = c.tensors("cpu")
        table = torch.full((3, width), -7, dtype=torch.int32)
        table[:, :t[5].shape[1]] = t[5]
        return [x.to(cuda_device) for x in (grow(t[0], pages, 1), grow(t[1], pages, 1), grow(t[2], pages, 1.0),
                                            grow(t[3], pages, 1.0), t[4], table, t[6])]
    ta, tb = padded(a), padded(b)
    eager = [capi.paged_attention_decode_int8(*t, a.scale, max_seq_len=msl) for t in (ta, tb)]
    live = [t.clone() for t in ta]
    ws, out = capi.decode_workspace(3, 32, live[0]), torch.empty_like(eager[0])
    call = lambda: capi.paged_attention_decode_int8(*live, a.scale, max_seq_len=msl, out=out, workspace=ws)
    call()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    for t, want in ((tb, eager[1]), (ta, eager[0]), (tb, eager[1])):
        for x, y in zip(live, t):
            x.copy_(y)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    outs = []
    for _ in range(5):
        outs.append((capi.paged_attention_decode_int8(*ta, a.scale, max_seq_len=msl, stream=s1),
                     capi.paged_attention_decode_int8(*tb, a.scale, max_seq_len=msl, stream=s2)))
    torch.cuda.synchronize()
    for x, y in outs:
        assert torch.equal(x, eager[0]) and torch.equal(y, eager[1])
    assert capi.device_error() == (0, 0)


@pytest.mark.parametrize("new,cached", [([150], [3000]), ([40] * 30, [900] * 30), ([2000, 3, 700], [0, 2500, 100])])
def test_prefill_long_items(cuda_device, new, cached):
    """Items of many key tiles, alone on a CTA, shared by a cluster, and several in turn."""
    Case(new, cached, hq=16, hkv=4, d=64, ps=32, blk=32, seed=7).check(capi, cuda_device)


def test_prefill_many_sequences(cuda_device):
    """More sequences than a warp ranks at once, most of them short, some empty."""
    rng = np.random.default_rng(5)
    Case(rng.integers(0, 40, size=300), rng.integers(0, 300, size=300), hq=8, hkv=2, d=64, seed=3).check(capi, cuda_device)


def test_prefill_first_block_with_tiny_values(cuda_device):
    """Most of the weight on a block whose V is almost 0, in a tile of its own."""
    c = Case([70], [200], hq=4, hkv=1, d=64, ps=128, blk=128, seed=9)
    p = c.table[0, 0]
    c.vs[p] *= 2.0 ** -20
    c.ks[p] *= 3.0
    c.check(capi, cuda_device)


@pytest.mark.parametrize("value", [0.0, float("nan"), 2.0 ** -60, 2.0 ** 60])
def test_prefill_scales_are_clamped(cuda_device, value):
    c = Case([30], [60], hq=4, hkv=2, seed=2)
    c.vs[c.table[0, 1]] = value
    if not value > 1:
        c.ks[c.table[0, 3]] = value
    c.check(capi, cuda_device)


def test_prefill_replayed_on_other_inputs(cuda_device):
    """Captured once, replayed on other lengths, chunks, tables, codes and scales: the bits
    of an eager call (sequences shared by clusters, whose parts depend on the launch alone)."""
    cases = [Case(n, c, hq=8, hkv=2, d=128, seed=i) for i, (n, c) in
             enumerate([([40, 0, 100], [300, 5, 0]), ([1, 130, 9], [0, 200, 333]), ([50, 50, 40], [0, 0, 0])])]
    pages, width = max(c.kp.shape[0] for c in cases), max(c.table.shape[1] for c in cases)
    live = None
    for k, c in enumerate(cases):
        t = c.tensors("cpu")
        grow = lambda x, v: torch.cat([x, torch.full((pages - x.shape[0],) + x.shape[1:], v, dtype=x.dtype)])
        table = torch.full((3, width), -7, dtype=torch.int32)
        table[:, :t[5].shape[1]] = t[5]
        q = torch.zeros(150, 8, 128, dtype=torch.bfloat16)
        q[:t[4].shape[0]] = t[4]
        now = [x.to(cuda_device) for x in (grow(t[0], 1), grow(t[1], 1), grow(t[2], 1.0), grow(t[3], 1.0), q, t[7], table, t[6])]
        want = capi.paged_attention_prefill_int8(*now, c.scale, 130, max_seq_len=340, out=torch.zeros_like(now[4]))
        if live is None:
            live, out = [x.clone() for x in now], torch.zeros_like(now[4])
            torch.cuda.synchronize()
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g):
                capi.paged_attention_prefill_int8(*live, c.scale, 130, max_seq_len=340, out=out)
        for x, y in zip(live, now):
            x.copy_(y)
        out.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)
        n = int(c.n.sum())
        assert (out[n:] == 0).all()          # rows behind the last sequence
        c.compare(out[:n])
    assert capi.device_error() == (0, 0)

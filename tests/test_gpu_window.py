"""Sliding-window attention (paged_attention_decode_window,
paged_attention_prefill_window) against the oracle, element by element (see
_window.py for the inputs and the tolerance)."""
import numpy as np
import pytest
import torch

from serving_slot_mapping_gb300 import build as build_mod
from serving_slot_mapping_gb300 import capi

from _window import Case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib(cuda_device):
    build_mod.build()
    capi.lib()
    capi.device_error()  # clear


def _decode(lens, *a, **k):
    lens = np.asarray(lens)
    return Case((lens > 0).astype(int), np.maximum(lens - 1, 0), *a, **k)


# empty, one key, block and page edges, around window + sinks, long
LENS = [0, 1, 2, 15, 16, 17, 33, 64, 100, 101, 128, 129, 255, 700, 1500]


@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (16, 0), (16, 16), (17, 4), (100, 0), (100, 1), (33, 100),
                                          (96, 33), (1499, 0), (1000, 700), (5000, 4)])
def test_decode_windows(cuda_device, window, sinks):
    _decode(LENS, window, sinks, seed=window + sinks).check(capi, cuda_device)


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("hq,hkv,d,ps", [(32, 8, 128, 16), (32, 8, 128, 8), (8, 8, 64, 8), (16, 2, 64, 64),
                                         (32, 1, 128, 16), (32, 1, 128, 8), (4, 4, 128, 256), (40, 8, 128, 32),
                                         (64, 2, 128, 16), (64, 4, 64, 16), (24, 1, 64, 16), (3, 1, 128, 16),
                                         (12, 4, 64, 16), (128, 4, 128, 16)])
def test_decode_layouts(cuda_device, dtype, hq, hkv, d, ps):
    _decode([0, 1, 40, 333, 77, 600], 90, 5, hq=hq, hkv=hkv, d=d, ps=ps, dtype=dtype, seed=hq + d + ps).check(
        capi, cuda_device)


@pytest.mark.parametrize("ps,dtype", [(1, "bf16"), (4, "bf16"), (12, "bf16"), (16, "f32"), (5, "f32")])
def test_decode_core_path(cuda_device, ps, dtype):
    _decode([0, 1, 7, 40, 130, 300], 50, 6, ps=ps, dtype=dtype, seed=ps).check(capi, cuda_device)


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
def test_decode_many_short_and_few_long(cuda_device, dtype):
    rng = np.random.default_rng(3)
    # hundreds of sequences, one CTA each; 3 long ones: clusters of 8
    _decode(rng.integers(0, 400, 300), 64, 4, hq=8, hkv=2, d=64, dtype=dtype, seed=9).check(capi, cuda_device)
    # over 608 CTAs: three of them an SM, with shorter rings
    _decode(rng.integers(0, 300, 420), 100, 4, hq=8, hkv=2, d=128, dtype=dtype, seed=12).check(capi, cuda_device)
    _decode([5000, 4000, 3], 2500, 20, hq=32, hkv=8, d=128, dtype=dtype, seed=10).check(capi, cuda_device)
    _decode([5000, 4000, 3], 2500, 20, hq=32, hkv=1, d=128, dtype=dtype, seed=11).check(capi, cuda_device)


def test_decode_infinities_in_hidden_slots(cuda_device):
    _decode(LENS, 40, 3, seed=5, poison=float("inf")).check(capi, cuda_device)
    _decode(LENS, 40, 3, seed=6, ps=8, poison=-float("inf")).check(capi, cuda_device)


@pytest.mark.parametrize("dtype", ["bf16", "e4m3", "f32"])
@pytest.mark.parametrize("scale", [0.0, -0.2, 1.5])
def test_scales(cuda_device, dtype, scale):
    _decode([0, 1, 40, 333, 77, 600], 90, 5, hq=6, hkv=2, dtype=dtype, seed=31, scale=scale).check(capi, cuda_device)
    Case([60, 1, 30], [300, 0, 70], 90, 5, hq=6, hkv=2, dtype=dtype, seed=32, scale=scale).check(capi, cuda_device)


def test_decode_a_wide_window_is_the_plain_call(cuda_device):
    c = _decode([1, 50, 400], 400, 0, seed=2)
    out = c.run(capi, cuda_device)
    kp, vp, q = c.args
    dev = lambda a: torch.from_numpy(a).to(cuda_device)
    plain = capi.paged_attention_decode(kp, vp, q, dev(c.table), dev(c.lens), c.scale, max_seq_len=400)
    torch.cuda.synchronize()
    assert torch.equal(out.view(torch.int16), plain.view(torch.int16))


def test_decode_upper_bound_of_lengths_and_garbage_workspace(cuda_device):
    c = _decode([9, 300, 1200], 128, 4, hq=32, hkv=8, d=128, seed=3)
    n = capi.decode_workspace_size(3, 32, 8, 128)
    for fill in (0, 255):
        ws = torch.full((n,), fill, dtype=torch.uint8, device=cuda_device)
        c.check(capi, cuda_device, workspace=ws, max_seq_len=1200)
        # the table may be longer than any sequence, and the bound loose
        c.table = np.concatenate([c.table, np.full((3, 40), -1, dtype=np.int32)], axis=1)
        c.check(capi, cuda_device, workspace=ws, max_seq_len=c.table.shape[1] * 16)


def test_decode_captured_and_replayed(cuda_device):
    c = _decode([30, 700, 2000, 0], 333, 7, hq=32, hkv=8, d=128, seed=4)
    eager = c.check(capi, cuda_device)
    dev = lambda a: torch.from_numpy(a).to(cuda_device)
    kp, vp, q = c.args
    table, lens, out = dev(c.table), dev(c.lens), torch.zeros_like(q)
    ws = capi.decode_workspace(4, 32, kp)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        capi.paged_attention_decode_window(kp, vp, q, table, lens, c.scale, 333, 7, max_seq_len=2000, out=out,
                                           workspace=ws)
    for _ in range(3):
        out.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out.view(torch.int16), eager.view(torch.int16))
    # the same graph serves other lengths
    lens.copy_(torch.tensor([0, 700, 1000, 0], dtype=torch.int32))
    c.table[2, :] = c.table[1, 0]
    table.copy_(dev(c.table))
    c2 = c
    c2.lens = np.array([0, 700, 1000, 0], dtype=np.int32)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out[1].view(torch.int16), eager[1].view(torch.int16))
    assert torch.all(out[0] == 0) and torch.all(out[3] == 0)
    capi.device_error()


def test_decode_bad_pages_are_recorded(cuda_device):
    c = _decode([300, 40], 100, 4, seed=8)
    c.table[0, 0] = 1 << 29                       # a sink's page
    c.run(capi, cuda_device)
    torch.cuda.synchronize()
    assert capi.device_error() == (1, 1 << 29)
    out = _decode([300, 40], 100, 4, seed=8).check(capi, cuda_device)
    assert torch.isfinite(out).all()


# ---- prefill ----------------------------------------------------------------

NEW = [1, 7, 130, 40, 300, 16, 260]
CACHED = [0, 500, 0, 90, 1000, 3, 128]


@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 3), (16, 0), (64, 64), (100, 1), (128, 4), (33, 140),
                                          (300, 0), (1000, 130), (9000, 4)])
def test_prefill_windows(cuda_device, window, sinks):
    Case(NEW, CACHED, window, sinks, hq=4, hkv=2, d=64, seed=window + sinks).check(capi, cuda_device)


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("hq,hkv,d,ps", [(8, 2, 128, 16), (8, 2, 128, 8), (2, 2, 64, 64), (4, 1, 128, 128),
                                         (4, 1, 64, 256), (5, 1, 128, 32), (32, 1, 128, 16)])
def test_prefill_layouts(cuda_device, dtype, hq, hkv, d, ps):
    Case([60, 1, 200], [300, 0, 70], 90, 5, hq=hq, hkv=hkv, d=d, ps=ps, dtype=dtype, seed=hq + d + ps).check(
        capi, cuda_device)


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("hq,hkv,d,ps", [(8, 2, 128, 16), (2, 2, 64, 8), (4, 1, 128, 128), (5, 1, 64, 32), (16, 1, 128, 256)])
def test_prefill_few_rows_long_windows(cuda_device, dtype, hq, hkv, d, ps):
    """Few items with many key tiles each: their parts are computed by the CTAs of
    a cluster and joined (some CTAs of a cluster without a tile, rows without a key)."""
    Case([33, 1, 70, 12], [900, 1500, 0, -12], 1300, 40, hq=hq, hkv=hkv, d=d, ps=ps, dtype=dtype, seed=d + ps).check(
        capi, cuda_device)
    Case([64], [5000], 3000, 4, hq=hq, hkv=hkv, d=d, ps=ps, dtype=dtype, seed=d + ps + 1).check(capi, cuda_device)


@pytest.mark.parametrize("dtype,ps", [("bf16", 1), ("bf16", 12), ("f32", 16)])
def test_prefill_core_path(cuda_device, dtype, ps):
    Case([20, 1, 50], [60, 0, 10], 30, 3, dtype=dtype, ps=ps, seed=ps).check(capi, cuda_device)


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
def test_prefill_rows_without_keys_and_infinities(cuda_device, dtype):
    # sequences with fewer keys than new rows: the rows below position 0 give 0
    poison = float("inf") if dtype == "bf16" else float("nan")
    c = Case([40, 300, 9], [-10, -280, -9], 12, 2, dtype=dtype, seed=4, poison=poison)
    out = c.check(capi, cuda_device)
    assert torch.all(out[:10] == 0) and torch.all(out[-9:] == 0)


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("hq,hkv,d", [(8, 8, 64), (16, 4, 128)])
def test_prefill_many_items(cuda_device, dtype, hq, hkv, d):
    """Several hundred (sequence, head, row tile) items, so that a CTA walks
    through several; sequences without new tokens, with fewer keys than rows
    (tiles that see no key between others) and chunks of more than 32 of them."""
    rng = np.random.default_rng(21)
    new = rng.integers(0, 40, 90)
    cached = rng.integers(-30, 200, 90)
    new[40:75] = 0                                  # a whole stretch of sequences without rows
    new[[3, 80]] = [150, 290]
    Case(new, cached, 24, 3, hq=hq, hkv=hkv, d=d, dtype=dtype, seed=22).check(capi, cuda_device)


def test_prefill_long_rows_many_tiles(cuda_device):
    # hundreds of 256-row tiles of few sequences
    Case([1500, 700], [100, 2000], 70, 5, hq=32, hkv=2, d=64, seed=23).check(capi, cuda_device)


def test_prefill_rows_past_the_batch_are_left(cuda_device):
    c = Case([20, 31], [40, 0], 16, 2, seed=6)
    full = torch.full((60, 8, 64), 7.0, dtype=torch.bfloat16, device=cuda_device)
    c.check(capi, cuda_device, out=full[:51])
    assert torch.all(full[51:] == 7.0)


def test_prefill_a_wide_window_is_the_plain_call(cuda_device):
    c = Case([70, 300], [100, 0], 300, 0, seed=7)
    out = c.run(capi, cuda_device)
    kp, vp, q = c.args
    dev = lambda a: torch.from_numpy(a).to(cuda_device)
    plain = capi.paged_attention_prefill(kp, vp, q, dev(c.qsl), dev(c.table), dev(c.lens), c.scale, max_q_len=300,
                                         max_seq_len=300)
    torch.cuda.synchronize()
    assert torch.equal(out.view(torch.int16), plain.view(torch.int16))


def test_on_a_stream_of_its_own_without_buffers(cuda_device):
    c = _decode([30, 700, 2000], 333, 7, hq=32, hkv=8, d=128, seed=14)
    c.run(capi, cuda_device)
    torch.cuda.synchronize()
    kp, vp, q = c.args
    dev = lambda a: torch.from_numpy(a).to(cuda_device)
    table, lens, side = dev(c.table), dev(c.lens), torch.cuda.Stream()
    torch.cuda.synchronize()
    y, tol = c.oracle()
    outs = []
    for _ in range(6):  # workspace and output are made by the call and used on the other stream
        outs.append(capi.paged_attention_decode_window(kp, vp, q, table, lens, c.scale, 333, 7, max_seq_len=2000,
                                                       stream=side))
        torch.full((1 << 20,), 255, dtype=torch.uint8, device=cuda_device)  # would reuse freed memory
    torch.cuda.synchronize()
    for out in outs:
        assert (np.abs(out.float().cpu().numpy().astype(np.float64) - y) <= tol).all()


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("bad", [1 << 29, -7])
def test_prefill_bad_pages_are_recorded(cuda_device, dtype, bad):
    def case():
        return Case([60, 300, 20], [0, 200, 5], 70, 4, dtype=dtype, seed=41)

    good = case().check(capi, cuda_device)
    c = case()
    c.table[1, 0] = bad                           # a sink's page of the middle sequence
    out = c.run(capi, cuda_device)
    torch.cuda.synchronize()
    assert capi.device_error() == (1, bad)
    # the sequences beside it are what they were, and so is the next call
    assert torch.equal(out[:60].view(torch.int16), good[:60].view(torch.int16))
    assert torch.equal(out[360:].view(torch.int16), good[360:].view(torch.int16))
    again = case().check(capi, cuda_device)
    assert torch.equal(again.view(torch.int16), good.view(torch.int16))


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("new,cached", [([130, 40, 300], [0, 900, 128]), ([20], [2000])])   # persistent grid; clusters
def test_prefill_captured_and_replayed(cuda_device, dtype, new, cached):
    c = Case(new, cached, 333, 7, hq=8, hkv=2, d=128, dtype=dtype, seed=42)
    eager = c.check(capi, cuda_device)
    dev = lambda a: torch.from_numpy(a).to(cuda_device)
    kp, vp, q = c.args
    qsl, table, lens, out = dev(c.qsl), dev(c.table), dev(c.lens), torch.zeros_like(q)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        capi.paged_attention_prefill_window(kp, vp, q, qsl, table, lens, c.scale, int(c.n.max()), 333, 7,
                                            max_seq_len=int(c.lens.max()), out=out, k_scale=c.k_scale,
                                            v_scale=c.v_scale)
    for _ in range(3):
        out.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out.view(torch.int16), eager.view(torch.int16))
    # the same graph serves a batch whose last sequence has no rows
    last = int(c.n[-1])
    out.fill_(7.0)
    qsl[-1] = qsl[-2]
    graph.replay()
    torch.cuda.synchronize()
    rows = int(c.n[:-1].sum())
    assert torch.equal(out[:rows].view(torch.int16), eager[:rows].view(torch.int16))
    assert torch.all(out[rows:rows + last] == 7.0)
    assert capi.device_error() == (0, 0)


def test_two_calls_at_once(cuda_device):
    """Decodes and prefills on two streams at a time, each with clusters or a grid
    that fills the GPU, give what they give alone, bit for bit."""
    cases = [_decode([3000, 2000, 5], 1500, 4, hq=32, hkv=8, d=128, seed=43),
             Case([300, 40, 700], [200, 1000, 0], 200, 4, hq=16, hkv=4, d=128, seed=44)]
    alone = [c.check(capi, cuda_device) for c in cases]
    calls = []
    for c in cases:
        dev = lambda a: torch.from_numpy(a).to(cuda_device)
        kp, vp, q = c.args
        msl = int(c.lens.max())
        if c.is_decode:
            args = (kp, vp, q, dev(c.table), dev(c.lens), c.scale, c.window, c.sinks)
            calls.append((capi.paged_attention_decode_window, args, dict(max_seq_len=msl)))
        else:
            args = (kp, vp, q, dev(c.qsl), dev(c.table), dev(c.lens), c.scale, int(c.n.max()), c.window, c.sinks)
            calls.append((capi.paged_attention_prefill_window, args, dict(max_seq_len=msl)))
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    outs = []
    for i in range(20):
        for k, st in enumerate(streams):
            f, args, kw = calls[(k + i) % 2]
            outs.append(((k + i) % 2, f(*args, stream=st, **kw)))
    torch.cuda.synchronize()
    assert capi.device_error() == (0, 0)
    for k, out in outs:
        assert torch.equal(out.view(torch.int16), alone[k].view(torch.int16))

"""One captured windowed call serves other batches: lengths, tables, chunk bounds,
queries and pool rows changed between replays, every row compared bit for bit with
an eager call on the same inputs and with the oracle."""
import numpy as np
import pytest
import torch

from serving_slot_mapping_gb300 import build as build_mod
from serving_slot_mapping_gb300 import capi

from _parity import bits, to_f64
from _window import Case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib(cuda_device):
    build_mod.build()
    capi.lib()
    capi.device_error()  # clear


class Chunks(Case):
    is_decode = False  # a prefill, whatever the chunks


def _replays(device, cases, rows, pages, blocks, max_q_len):
    """`cases`: batches of one number of sequences; their rows, pools and tables are
    copied into buffers of `rows` rows, `pages` pages and `blocks` entries a row."""
    c = cases[0]
    hkv, d = c.kp.shape[2:]
    kp, vp = (torch.zeros(pages, c.ps, hkv, d, device=device).to(c.kp.dtype) for _ in range(2))
    q, out = (torch.zeros(rows, c.q.shape[1], d, dtype=c.q.dtype, device=device) for _ in range(2))
    table = torch.zeros(len(c.lens), blocks, dtype=torch.int32, device=device)
    lens = torch.zeros(len(c.lens), dtype=torch.int32, device=device)
    qsl = torch.zeros(len(c.lens) + 1, dtype=torch.int32, device=device)
    kw = dict(max_seq_len=blocks * c.ps, k_scale=c.k_scale, v_scale=c.v_scale)
    if max_q_len is None:
        ws = capi.decode_workspace(rows, c.q.shape[1], kp)
        call = lambda out: capi.paged_attention_decode_window(kp, vp, q, table, lens, c.scale, c.window, c.sinks, out=out,
                                                              workspace=ws, **kw)
    else:
        call = lambda out: capi.paged_attention_prefill_window(kp, vp, q, qsl, table, lens, c.scale, max_q_len, c.window,
                                                               c.sinks, out=out, **kw)
    call(out)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(out)
    raw = lambda t: t.view(torch.uint8) if t.dtype == torch.float8_e4m3fn else t
    for c in [*cases, cases[0]]:
        raw(kp)[:len(c.kp)].copy_(raw(c.kp))
        raw(vp)[:len(c.vp)].copy_(raw(c.vp))
        q[:len(c.q)].copy_(c.q)
        table.fill_(-1)
        table[:, :c.table.shape[1]].copy_(torch.from_numpy(c.table))
        lens.copy_(torch.from_numpy(c.lens))
        qsl.copy_(torch.from_numpy(c.qsl))
        out.fill_(7.0)
        eager = call(torch.full_like(out, 7.0))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out.view(torch.int16), eager.view(torch.int16))
        n = len(c.q)
        if max_q_len is not None:
            assert torch.all(out[n:] == 7.0)
        y, tol = c.oracle()
        err = np.abs(to_f64(bits(out[:n])) - y)
        assert (err <= tol).all(), f"error {err.max():.3e}"
        assert capi.device_error() == (0, 0)


@pytest.mark.parametrize("dtype,hq,hkv,d", [("bf16", 32, 8, 128), ("e4m3", 32, 1, 128), ("bf16", 8, 2, 64)])
def test_decode(cuda_device, dtype, hq, hkv, d):
    rng = np.random.default_rng(71)
    batches = [[30, 700, 2000, 0], [0, 700, 1000, 0], [1, 2, 3, 4], [2000, 1999, 340, 333], rng.integers(0, 2000, 4)]
    cases = [Case((np.asarray(b) > 0).astype(int), np.maximum(np.asarray(b) - 1, 0), 333, 7, hq=hq, hkv=hkv, d=d,
                  dtype=dtype, seed=72 + i) for i, b in enumerate(batches)]
    _replays(cuda_device, cases, 4, max(len(c.kp) for c in cases), 130, None)


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("batches,rows,bound", [
    ([([130, 40, 300], [0, 900, 128]), ([1, 1, 1], [0, 40, 1200]), ([0, 300, 0], [5, 0, 0]), ([256, 2, 64], [64, 700, 0])],
     600, 300),
    ([([20], [1100]), ([64], [0]), ([1], [1200]), ([0], [900])], 64, 64)])       # clusters
def test_prefill(cuda_device, dtype, batches, rows, bound):
    cases = [Chunks(n, m, 333, 7, hq=8, hkv=2, d=128, dtype=dtype, seed=81 + i) for i, (n, m) in enumerate(batches)]
    _replays(cuda_device, cases, rows, max(len(c.kp) for c in cases), 90, bound)

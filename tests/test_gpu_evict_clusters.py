"""Evictions on clusters of each size, against the oracle."""
import numpy as np
import pytest
import torch

from serving_slot_mapping_gb300 import build as build_mod
from serving_slot_mapping_gb300 import capi

from test_gpu_mass_evict import check_pages, check_rows, masses

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib(cuda_device):
    build_mod.build()
    capi.lib()
    capi.device_error()  # clear


# on 152 SMs: 16 CTAs a sequence, 8 (where a GPU cannot place 16 these are what remains), 4, 2
@pytest.mark.parametrize("B,width", [(1, 140000), (10, 70000), (20, 35000), (40, 17000)])
def test_rows(cuda_device, B, width):
    lens = [width - 7 * b for b in range(B)]
    check_rows(cuda_device, masses(B, width, B, ties=0.3), lens, width // 5, 4, 100)


@pytest.mark.parametrize("B,pages", [(1, 9000), (10, 5000), (20, 2500)])
def test_pages(cuda_device, B, pages):
    ps = 16
    lens = [pages * ps - 37 * b - 5 for b in range(B)]
    check_pages(cuda_device, masses(B, pages * ps, 3, ties=0.4), lens, ps, pages // 4, 4, 100)


def test_captured_on_sixteen(cuda_device):
    """Long sequences in a captured graph, replayed on other masses and lengths."""
    width, ps = 140000, 16
    m = torch.empty(1, width, device=cuda_device)
    L = torch.empty(1, dtype=torch.int32, device=cuda_device)
    bt = torch.arange(width // ps, dtype=torch.int32, device=cuda_device).view(1, -1)
    m.fill_(1.0)
    L.fill_(width)
    rows = [t.clone() for t in capi.paged_kv_evict_rows(m, L, 9000, 4, 100)]
    pages = [t.clone() for t in capi.paged_kv_evict_pages(m, bt, L, ps, 700, 4, 100)]
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        capi.paged_kv_evict_rows(m, L, 9000, 4, 100, keep_indptr=rows[0], keep=rows[1], base=rows[2], new_mass=rows[3])
        capi.paged_kv_evict_pages(m, bt, L, ps, 700, 4, 100, new_block_table=pages[0], new_seq_lens=pages[1],
                                  new_mass=pages[2])
    for seed, n in enumerate((width, 100001, 8999)):
        m.copy_(torch.from_numpy(masses(1, width, seed)))
        L.fill_(n)
        for t in rows + pages:
            t.zero_()
        g.replay()
        torch.cuda.synchronize()
        kept = int(rows[0][-1])
        for got, want in zip(rows, capi.paged_kv_evict_rows(m, L, 9000, 4, 100)):
            cut = kept if got is rows[1] else None
            assert torch.equal(got[:cut], want[:cut])
        for got, want in zip(pages, capi.paged_kv_evict_pages(m, bt, L, ps, 700, 4, 100)):
            assert torch.equal(got, want)
    assert capi.device_error() == (0, 0)

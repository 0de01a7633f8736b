"""Evictions on clusters of each size, against the oracle."""
import numpy as np
import pytest

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

"""Evictions of rows whose width comes close to 2^31: refused before anything is launched
(no GPU).  The kernels count rows in 32 bits, and their last steps go past the end."""
import ctypes

import pytest

from serving_slot_mapping_gb300 import build as build_mod
from serving_slot_mapping_gb300 import capi

LIMIT = 2 ** 31 - 65536
P = [ctypes.c_void_p((i + 1) << 40) for i in range(6)]  # far apart; never read


@pytest.fixture(scope="module")
def L():
    build_mod.build()
    return capi.lib()


def rows(L, width, B=1, **k):
    return L.paged_kv_evict_rows(P[0], width, P[1], B, width, k.get("budget", 100), 4, 8, P[2], k.get("keep", P[3]), 1 << 20, P[4],
                                 k.get("new", P[5]), width, None)


def pages(L, width, blocks, ps, B=1, **k):
    return L.paged_kv_evict_pages(P[0], width, P[1], blocks, P[2], B, width, ps, 100, 4, 8, P[3], P[4], k.get("new", P[5]), width,
                                  None)


@pytest.mark.parametrize("width", [LIMIT + 1, 2 ** 31 - 32769, 2 ** 31 - 8, 2 ** 31 - 1])
def test_rows_too_wide(L, width):
    assert rows(L, width) == capi.PA_ERR_RANGE
    assert rows(L, width, budget=width) == capi.PA_ERR_RANGE
    assert pages(L, width, 128, 1024) == capi.PA_ERR_RANGE


@pytest.mark.parametrize("blocks", [LIMIT + 1, 2 ** 31 - 1])
def test_tables_too_wide(L, blocks):
    assert pages(L, 4096, blocks, 1) == capi.PA_ERR_RANGE


def test_the_widest(L):
    """Taken: the next check is the one that refuses."""
    odd = ctypes.c_void_p(P[5].value + 2)
    assert rows(L, LIMIT, new=odd) == capi.PA_ERR_ALIGN
    assert rows(L, LIMIT, B=0) == capi.PA_OK
    assert pages(L, LIMIT, 128, 1024, new=odd) == capi.PA_ERR_ALIGN
    assert pages(L, 4096, LIMIT, 1, new=odd) == capi.PA_ERR_ALIGN

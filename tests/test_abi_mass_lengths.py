"""Decode with weights for lengths next to 2^31: refused before anything is launched (no
GPU).  The kernel of the weights counts the keys of its last block in 32 bits."""
import ctypes

import pytest

from serving_slot_mapping_gb300 import build as build_mod
from serving_slot_mapping_gb300 import capi

from test_abi_int8_evict import _mass, _pool

LIMIT = 2 ** 31 - 1024


@pytest.fixture(scope="module")
def L():
    build_mod.build()
    return capi.lib()


def call(L, msl, **k):
    return _mass(L, pool=_pool(dtype=capi.PA_DTYPE_BF16), scales=None, batch=1, mb=(2 ** 31 - 1) // 16, msl=msl, stride=2 ** 31 - 1,
                 **k)


@pytest.mark.parametrize("msl", [LIMIT + 1, 2 ** 31 - 129, 2 ** 31 - 16])
def test_lengths_past_the_limit(L, msl):
    assert call(L, msl) == capi.PA_ERR_RANGE


def test_the_longest(L):
    """Taken: the next check is the one that refuses."""
    assert call(L, LIMIT, mass_out=None) == capi.PA_ERR_NULL
    assert call(L, LIMIT, mass_out=ctypes.c_void_p(0x9000002)) == capi.PA_ERR_ALIGN

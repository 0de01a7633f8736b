"""The launch rule of the attention weights (host code, no GPU)."""
import ctypes

import pytest

from serving_slot_mapping_gb300 import build as build_mod


@pytest.mark.parametrize("sms", [152, 148, 76, 1])
def test_tiles_of_a_block_follow_the_sms(sms):
    build_mod.build()
    rule = ctypes.CDLL(build_mod.LIB_PATH)["_ZN2pa14key_mass_tilesEiii"]
    full = 8 * sms           # blocks of one tile that the SMs hold at once
    assert rule(sms, 1, 128 * full) == 1 and rule(sms, 1, 128 * full + 1) == 2
    assert rule(sms, full, 128) == 1 and rule(sms, full, 129) == 2 and rule(sms, full + 1, 1) == 2
    assert rule(sms, 65535, 2 ** 31 - 1024) == 2 and rule(sms, 1, 1) == 1

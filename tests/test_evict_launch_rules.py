"""Launch rules of the evictions (host code, no GPU)."""
import ctypes
import os
import re

import pytest

from serving_slot_mapping_gb300 import build as build_mod

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "serving_slot_mapping_gb300", "csrc")
MAX_PAGES = 8 * 40928        # of a sequence: their weights stay in shared memory
CACHE = MAX_PAGES // 8 + 32  # weights in the shared memory of a CTA


@pytest.fixture(scope="module")
def rule():
    build_mod.build()
    f = ctypes.CDLL(build_mod.LIB_PATH)["_ZN2pa13evict_clusterEiilli"]
    f.argtypes = [ctypes.c_int] * 2 + [ctypes.c_int64] * 2 + [ctypes.c_int]
    return f


@pytest.mark.parametrize("sms", [152, 148, 76, 8, 1])
@pytest.mark.parametrize("most", [8, 16])
def test_clusters(rule, sms, most):
    """At most `most` CTAs; the pages of every sequence that the call takes fit in the shared
    memory of 8, which every GPU can place."""
    for batch in (1, 2, 9, 10, 19, 38, 152, 1000):
        for units in (1, 8192, 32768, 40928, 40929, 131072, MAX_PAGES, 1 << 22):
            for page in (1, 16, 1024):
                c = rule(sms, batch, units, units * page, most)
                assert c in (1, 2, 4, 8, 16) and c <= most
                if units <= MAX_PAGES:
                    assert -(-units // c) + 32 <= CACHE   # a stretch, rounded up to a warp's units
    assert rule(152, 1, 131072, 131072, 16) == 16 and rule(152, 1, 131072, 131072, 8) == 8
    assert rule(152, 10, 131072, 131072, 16) == 8 and rule(152, 32, 4096, 4096, 16) == 1


def test_clusters_past_eight_are_asked_for():
    """A cluster of more than 8 CTAs, which a GPU or a part of one need not be able to place,
    is launched only where the runtime says that it fits; else one of 8."""
    src = re.sub(r"//[^\n]*", "", open(os.path.join(CSRC, "evict.cu")).read())
    launch = src[src.index("cudaError_t launch_evict"):]
    assert "cudaOccupancyMaxActiveClusters" in src
    assert re.search(r"csize > 8 && !most_fit\(", launch)
    assert launch.index("most_fit(") < launch.index("launch_pdl_cluster(")

"""What the package offers under its own name is the binding's."""
import pytest

import serving_slot_mapping_gb300 as package
from serving_slot_mapping_gb300 import capi


@pytest.mark.parametrize("name", ["paged_kv_append_int8", "paged_attention_decode_int8", "paged_attention_prefill_int8",
                                  "paged_attention_decode_mass", "paged_kv_evict_rows", "paged_kv_evict_pages",
                                  "decode_mass_workspace"])
def test_the_calls_of_the_int8_cache_and_the_evictions(name):
    assert getattr(package, name) is getattr(capi, name)

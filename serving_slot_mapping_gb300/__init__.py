"""Paged (block-table) KV-cache append and attention for one GB300 (sm_103a).

The computation lives in ``libpagedattn.so`` (C ABI: ``include/paged_attn.h``);
:mod:`serving_slot_mapping_gb300.capi` is its thin Python binding and
:mod:`serving_slot_mapping_gb300.build` compiles it.
"""
from .capi import (  # noqa: F401
    paged_kv_append,
    paged_attention_decode,
    paged_attention_prefill,
    paged_attention_decode_window,
    paged_attention_prefill_window,
    paged_qk_norm_rope_append,
    paged_kv_copy_pages,
    paged_kv_compact,
    paged_kv_append_int8,
    paged_attention_decode_int8,
    paged_attention_prefill_int8,
    paged_attention_decode_mass,
    paged_kv_evict_rows,
    paged_kv_evict_pages,
    make_pools,
    decode_workspace,
    decode_workspace_size,
    decode_mass_workspace,
    device_error,
    PagedAttnError,
    make_pool,
)

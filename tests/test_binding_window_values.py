"""Integers that the windowed calls of the binding hand to the library (no GPU: the
library is a stand-in that records its arguments).  The C arguments are int32 and
ctypes keeps the low 32 bits of whatever it gets."""
import types

import pytest
import torch

from serving_slot_mapping_gb300 import capi

INT32 = 2 ** 31 - 1


@pytest.fixture
def calls(monkeypatch):
    seen = []

    def record(*args):
        seen.append(args)
        return capi.PA_OK

    fake = types.SimpleNamespace(paged_attention_decode_window=record, paged_attention_prefill_window=record)
    monkeypatch.setattr(capi, "lib", lambda: fake)
    monkeypatch.setattr(capi, "_here", lambda names, tensors: 0)
    monkeypatch.setattr(capi, "_raw_stream", lambda stream, device: 0)
    return seen


def _call(kind, window=8, num_sinks=0, max_q_len=1, max_seq_len=32):
    kp = torch.zeros(4, 16, 2, 64, dtype=torch.bfloat16)
    vp, q = torch.zeros_like(kp), torch.zeros(3, 4, 64, dtype=torch.bfloat16)
    bt, sl = torch.zeros(3, 2, dtype=torch.int32), torch.ones(3, dtype=torch.int32)
    if kind == "decode":
        return capi.paged_attention_decode_window(kp, vp, q, bt, sl, 0.1, window, num_sinks, max_seq_len=max_seq_len,
                                                  workspace=torch.zeros(16, dtype=torch.uint8))
    return capi.paged_attention_prefill_window(kp, vp, q, torch.tensor([0, 1, 2, 3], dtype=torch.int32), bt, sl, 0.1,
                                               max_q_len, window, num_sinks, max_seq_len=max_seq_len)


@pytest.mark.parametrize("kind", ["decode", "prefill"])
@pytest.mark.parametrize("given,passed", [(1, 1), (INT32, INT32), (2 ** 31, INT32), (2 ** 32 + 5, INT32),
                                          (2 ** 63 - 1, INT32), (-3, -1), (-2 ** 32 + 5, -1)])
def test_windows_and_sinks_of_any_size_keep_their_meaning(calls, kind, given, passed):
    at = {"decode": 10, "prefill": 13}[kind]
    _call(kind, window=given)
    _call(kind, num_sinks=given)
    assert calls[0][at:at + 2] == (passed, 0)
    assert calls[1][at:at + 2] == (8, passed)


@pytest.mark.parametrize("kind,name", [("decode", "max_seq_len"), ("prefill", "max_seq_len"), ("prefill", "max_q_len")])
def test_bounds_beyond_32_bits_are_refused(calls, kind, name):
    for n in (2 ** 31, 2 ** 32 + 1, -2 ** 31 - 1):
        with pytest.raises(ValueError, match=name):
            _call(kind, **{name: n})
    assert not calls

"""How the kernels of the windowed layer read their inputs, checked in the sources (no
GPU).  They start before the kernel ahead of them has ended, so an input may be
written while they run: loads that promise the opposite (ld.global.nc, __ldg, and the
other cached-load intrinsics, which the compiler may move ahead of the wait) are not
for them, nor helpers that use them."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "serving_slot_mapping_gb300", "csrc")


def _code(name):
    return re.sub(r"//[^\n]*", "", open(os.path.join(CSRC, name)).read())


@pytest.mark.parametrize("name", ["decode_window.cu", "prefill_window.cu", "norm_rope.cu", "pages.cu", "inputs.cuh"])
def test_no_load_promises_read_only_data(name):
    src = _code(name)
    assert not re.search(r"__ldg|__ldc[sagv]|__ldlu|\.nc\b|__restrict__", src)
    assert not re.search(r"\b(seq_keys|page_list_start)\b", src)  # common.cuh's use __ldg
    for asm in re.findall(r'asm\s*(volatile)?\s*\("ld\.global', src):
        assert asm == "volatile"


def _without_lambdas(src):
    """What runs where it stands: the bodies of named lambdas are taken out."""
    out, at = "", 0
    for m in re.finditer(r"auto \w+ = \[&\]\([^)]*\)[^{;]*\{", src):
        if m.start() < at:
            continue  # inside one that is gone
        out += src[at:m.start()]
        depth, at = 1, m.end()
        while depth and at < len(src):
            depth += {"{": 1, "}": -1}.get(src[at], 0)
            at += 1
    return out + src[at:]


@pytest.mark.parametrize("name,kernels", [("decode_window.cu", 1), ("prefill_window.cu", 1), ("norm_rope.cu", 2),
                                          ("pages.cu", 2)])
def test_every_kernel_waits_ahead_of_its_first_read(name, kernels):
    src = _code(name)
    bodies = [src[m.start():] for m in re.finditer(r"__global__ void", src)]
    assert len(bodies) == kernels
    for body in bodies:
        ahead = _without_lambdas(body[:body.index("griddep_wait()")])
        assert not re.search(r"ld_input\(|ld_stream\(|ld_seq_len\(|seq_rows\(|wk\.start\(|tma_load|bulk_load\(|cp_async_16\(",
                             ahead)

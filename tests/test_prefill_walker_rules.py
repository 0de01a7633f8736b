"""How the prefill's warps find their items, checked in the source (no GPU): every search
ends with the batch, so that lengths which somebody writes while the kernel runs cost
rows and not a kernel that never ends."""
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "serving_slot_mapping_gb300", "csrc")


def test_every_search_ends_with_the_batch():
    src = re.sub(r"//[^\n]*", "", open(os.path.join(CSRC, "prefill_window.cu")).read())
    walkers = src[src.index("struct Walker"):src.index("struct AnyWalker")]
    loops = re.findall(r"\b(for|while)\s*\(([^{;]*(?:;[^{;]*;[^{]*)?)\)\s*\{?", walkers)
    assert len(loops) >= 6
    for kind, head in loops:
        condition = head.split(";")[1] if kind == "for" else head
        assert condition.strip() not in ("", "true", "1"), (kind, head)
    assert "base < p.batch" in walkers and "base + 32 >= p.batch" in walkers and "level == 0" in walkers

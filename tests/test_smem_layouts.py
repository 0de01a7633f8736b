"""Shared-memory layouts of the tensor-core prefill kernels, worked out from their
sources (no GPU): the word that tcgen05.alloc writes the TMEM base to lies on no
mbarrier.  Both are written before the same __syncthreads, the barriers by thread
0 and the word by the allocating warp, so an overlap is a race."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "serving_slot_mapping_gb300", "csrc")


def _constants(*names):
    """{name: expression} of the constexpr ints and enumerators of the sources."""
    out = {}
    for n in names:
        src = re.sub(r"//[^\n]*", "", open(os.path.join(CSRC, n)).read())
        for m in re.finditer(r"constexpr (?:int|uint32_t) ([^;]*);", src):
            for part in re.findall(r"(\w+) = ([^=]+?)(?=, \w+ = |$)", m.group(1).replace("\n", " ")):
                out.setdefault(*part)
        for m in re.finditer(r"enum \{([^}]*)\}", src):
            for name, expr in (e.split("=") for e in m.group(1).split(",") if "=" in e):
                out.setdefault(name.strip(), expr.strip())
            last = [e.strip() for e in m.group(1).split(",")]
            assert all("=" in e for e in last), "every enumerator is given its value"
    return out


def _value(expr, consts, D):
    expr = re.sub(r"\b(C|Base)::", "", expr)
    expr = re.sub(r"\bsizeof\(\w+\)", "4", expr)
    names = {n for n in re.findall(r"[A-Za-z_]\w*", expr)} - {"D"}
    env = {n: _value(consts[n], consts, D) for n in names}
    return eval(expr.replace("/", "//"), {}, dict(env, D=D))


@pytest.mark.parametrize("source,first,count", [("prefill_tc.cuh", "kBarOff", "B_COUNT"),
                                                ("prefill_window.cu", "kWBarOff", "W_COUNT")])
@pytest.mark.parametrize("D", [64, 128])
def test_the_tmem_base_lies_on_no_barrier(source, first, count, D):
    src = open(os.path.join(CSRC, source)).read()
    consts = _constants(source, "prefill_tc.cuh")
    word = re.search(r"tmem_slot = reinterpret_cast<uint32_t\*>\(smem \+ ([^;]+)\);", src).group(1)
    at, bars = _value(word, consts, D), _value(first, consts, D)
    assert at % 4 == 0 and bars % 8 == 0
    assert at >= bars + 8 * _value(count, consts, D) or at + 4 <= bars

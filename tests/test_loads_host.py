"""What kernels that start while the one before still runs read by which loads. Such a start (griddepcontrol) comes before the
wait for the other kernel's writes, so that a load of memory that is read-only for the kernel's whole life (__ldg, ld.global.nc)
is allowed for weights alone."""
from __future__ import annotations

import glob
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "bit_affine_quantized_group_gb300", "csrc")
SOURCES = sorted(glob.glob(os.path.join(CSRC, "*.cu*")))

# file: what it may read so
WEIGHTS = {
    "qmm_adapter.cu": (r"__ldg\(p\.scale \+", r"load_weights\(const uint16_t\* p\) \{ return __ldg\("),
    "qmm_append.cu": (r"__ldg\(reinterpret_cast<const float4\*>\(weight \+ e0",),
}


def _code(path):
    return [re.sub(r"//.*", "", line) for line in open(path)]


@pytest.mark.parametrize("path", SOURCES, ids=os.path.basename)
def test_read_only_loads_are_of_weights(path):
    allowed = WEIGHTS.get(os.path.basename(path), ())
    for n, line in enumerate(_code(path), 1):
        assert "ld.global.nc" not in line, (n, line)
        if "__ldg(" in line:
            assert any(re.search(a, line) for a in allowed), (n, line)


def test_weights_of_adapters_are_b_alone():
    text = "".join(_code(os.path.join(CSRC, "qmm_adapter.cu")))
    calls = re.findall(r"load_weights\(([^;]*?) \+ k \* 32\)", text)
    assert len(calls) == 3 and all("b_next" in c for c in calls)


def test_what_adapters_read_before_their_wait_comes_from_l2():
    text = "".join(_code(os.path.join(CSRC, "qmm_adapter.cu")))
    assert "__ldcg(p.ids" in text and not re.search(r"[^(]p\.ids\[", text)
    assert re.search(r"wy\[h\]\[k\] = F32 && !early \? \*from : __ldcg\(from\)", text)
    assert len(re.findall(r"load_y\(0, left, !waited\)", text)) == 2 and len(re.findall(r"load_y\(32, left_next, false\)", text)) == 1

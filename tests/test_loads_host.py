"""What kernels that start while the one before still runs read by which loads."""
from __future__ import annotations

import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "bit_affine_quantized_group_gb300", "csrc")


def _code(path):
    return [re.sub(r"//.*", "", line) for line in open(path)]


def test_what_adapters_read_before_their_wait_comes_from_l2():
    text = "".join(_code(os.path.join(CSRC, "qmm_adapter.cu")))
    assert "__ldcg(p.ids" in text and not re.search(r"[^(]p\.ids\[", text)
    assert re.search(r"wy\[h\]\[k\] = F32 && !early \? \*from : __ldcg\(from\)", text)
    assert len(re.findall(r"load_y\(0, left, !waited\)", text)) == 2 and len(re.findall(r"load_y\(32, left_next, false\)", text)) == 1

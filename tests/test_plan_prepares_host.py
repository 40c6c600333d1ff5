"""What a plan of the cache operators prepares: the kernels of bfloat16 caches, and those of caches of codes not before a call over
one, so that users of bfloat16 caches do not pay for them."""
from __future__ import annotations

import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "bit_affine_quantized_group_gb300", "csrc")


def _body(file, start):
    text = open(os.path.join(CSRC, file)).read()
    at = text.index(start)
    return text[at:text.index("\n}", at)]


def test_plans_configure_no_kernels_of_codes():
    assert "codes" not in re.sub(r"//.*", "", _body("qmm_attention.cu", "cudaError_t configure_attention()"))
    assert "codes" not in re.sub(r"//.*", "", _body("qmm_kv_api.cu", "int qmm_kv_plan("))


def test_calls_over_codes_do():
    attend = _body("qmm_kv_api.cu", "int attend(")
    assert attend.index("configure_attention_codes(bits, p->device)") < attend.index("launch_attention(")

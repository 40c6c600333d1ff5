"""Errors of the operators name the call that failed, for each kind of cache. No test here makes a CUDA call."""
from __future__ import annotations

import contextlib

import pytest


@pytest.fixture(scope="module")
def q():
    from bit_affine_quantized_group_gb300 import _build
    _build.build()
    import bit_affine_quantized_group_gb300 as q
    return q


class Failing:
    """The real library, but plans succeed and launches fail."""

    def __init__(self, real):
        self.real = real

    def __getattr__(self, name):
        if name in ("qmm_kv_plan", "qmm_adapter_plan"):
            return lambda *a: 0
        if name in ("qmm_kvq_qk_norm_rope", "qmm_kvq_attention", "qmm_kvq_read", "qmm_attention", "qmm_qk_norm_rope"):
            return lambda *a: 4
        return getattr(self.real, name)


def test_errors_name_their_call(q, monkeypatch):
    import torch
    monkeypatch.setattr(q, "_LIB", Failing(q.lib))
    monkeypatch.setattr(torch.cuda, "device", lambda d: contextlib.nullcontext())
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    plan = q.KVPlan(4, 2, 128, 16, max_seqs=2, max_rows=2, max_pages=3, torch_workspace=False, device="cpu:0", rot_dim=0)
    plan._device_index = -1   # what CPU tensors give for their device
    code = torch.zeros((3, 2, 16, 128), dtype=torch.uint8)
    affine = torch.zeros((3, 2, 16, 2, 2), dtype=torch.float16)
    dense = torch.zeros((3, 2, 16, 128), dtype=torch.bfloat16)
    x, kv = torch.zeros((2, 512), dtype=torch.bfloat16), torch.zeros((2, 256), dtype=torch.bfloat16)
    lens, table = torch.zeros(2, dtype=torch.int32), torch.zeros((2, 3), dtype=torch.int32)
    for cache, prefix in ((q.QuantKVCache(code, code, affine, affine, 8), "qmm_kvq_"), (q.KVCache(dense, dense), "qmm_")):
        for call, name in ((lambda: q.attention(plan, x, cache, table, lens, x, stream=0), "attention"),
                           (lambda: q.qk_norm_rope(plan, x, kv, kv, None, None, None, lens, table, cache, x, stream=0), "qk_norm_rope")):
            with pytest.raises(q.QmmError) as e:
                call()
            assert str(e.value).startswith(prefix + name + ":") and e.value.status == 4
    with pytest.raises(q.QmmError, match="^qmm_kvq_read:"):
        out = torch.zeros((2, 5, 2, 128))
        q.kv_read(plan, q.QuantKVCache(code, code, affine, affine, 8), table, lens, out, out.clone(), stream=0)
    plan._handle.value = None

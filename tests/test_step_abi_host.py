"""Host-only tests of the operators between two projections (cache append, attention, sampling): descriptors and
arguments are refused before anything is launched. No test here makes a CUDA call that needs a GPU."""
from __future__ import annotations

import ctypes

import pytest


@pytest.fixture(scope="module")
def q():
    from bit_affine_quantized_group_gb300 import _build
    _build.build()
    import bit_affine_quantized_group_gb300 as q
    return q


GOOD = dict(q_heads=32, kv_heads=8, head_dim=128, page_size=16, max_seqs=4, max_rows=8, max_pages=100)


@pytest.mark.parametrize("change,expect", [
    ({}, 0), ({"head_dim": 64}, 0), ({"head_dim": 256}, 0), ({"page_size": 1}, 0), ({"page_size": 1024}, 0),
    ({"rot_dim": 0}, 0), ({"rot_dim": 16}, 0), ({"window": 1}, 0), ({"sinks": 7}, 0), ({"q_heads": 8 * 64}, 0),
    ({"q_heads": 0}, 1), ({"kv_heads": 0}, 1), ({"q_heads": 33}, 1), ({"max_seqs": 0}, 1), ({"max_seqs": 65537}, 1),
    ({"max_rows": 0}, 1), ({"max_rows": 17}, 1), ({"max_pages": 0}, 1), ({"window": -1}, 1), ({"sinks": -1}, 1),
    ({"rot_dim": -16}, 1), ({"rot_dim": 144}, 1), ({"scale": float("nan")}, 1), ({"scale": float("inf")}, 1),
    ({"eps": -1.0}, 1), ({"eps": float("nan")}, 1), ({"page_size": 0}, 1), ({"page_size": 1024, "max_pages": 1 << 21}, 1),
    ({"head_dim": 96}, 2), ({"head_dim": 512}, 2), ({"page_size": 24}, 2), ({"page_size": 2048}, 2),
    ({"q_heads": 8 * 65}, 2), ({"rot_dim": 24}, 2),
])
def test_validate_kv_desc(q, change, expect):
    d = q.make_kv_desc(**{**GOOD, **change})
    assert q.kv_validate_desc(d) == expect
    assert (q.kv_workspace_bytes(d) > 0) == (expect == 0)


def test_null_handles(q):
    lib = q.lib
    assert lib.qmm_kv_validate_desc(None) == q.QMM_ERR_INVALID_ARG
    assert lib.qmm_kv_plan(None, None, None, 0) == q.QMM_ERR_INVALID_ARG
    assert lib.qmm_kv_error(None, None) == q.QMM_ERR_INVALID_ARG
    assert lib.qmm_qk_norm_rope(None, None, None, None) == q.QMM_ERR_INVALID_ARG
    assert lib.qmm_attention(None, None, None, None) == q.QMM_ERR_INVALID_ARG
    lib.qmm_kv_destroy(None)   # accepted
    out = ctypes.c_void_p(1)
    bad = q.make_kv_desc(**{**GOOD, "head_dim": 96})
    assert lib.qmm_kv_plan(ctypes.byref(out), ctypes.byref(bad), None, 0) == q.QMM_ERR_UNSUPPORTED
    assert out.value is None
    good = q.make_kv_desc(**GOOD)
    need = q.kv_workspace_bytes(good)   # a workspace that is too small or misaligned
    assert lib.qmm_kv_plan(ctypes.byref(out), ctypes.byref(good), 0x1000, need - 1) == q.QMM_ERR_INVALID_ARG
    assert lib.qmm_kv_plan(ctypes.byref(out), ctypes.byref(good), 0x1010, need) == q.QMM_ERR_INVALID_ARG


def _cache(q, **kw):
    d, page = 128, 16
    f = dict(k=0x100000, v=0x200000, num_pages=50, k_page_stride=8 * page * d, k_head_stride=page * d, k_slot_stride=d,
             v_page_stride=8 * page * d, v_head_stride=page * d, v_slot_stride=d)
    f.update(kw)
    return q.QmmKvCache(**f)


CACHE_FAULTS = [{"k": 0}, {"v": 0}, {"k": 0x100008}, {"v": 0x200002}, {"num_pages": -1}, {"k_page_stride": 4},
                {"v_slot_stride": 12}, {"k_head_stride": -8}, {"v_page_stride": 1 << 41}]


@pytest.mark.parametrize("kw,expect", [
    ({}, 0), ({"seqs": 0, "q": 0, "out": 0}, 0), ({"rows": 0, "q": 0}, 0), ({"rows": 8}, 0),
    ({"rows": 9}, 1), ({"rows": -1}, 1), ({"seqs": 5}, 1), ({"seqs": -1}, 1), ({"q": 0}, 1), ({"q": 0x3008}, 1),
    ({"out": 0}, 1), ({"out": 0x4002}, 1), ({"page_table": 0}, 1), ({"page_table": 0x5002}, 1), ({"lengths": 0}, 1),
    ({"q_stride": 4095}, 1), ({"q_stride": 4104}, 0), ({"q_stride": 4100}, 1), ({"out_stride": 4088}, 1),
    ({"seqs": 1, "rows": 1, "q_stride": 0}, 0),
])
def test_attention_args(q, kw, expect):
    a = dict(q=0x3000, q_stride=4096, page_table=0x5000, lengths=0x6000, seqs=2, rows=1, out=0x4000, out_stride=4096)
    a.update(kw)
    d, c, args = q.make_kv_desc(**GOOD), _cache(q), q.QmmAttentionArgs(**a)
    assert q.lib.qmm_check_attention_args(ctypes.byref(d), ctypes.byref(c), ctypes.byref(args)) == expect


@pytest.mark.parametrize("fault", CACHE_FAULTS)
def test_cache_faults(q, fault):
    d, c = q.make_kv_desc(**GOOD), _cache(q, **fault)
    a = q.QmmAttentionArgs(q=0x3000, q_stride=4096, page_table=0x5000, lengths=0x6000, seqs=2, rows=1, out=0x4000,
                           out_stride=4096)
    args = (ctypes.byref(d), ctypes.byref(c), ctypes.byref(a))
    assert q.lib.qmm_check_attention_args(*args) == q.QMM_ERR_INVALID_ARG
    assert q.lib.qmm_check_attention_args(None, *args[1:]) == q.QMM_ERR_INVALID_ARG
    assert q.lib.qmm_check_attention_args(args[0], None, args[2]) == q.QMM_ERR_INVALID_ARG
    assert q.lib.qmm_check_attention_args(*args[:2], None) == q.QMM_ERR_INVALID_ARG


@pytest.mark.parametrize("kw,expect", [
    ({}, 0), ({"in_dtype": 0}, 0), ({"q_weight": 0, "k_weight": 0}, 0), ({"positions": 0x9000}, 0), ({"rows": 5000}, 0),
    ({"rows": 0, "q": 0}, 0), ({"seqs": 0, "q_out": 0}, 0),
    ({"q": 0}, 1), ({"k": 0}, 1), ({"v": 0x10008}, 1), ({"q_out": 0}, 1), ({"q_out": 0x8}, 1), ({"rope": 0}, 1),
    ({"rope": 0x8008}, 1), ({"rope_len": 0}, 1), ({"lengths": 0}, 1), ({"lengths": 0x6001}, 1), ({"page_table": 0}, 1),
    ({"q_weight": 0x7004}, 1), ({"k_weight": 0x7008}, 1), ({"positions": 0x9002}, 1), ({"in_dtype": 2}, 1),
    ({"seqs": 5}, 1), ({"seqs": -1}, 1), ({"rows": -2}, 1), ({"q_stride": 6140}, 1), ({"k_stride": 1000}, 1),
    ({"in_dtype": 0, "v_stride": 6148}, 0), ({"in_dtype": 1, "v_stride": 6148}, 1), ({"q_out_stride": 4090}, 1),
    ({"seqs": 4, "rows": 1 << 28}, 2),
])
def test_append_args(q, kw, expect):
    a = dict(q=0x10000, k=0x12000, v=0x14000, q_stride=6144, k_stride=6144, v_stride=6144, q_weight=0x7000,
             k_weight=0x7200, rope=0x8000, rope_len=1000, lengths=0x6000, positions=0, page_table=0x5000, q_out=0x20000,
             q_out_stride=4096, seqs=2, rows=3, in_dtype=1)
    a.update(kw)
    d, c = q.make_kv_desc(**GOOD), _cache(q)
    args = q.QmmAppendArgs(**a)
    assert q.lib.qmm_check_qk_norm_rope_args(ctypes.byref(d), ctypes.byref(c), ctypes.byref(args)) == expect
    assert q.lib.qmm_check_qk_norm_rope_args(ctypes.byref(d), ctypes.byref(c), None) == q.QMM_ERR_INVALID_ARG


def test_append_without_rotation_needs_no_table(q):
    d, c = q.make_kv_desc(**GOOD, rot_dim=0), _cache(q)
    a = q.QmmAppendArgs(q=0x10000, k=0x12000, v=0x14000, q_stride=6144, k_stride=6144, v_stride=6144, lengths=0x6000,
                        page_table=0x5000, q_out=0x20000, q_out_stride=4096, seqs=2, rows=3, in_dtype=1)
    assert q.lib.qmm_check_qk_norm_rope_args(ctypes.byref(d), ctypes.byref(c), ctypes.byref(a)) == q.QMM_OK


@pytest.mark.parametrize("kw,expect", [
    ({"M": 0, "logits": 0}, 0), ({"M": -1}, 1), ({"vocab": 0}, 1), ({"vocab": 393217}, 2), ({"logits": 0}, 1),
    ({"logits": 0x1002}, 1), ({"stride": 999}, 1), ({"dtype": 2}, 1), ({"temperature": 0}, 1), ({"top_k": 0}, 1),
    ({"top_p": 0x3001}, 1), ({"min_p": 0}, 1), ({"u": 0}, 1), ({"tokens": 0}, 1), ({"probs": 0x8002}, 1),
])
def test_sample_args(q, kw, expect):
    a = dict(logits=0x1000, M=2, vocab=1000, stride=1000, dtype=0, temperature=0x2000, top_k=0x2100, top_p=0x2200,
             min_p=0x2300, u=0x2400, tokens=0x2500, probs=0x2600)
    a.update(kw)
    assert q.lib.qmm_sample(a["logits"], a["M"], a["vocab"], a["stride"], a["dtype"], a["temperature"], a["top_k"],
                            a["top_p"], a["min_p"], a["u"], a["tokens"], a["probs"], None) == expect


def test_binding_refusals(q):
    """The Python entry points name the tensor that does not fit before they call the library."""
    torch = pytest.importorskip("torch")
    k = torch.zeros((3, 2, 16, 64), dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        q.KVCache(k.float(), k.float())
    with pytest.raises(ValueError):
        q.KVCache(k, k[:2])
    with pytest.raises(ValueError):
        q.KVCache(k.transpose(2, 3), k.transpose(2, 3))
    f, i = torch.zeros(2), torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError):
        q.sample(torch.zeros((2, 10), dtype=torch.float16), f, i, f, f, f, i)
    with pytest.raises(ValueError):
        q.sample(torch.zeros((2, 10)), f, f, f, f, f, i)
    with pytest.raises(ValueError):
        q.sample(torch.zeros((2, 10)), f, i, f, f, f, i, probs=torch.zeros(3))

"""Host-only tests of the operators that serve many requests (caches of codes, adapters, log probabilities): descriptors and
arguments are refused before anything is launched. No test here makes a CUDA call that needs a GPU."""
from __future__ import annotations

import contextlib
import ctypes

import pytest

GOOD = dict(q_heads=32, kv_heads=8, head_dim=128, page_size=16, max_seqs=4, max_rows=8, max_pages=100)


@pytest.fixture(scope="module")
def q():
    from bit_affine_quantized_group_gb300 import _build
    _build.build()
    import bit_affine_quantized_group_gb300 as q
    return q


def _cache(q, **kw):
    f = dict(k=0x100000, v=0x200000, k_affine=0x300000, v_affine=0x400000, num_pages=50, bits=8)
    for s in "kv":
        f.update({f"{s}_page_stride": 8 * 16 * 128, f"{s}_head_stride": 16 * 128, f"{s}_slot_stride": 128,
                  f"{s}a_page_stride": 8 * 16 * 2, f"{s}a_head_stride": 16 * 2, f"{s}a_slot_stride": 2})
    f.update(kw)
    return q.QmmKvqCache(**f)


ATTEND = dict(q=0x3000, q_stride=4096, page_table=0x5000, lengths=0x6000, seqs=2, rows=1, out=0x4000, out_stride=4096)
APPEND = dict(q=0x10000, k=0x12000, v=0x14000, q_stride=6144, k_stride=6144, v_stride=6144, q_weight=0x7000, k_weight=0x7200,
              rope=0x8000, rope_len=1000, lengths=0x6000, positions=0, page_table=0x5000, q_out=0x20000, q_out_stride=4096,
              seqs=2, rows=3, in_dtype=1)
READ = dict(k_out=0x10000, v_out=0x20000, k_seq_stride=10240, k_row_stride=1024, v_seq_stride=10240, v_row_stride=1024,
            lengths=0x6000, starts=0, page_table=0x5000, seqs=2, rows=10, out_dtype=1)


def _calls(q):
    return [(q.lib.qmm_check_kvq_attention_args, q.QmmAttentionArgs(**ATTEND)),
            (q.lib.qmm_check_kvq_qk_norm_rope_args, q.QmmAppendArgs(**APPEND)),
            (q.lib.qmm_check_kvq_read_args, q.QmmReadArgs(**READ))]


@pytest.mark.parametrize("change,expect", [
    ({}, 0), ({"bits": 4}, 0), ({"num_pages": 0}, 0), ({"k_page_stride": 16}, 0), ({"va_slot_stride": 4}, 0), ({"ka_page_stride": 0}, 0),
    ({"k": 0}, 1), ({"v": 0}, 1), ({"k_affine": 0}, 1), ({"v_affine": 0}, 1), ({"k": 0x100008}, 1), ({"v": 0x200001}, 1),
    ({"k_affine": 0x300008}, 1), ({"v_affine": 0x400004}, 1), ({"num_pages": -1}, 1), ({"num_pages": 1 << 31}, 1),
    ({"k_page_stride": 8}, 1), ({"v_slot_stride": 120}, 1), ({"k_head_stride": -16}, 1), ({"v_page_stride": 1 << 41}, 1),
    ({"ka_slot_stride": 1}, 1), ({"va_head_stride": 33}, 1), ({"ka_page_stride": -2}, 1), ({"va_page_stride": 1 << 41}, 1),
    ({"bits": 16}, 2), ({"bits": 0}, 2), ({"bits": 5}, 2),
])
def test_cache_of_codes(q, change, expect):
    d, c = q.make_kv_desc(**GOOD), _cache(q, **change)
    for check, args in _calls(q):
        assert check(ctypes.byref(d), ctypes.byref(c), ctypes.byref(args)) == expect


def test_null_arguments(q):
    d, c = q.make_kv_desc(**GOOD), _cache(q)
    bad = q.make_kv_desc(**{**GOOD, "head_dim": 96})
    for check, args in _calls(q):
        assert check(None, ctypes.byref(c), ctypes.byref(args)) == 1
        assert check(ctypes.byref(d), None, ctypes.byref(args)) == 1
        assert check(ctypes.byref(d), ctypes.byref(c), None) == 1
        assert check(ctypes.byref(bad), ctypes.byref(c), ctypes.byref(args)) == 2
    for call in (q.lib.qmm_kvq_attention, q.lib.qmm_kvq_qk_norm_rope, q.lib.qmm_kvq_read):
        assert call(None, None, None, None) == 1
    assert q.lib.qmm_add_adapters(None, None, None) == 1
    assert q.lib.qmm_adapter_plan(None, None, None, 0) == 1
    assert q.lib.qmm_adapter_error(None, None) == 1
    assert q.lib.qmm_adapter_validate_desc(None) == 1
    q.lib.qmm_adapter_destroy(None)   # accepted


@pytest.mark.parametrize("kw,expect", [
    ({}, 0), ({"rows": 9}, 1), ({"rows": -1}, 1), ({"seqs": 5}, 1), ({"q": 0}, 1), ({"out": 0x4002}, 1), ({"page_table": 0}, 1),
    ({"lengths": 0x6002}, 1), ({"q_stride": 4100}, 1), ({"seqs": 0, "q": 0}, 0),
])
def test_attention_args(q, kw, expect):
    d, c, a = q.make_kv_desc(**GOOD), _cache(q), q.QmmAttentionArgs(**{**ATTEND, **kw})
    assert q.lib.qmm_check_kvq_attention_args(ctypes.byref(d), ctypes.byref(c), ctypes.byref(a)) == expect


@pytest.mark.parametrize("kw,expect", [
    ({}, 0), ({"rows": 5000}, 0), ({"q": 0}, 1), ({"rope": 0}, 1), ({"k_weight": 0x7008}, 1), ({"in_dtype": 2}, 1), ({"rows": -2}, 1),
    ({"v_stride": 6148}, 1), ({"q_out": 0x8}, 1), ({"rows": 0, "q": 0}, 0), ({"seqs": 4, "rows": 1 << 28}, 2),
])
def test_append_args(q, kw, expect):
    d, c, a = q.make_kv_desc(**GOOD), _cache(q), q.QmmAppendArgs(**{**APPEND, **kw})
    assert q.lib.qmm_check_kvq_qk_norm_rope_args(ctypes.byref(d), ctypes.byref(c), ctypes.byref(a)) == expect


@pytest.mark.parametrize("kw,expect", [
    ({}, 0), ({"out_dtype": 0}, 0), ({"starts": 0x9000}, 0), ({"rows": 0, "k_out": 0}, 0), ({"seqs": 0, "v_out": 0}, 0),
    ({"k_seq_stride": 1024, "k_row_stride": 2048}, 0), ({"k_seq_stride": 1024}, 1), ({"v_seq_stride": 10224}, 1), ({"seqs": 1, "k_seq_stride": 0}, 0), ({"rows": 1, "v_row_stride": 0}, 0),
    ({"k_out": 0}, 1), ({"v_out": 0}, 1), ({"k_out": 0x10008}, 1), ({"v_out": 0x20001}, 1), ({"lengths": 0}, 1),
    ({"lengths": 0x6001}, 1), ({"starts": 0x9002}, 1), ({"page_table": 0}, 1), ({"out_dtype": 2}, 1), ({"out_dtype": -1}, 1),
    ({"seqs": 5}, 1), ({"seqs": -1}, 1), ({"rows": -1}, 1), ({"k_row_stride": 1020}, 1), ({"v_row_stride": 1028}, 1),
    ({"out_dtype": 0, "v_row_stride": 1028, "v_seq_stride": 10280}, 0), ({"k_seq_stride": 1000}, 1), ({"v_seq_stride": 1 << 41}, 1),
    ({"rows": 1 << 30}, 2), ({"rows": 0x7FFFFFFF, "out_dtype": 0}, 2),
])
def test_read_args(q, kw, expect):
    d, c, a = q.make_kv_desc(**GOOD), _cache(q), q.QmmReadArgs(**{**READ, **kw})
    assert q.lib.qmm_check_kvq_read_args(ctypes.byref(d), ctypes.byref(c), ctypes.byref(a)) == expect


@pytest.mark.parametrize("kw", [{}, {"out_dtype": 0}, {"rows": 1}])
def test_keys_and_values_are_not_read_to_one_place(q, kw):
    d, c, a = q.make_kv_desc(**GOOD), _cache(q), q.QmmReadArgs(**{**READ, "v_out": READ["k_out"], **kw})
    assert q.lib.qmm_check_kvq_read_args(ctypes.byref(d), ctypes.byref(c), ctypes.byref(a)) == q.QMM_ERR_INVALID_ARG


ADAPTER = dict(K=4096, N=1000, rank=16, adapters=8, max_rows=64, out_dtype="bf16")


@pytest.mark.parametrize("change,expect", [
    ({}, 0), ({"out_dtype": "f32"}, 0), ({"rank": 8}, 0), ({"rank": 128}, 0), ({"N": 1}, 0), ({"K": 64}, 0), ({"max_rows": 1 << 20}, 0),
    ({"K": 0}, 1), ({"N": 0}, 1), ({"rank": 0}, 1), ({"rank": -8}, 1), ({"adapters": 0}, 1), ({"max_rows": 0}, 1),
    ({"max_rows": (1 << 20) + 1}, 1), ({"K": 1 << 31}, 1), ({"N": 1 << 31}, 1),
    ({"K": 4100}, 2), ({"rank": 12}, 2), ({"rank": 136}, 2),
])
def test_adapter_desc(q, change, expect):
    d = q.make_adapter_desc(**{**ADAPTER, **change})
    assert q.adapter_validate_desc(d) == expect
    assert (q.adapter_workspace_bytes(d) > 0) == (expect == 0)
    out = ctypes.c_void_p(1)
    if expect:
        assert q.lib.qmm_adapter_plan(ctypes.byref(out), ctypes.byref(d), None, 0) == expect
        assert out.value is None
        with pytest.raises(q.QmmError):
            q.AdapterPlan(**{**ADAPTER, **change})
    else:
        need = q.adapter_workspace_bytes(d)
        assert q.lib.qmm_adapter_plan(ctypes.byref(out), ctypes.byref(d), 0x1000, need - 1) == 1
        assert q.lib.qmm_adapter_plan(ctypes.byref(out), ctypes.byref(d), 0x1010, need) == 1


def test_adapter_out_dtype(q):
    d = q.make_adapter_desc(**ADAPTER)
    d.out_dtype = 2
    assert q.adapter_validate_desc(d) == 1
    with pytest.raises(ValueError):
        q.make_adapter_desc(**{**ADAPTER, "out_dtype": "f16"})


@pytest.mark.parametrize("kw,expect", [
    ({}, 0), ({"scale": 0}, 0), ({"y": 0x5000, "out": 0x5000}, 0), ({"rows": 0, "x": 0}, 0), ({"rows": 64}, 0),
    ({"rows": 1, "x_stride": 0, "y_stride": 0, "out_stride": 0}, 0), ({"y": 0x5002, "out": 0x6002}, 0),
    ({"rows": 65}, 1), ({"rows": -1}, 1), ({"x": 0}, 1), ({"a": 0}, 1), ({"b": 0}, 1), ({"ids": 0}, 1), ({"y": 0}, 1),
    ({"out": 0}, 1), ({"x": 0x1008}, 1), ({"a": 0x2004}, 1), ({"b": 0x3001}, 1), ({"ids": 0x4002}, 1), ({"y": 0x5001}, 1),
    ({"out": 0x6001}, 1), ({"scale": 0x7002}, 1), ({"x_stride": 4088}, 1), ({"x_stride": 4100}, 1), ({"y_stride": 999}, 1),
    ({"out_stride": 999}, 1), ({"out_stride": 1 << 41}, 1), ({"y": 0x5000, "out": 0x5000, "out_stride": 1008}, 1),
])
def test_adapter_args(q, kw, expect):
    a = dict(x=0x1000, a=0x2000, b=0x3000, scale=0x7000, ids=0x4000, y=0x5000, out=0x6000, x_stride=4096, y_stride=1000,
             out_stride=1000, rows=5)
    a.update(kw)
    d, args = q.make_adapter_desc(**ADAPTER), q.QmmAdapterArgs(**a)
    assert q.lib.qmm_check_adapter_args(ctypes.byref(d), ctypes.byref(args)) == expect
    assert q.lib.qmm_check_adapter_args(None, ctypes.byref(args)) == 1
    assert q.lib.qmm_check_adapter_args(ctypes.byref(d), None) == 1


@pytest.mark.parametrize("kw,expect", [
    ({"M": 0, "logits": 0}, 0), ({"M": -1}, 1), ({"vocab": 0}, 1), ({"vocab": 393217}, 2), ({"top": -1}, 1), ({"top": 33}, 2),
    ({"logits": 0}, 1), ({"logits": 0x1002}, 1), ({"stride": 999}, 1), ({"dtype": 2}, 1), ({"tokens": 0}, 1), ({"lp": 0}, 1),
    ({"tokens": 0x2002}, 1), ({"entropy": 0x2201}, 1), ({"tt": 0}, 1), ({"tl": 0}, 1), ({"top": 0}, 1), ({"tt": 0x2302}, 1),
    ({"tl": 0x2402}, 1),
])
def test_logprobs_args(q, kw, expect):
    a = dict(logits=0x1000, M=2, vocab=1000, stride=1000, dtype=0, tokens=0x2000, lp=0x2100, entropy=0x2200, top=4, tt=0x2300,
             tl=0x2400)
    a.update(kw)
    assert q.lib.qmm_logprobs(a["logits"], a["M"], a["vocab"], a["stride"], a["dtype"], a["tokens"], a["lp"], a["entropy"],
                              a["top"], a["tt"], a["tl"], None) == expect


# ---- the Python entry points, with CPU tensors in the place of the device's ----

def _codes(torch, bits=8, d=128, heads=2, page=16, pages=3):
    c = torch.zeros((pages, heads, page, d * bits // 8), dtype=torch.uint8)
    return c, torch.zeros((pages, heads, page, d // 64, 2), dtype=torch.float16)


def test_refusals_of_the_cache(q):
    import torch
    for bits in (8, 4):
        for d in (64, 128, 256):
            c, a = _codes(torch, bits, d)
            cache = q.QuantKVCache(c, c, a, a, bits)
            assert cache.page_shape == (2, 16, d)
            assert cache.struct.ka_slot_stride == d // 64 and cache.struct.k_slot_stride == d * bits // 8
    c, a = _codes(torch)
    wrong = [(c, c, a, a, 16), (c.short(), c.short(), a, a, 8), (c, c[:2], a, a, 8), (c, c, a.float(), a, 8), (c, c, a, a[:2], 8),
             (c, c, a[..., :1], a, 8), (c, c, a[:, :, :, :1], a, 8), (c[..., :100], c[..., :100], a, a, 8), (c[0], c[0], a[0], a[0], 8),
             (c.transpose(2, 3), c.transpose(2, 3), a, a, 8), (c, c, a.transpose(3, 4), a, 8), (c, c, a, a, 4),
             (c, c, torch.zeros((3, 2, 16, 2, 3), dtype=torch.float16)[..., :2], a, 8)]
    for args in wrong:
        with pytest.raises((ValueError, IndexError)):
            q.QuantKVCache(*args)
    # pools laid out [pages, page_size, kv_heads, ...]
    c2, a2 = c.transpose(1, 2).contiguous().transpose(1, 2), a.transpose(1, 2).contiguous().transpose(1, 2)
    s = q.QuantKVCache(c2, c2, a2, a2, 8).struct
    assert (s.k_head_stride, s.k_slot_stride, s.ka_head_stride, s.va_slot_stride) == (128, 256, 2, 4)


class Library:
    """The real library, but for the calls that need a GPU."""

    def __init__(self, q):
        self.real, self.calls = q.lib, []

    def __getattr__(self, name):
        if name in ("qmm_kv_plan", "qmm_adapter_plan"):
            return lambda *a: 0
        if name in ("qmm_kvq_qk_norm_rope", "qmm_kvq_attention", "qmm_kvq_read", "qmm_add_adapters", "qmm_logprobs", "qmm_attention",
                    "qmm_qk_norm_rope"):
            return lambda *a: self.calls.append((name, a)) or 0
        return getattr(self.real, name)


@pytest.fixture
def fake(q, monkeypatch):
    import torch
    monkeypatch.setattr(q, "_LIB", Library(q))
    monkeypatch.setattr(torch.cuda, "device", lambda d: contextlib.nullcontext())
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    q._bind_torch()
    monkeypatch.setattr(q, "_CURRENT_DEVICE", lambda: 3, raising=False)
    return q


def _elsewhere(t):
    """t, as a tensor that says that it is on another device."""
    import torch

    class Elsewhere(torch.Tensor):
        def get_device(self):
            return 3
    return t.as_subclass(Elsewhere)


def _kv_plan(q):
    p = q.KVPlan(4, 2, 128, 16, max_seqs=2, max_rows=2, max_pages=3, torch_workspace=False, device="cpu:0", rot_dim=0)
    p._device_index = -1   # what CPU tensors give for their device
    return p


def test_the_kind_of_cache_chooses_the_call(fake):
    import torch
    q, plan = fake, _kv_plan(fake)
    c, a = _codes(torch)
    quant = q.QuantKVCache(c, c, a, a, 8)
    plain = q.KVCache(torch.zeros((3, 2, 16, 128), dtype=torch.bfloat16), torch.zeros((3, 2, 16, 128), dtype=torch.bfloat16))
    x, kv = torch.zeros((2, 512), dtype=torch.bfloat16), torch.zeros((2, 256), dtype=torch.bfloat16)
    lens, table = torch.zeros(2, dtype=torch.int32), torch.zeros((2, 3), dtype=torch.int32)
    for cache, prefix in ((quant, "qmm_kvq_"), (plain, "qmm_")):
        q.attention(plan, x, cache, table, lens, x, stream=0)
        q.qk_norm_rope(plan, x, kv, kv, None, None, None, lens, table, cache, x, stream=0)
        assert [n for n, _ in q._LIB.calls[-2:]] == [prefix + "attention", prefix + "qk_norm_rope"]
    other = q.QuantKVCache(*(t[:, :1] for t in (c, c, a, a)), 8)   # another number of heads
    with pytest.raises(ValueError, match="pages"):
        q.attention(plan, x, other, table, lens, x, stream=0)


def test_refusals_of_the_read_back(fake):
    import torch
    q, plan = fake, _kv_plan(fake)
    c, a = _codes(torch)
    cache = q.QuantKVCache(c, c, a, a, 8)
    lens, table = torch.zeros(2, dtype=torch.int32), torch.zeros((2, 3), dtype=torch.int32)
    out = torch.zeros((2, 5, 2, 128))
    good = dict(cache=cache, page_table=table, lengths=lens, k_out=out, v_out=out.clone(), starts=None)
    q.kv_read(plan, **good, stream=0)
    args = q.QmmReadArgs.from_buffer_copy(q._LIB.calls[-1][1][2])
    assert (args.seqs, args.rows, args.out_dtype, args.k_seq_stride, args.k_row_stride) == (2, 5, 0, 1280, 256)
    q.kv_read(plan, **{**good, "k_out": torch.zeros((5, 2, 2, 128)).transpose(0, 1)}, stream=0)
    plain = q.KVCache(torch.zeros((3, 2, 16, 128), dtype=torch.bfloat16), torch.zeros((3, 2, 16, 128), dtype=torch.bfloat16))
    n = len(q._LIB.calls)
    for change in (dict(cache=plain), dict(k_out=out.half()), dict(v_out=out.to(torch.bfloat16)), dict(v_out=out[:, :4]),
                   dict(k_out=out[:1]), dict(k_out=out[0]), dict(k_out=out[..., :64]), dict(k_out=out.transpose(2, 3)),
                   dict(k_out=torch.zeros((2, 5, 2, 256))[..., :128]), dict(starts=lens.long()), dict(starts=lens[:1]),
                   dict(lengths=lens.long()), dict(page_table=table[:, :2]), dict(lengths=torch.zeros(3, dtype=torch.int32)),
                   dict(k_out=_elsewhere(out)), dict(starts=_elsewhere(lens)), dict(page_table=_elsewhere(table))):
        with pytest.raises(ValueError):
            q.kv_read(plan, **{**good, **change}, stream=0)
    assert len(q._LIB.calls) == n


def test_refusals_of_adapters(fake):
    import torch
    q = fake
    plan = q.AdapterPlan(128, 70, 8, 3, 6, out_dtype="f32", torch_workspace=False, device="cpu:0")
    plan._device_index = -1
    bf = torch.bfloat16
    good = dict(x=torch.zeros((4, 128), dtype=bf), a=torch.zeros((3, 8, 128), dtype=bf), b=torch.zeros((3, 70, 8), dtype=bf),
                scale=torch.ones(3), ids=torch.zeros(4, dtype=torch.int32), y=torch.zeros((4, 70)), out=torch.zeros((4, 70)))
    q.add_adapters(plan, **good, stream=0)
    args = q.QmmAdapterArgs.from_buffer_copy(q._LIB.calls[-1][1][1])
    assert (args.rows, args.x_stride, args.y_stride, args.out_stride) == (4, 128, 70, 70)
    q.add_adapters(plan, **{**good, "scale": None, "y": good["out"]}, stream=0)
    q.add_adapters(plan, **{**good, "out": torch.zeros((4, 100))[:, 7:77]}, stream=0)
    n = len(q._LIB.calls)
    g = good
    for change in (dict(x=g["x"].float()), dict(x=g["x"][:, :64]), dict(x=g["x"][0]), dict(a=g["a"].float()), dict(a=g["a"][:2]),
                   dict(a=g["a"].transpose(1, 2)), dict(b=g["b"].transpose(1, 2)), dict(b=g["b"][:, :, :4]), dict(scale=torch.ones(2)),
                   dict(scale=torch.ones(3).double()), dict(ids=g["ids"].long()), dict(ids=g["ids"][:3]), dict(y=g["y"].to(bf)),
                   dict(out=g["out"].to(bf)), dict(y=g["y"][:3]), dict(out=torch.zeros((70, 4)).T), dict(out=torch.zeros((4, 140))[:, ::2]),
                   dict(x=_elsewhere(g["x"])), dict(ids=_elsewhere(g["ids"])), dict(out=_elsewhere(g["out"]))):
        with pytest.raises(ValueError):
            q.add_adapters(plan, **{**good, **change}, stream=0)
    assert len(q._LIB.calls) == n


def test_refusals_of_log_probabilities(q):
    import torch
    l, t, f = torch.zeros((3, 10)), torch.zeros(3, dtype=torch.int32), torch.zeros(3)
    tt, tl = torch.zeros((3, 2), dtype=torch.int32), torch.zeros((3, 2))
    for args in ((l.half(), t, f), (l[0], t, f), (l.T, t, f), (l, t.long(), f), (l, t, f.double()), (l, t, None), (l, None, f),
                 (l, t[:2], f), (l, t, f, f[:2]), (l, t, f, None, tt, None), (l, t, f, None, None, tl), (l, t, f, None, tt, tl[:, :1]),
                 (l, t, f, None, tt.long(), tl), (l, t, f, None, tt.T.contiguous(), tl.T.contiguous()), (l, t, f, None, tt[0], tl[0]),
                 (l, t, f)):
        with pytest.raises(ValueError):
            q.logprobs(*args)

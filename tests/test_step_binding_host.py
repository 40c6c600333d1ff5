"""Host-only tests of the Python entry points of the cache operators and of sampling, with a library in the place of the real
one that takes note of what it is passed. CPU tensors stand for those of the plan's device."""
from __future__ import annotations

import contextlib
import ctypes
import threading

import pytest

HQ, HKV, D, PAGE, MAX_PAGES, SEQS = 4, 2, 64, 16, 3, 2
KIND = {"qmm_attention": "QmmAttentionArgs", "qmm_qk_norm_rope": "QmmAppendArgs"}


class Library:
    """The real library, but for the calls that need a GPU."""

    def __init__(self, q):
        self.q, self.real, self.calls, self.inside = q, q.lib, [], lambda: None

    def __getattr__(self, name):
        if name == "qmm_kv_plan":
            return lambda *a: 0
        if name == "qmm_sample":
            return lambda *a: self.calls.append(a) or 0
        if name not in KIND:
            return getattr(self.real, name)

        def call(handle, cache, args, stream):
            self.inside()   # what other threads do before the library has read the arguments
            kind = getattr(self.q, KIND[name])
            raw = args if isinstance(args, bytes) else ctypes.string_at(args, ctypes.sizeof(kind))
            self.calls.append(kind.from_buffer_copy(raw))
            return 0
        return call


@pytest.fixture
def q(monkeypatch):
    torch = pytest.importorskip("torch")
    from bit_affine_quantized_group_gb300 import _build
    _build.build()
    import bit_affine_quantized_group_gb300 as q
    monkeypatch.setattr(q, "_LIB", Library(q))
    monkeypatch.setattr(torch.cuda, "device", lambda d: contextlib.nullcontext())
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    q._bind_torch()
    monkeypatch.setattr(q, "_CURRENT_DEVICE", lambda: 3, raising=False)
    return q


@pytest.fixture
def plan(q):
    p = q.KVPlan(HQ, HKV, D, PAGE, max_seqs=SEQS, max_rows=4, max_pages=MAX_PAGES, torch_workspace=False, device="cpu:0")
    p._device_index = -1   # what CPU tensors give for their device
    return p


class Args:
    """Arguments of a step that fit; changed by name."""

    def __init__(self, q, tokens=SEQS):
        import torch
        self.q_, self.tokens = q, tokens
        cache = lambda: torch.zeros((5, HKV, PAGE, D), dtype=torch.bfloat16)  # noqa: E731
        rows = lambda heads: torch.zeros((tokens, heads * D), dtype=torch.bfloat16)  # noqa: E731
        seqs = 1 if tokens == 1 else SEQS
        self.queries, self.keys, self.values, self.out = rows(HQ), rows(HKV), rows(HKV), rows(HQ)
        self.cache = q.KVCache(cache(), cache())
        self.weight = torch.ones(D)
        self.rope = torch.zeros((50, D))
        self.positions = None
        self.lengths = torch.zeros(seqs, dtype=torch.int32)
        self.table = torch.zeros((seqs, MAX_PAGES), dtype=torch.int32)

    def append(self, plan, **kw):
        a = {**self.__dict__, **kw}
        self.q_.qk_norm_rope(plan, a["queries"], a["keys"], a["values"], a["weight"], a["weight"], a["rope"], a["lengths"],
                             a["table"], a["cache"], a["out"], a["positions"], stream=0)

    def attend(self, plan, **kw):
        a = {**self.__dict__, **kw}
        self.q_.attention(plan, a["queries"], a["cache"], a["table"], a["lengths"], a["out"], stream=0)


def test_two_threads_share_a_plan(q, plan):
    """Another thread's call, of either operator, between a call's packing of its arguments and the library's reading."""
    one, two = Args(q), Args(q)
    for mine in (one.attend, one.append):
        for theirs in (two.attend, two.append):
            q._LIB.calls.clear()

            def other():
                q._LIB.inside = lambda: None
                t = threading.Thread(target=theirs, args=(plan,))
                t.start()
                t.join()

            q._LIB.inside = other
            mine(plan)
            second, first = q._LIB.calls
            assert type(first) is getattr(q, KIND["qmm_attention" if mine == one.attend else "qmm_qk_norm_rope"])
            assert first.q == one.queries.data_ptr() and first.lengths == one.lengths.data_ptr()
            assert second.q == two.queries.data_ptr() and second.lengths == two.lengths.data_ptr()
            assert (first.seqs, first.rows) == (SEQS, 1)


@pytest.mark.parametrize("shape", [(D,), (50 * D,), (2, 25, D), (50, 1, D), (50, D // 2), ()])
def test_the_rotation_table_has_two_dimensions(q, plan, shape):
    """Its first is the number of positions that the kernel holds positions against."""
    import torch
    a = Args(q)
    with pytest.raises(ValueError, match="rope"):
        a.append(plan, rope=torch.zeros(shape))
    assert not q._LIB.calls
    a.append(plan)
    assert q._LIB.calls[0].rope_len == 50


def _wide(heads, tokens=None):
    """Heads with gaps between them, as a slice of a wider tensor."""
    import torch
    shape = (heads, 2 * D) if tokens is None else (tokens, heads, 2 * D)
    return torch.zeros(shape, dtype=torch.bfloat16)[..., :D]


@pytest.mark.parametrize("name,heads", [("queries", HQ), ("keys", HKV), ("values", HKV), ("out", HQ)])
def test_rows_hold_all_their_heads_side_by_side(q, plan, name, heads):
    import torch
    for tokens in (1, SEQS):
        a = Args(q, tokens)
        t = getattr(a, name)
        wrong = [_wide(heads, tokens), t.view(tokens, heads, D).transpose(1, 2), torch.cat((t, t)), t[:, :-1], t.float(),
                 t.view(tokens, heads, 2, D // 2), t.view(-1)]
        if name != "queries":   # whose first dimension is the number of tokens
            wrong += [_wide(heads), t.view(tokens * heads, D)[::tokens] if tokens > 1 else _wide(2 * heads)[::2], t.new_zeros((tokens * heads * 2, D))[::2]]
        for w in wrong:
            if tokens == 1 and w.is_contiguous() and w.dtype is t.dtype and w.numel() == t.numel() and (name != "queries" or w.shape[0] == 1):
                continue   # one token's heads, whatever they are called
            with pytest.raises((ValueError, q.QmmError)):
                a.append(plan, **{name: w})
            if name in ("queries", "out"):
                with pytest.raises((ValueError, q.QmmError)):
                    a.attend(plan, **{name: w})
        assert not q._LIB.calls
        for fits in (t, t.view(tokens, heads, D), torch.cat((t, t), 1)[:, :heads * D], torch.cat((t, t), 1).view(tokens, 2 * heads, D)[:, :heads]):
            a.append(plan, **{name: fits})
        q._LIB.calls.clear()


def test_one_token_may_be_any_contiguous_tensor(q, plan):
    import torch
    a = Args(q, 1)
    a.append(plan, keys=a.keys.view(HKV, D), values=a.values.view(HKV, D), out=a.out.view(HQ, D))
    a.attend(plan, out=a.out.view(HQ, D))
    one = torch.zeros((1, SEQS, D), dtype=torch.bfloat16).transpose(0, 1)   # one head a token: its stride says nothing
    single = q.KVPlan(1, 1, D, PAGE, max_seqs=SEQS, max_rows=1, max_pages=MAX_PAGES, torch_workspace=False, device="cpu:0")
    single._device_index = -1
    b = Args(q)
    pool = torch.zeros((5, 1, PAGE, D), dtype=torch.bfloat16)
    b.attend(single, queries=one, out=one.clone(), cache=q.KVCache(pool, pool))
    assert q._LIB.calls[-1].q_stride == D


def _elsewhere(t):
    """t, as a tensor that says that it is on another device."""
    import torch

    class Elsewhere(torch.Tensor):
        def get_device(self):
            return 3
    return t.as_subclass(Elsewhere)


def test_tensors_of_another_device_are_refused(q, plan):
    import torch
    a = Args(q)
    positions = torch.zeros(SEQS, dtype=torch.int32)
    a.append(plan, positions=positions)
    a.attend(plan)
    q._LIB.calls.clear()
    for name in ("queries", "keys", "values", "weight", "rope", "lengths", "table", "out"):
        with pytest.raises(ValueError, match="device"):
            a.append(plan, **{name: _elsewhere(getattr(a, name))})
    with pytest.raises(ValueError, match="device"):
        a.append(plan, positions=_elsewhere(positions))
    for name in ("queries", "lengths", "table", "out"):
        with pytest.raises(ValueError, match="device"):
            a.attend(plan, **{name: _elsewhere(getattr(a, name))})
    with pytest.raises(ValueError, match="device"):
        q.KVCache(a.cache.k, _elsewhere(a.cache.v))
    far = q.KVCache(_elsewhere(a.cache.k), _elsewhere(a.cache.v))
    for call in (a.append, a.attend):
        with pytest.raises(ValueError, match="device"):
            call(plan, cache=far)
    plan._device_index = 0   # a plan on a GPU, and tensors on the CPU
    for call in (a.append, a.attend):
        with pytest.raises(ValueError, match="device"):
            call(plan)
    assert not q._LIB.calls


def test_sampling_refuses_tensors_of_another_device(q):
    import torch
    names = ("logits", "temperature", "top_k", "top_p", "min_p", "u", "tokens", "probs")
    f, i = torch.zeros(2), torch.zeros(2, dtype=torch.int32)
    plain = dict(zip(names, (torch.zeros((2, 10)), f, i, f, f, f, i, f)))
    with pytest.raises(ValueError, match="device"):
        q.sample(**plain, stream=0)
    far = {n: _elsewhere(t) for n, t in plain.items()}
    for name in names:
        with pytest.raises(ValueError, match="device"):
            q.sample(**{**far, name: plain[name]}, stream=0)
    assert not q._LIB.calls
    q.sample(**far, stream=0)
    assert len(q._LIB.calls) == 1


def test_sampling_launches_on_the_logits_device(q, monkeypatch):
    """Where another device is current, that of the logits is made the current one around the call."""
    import torch
    events = []

    @contextlib.contextmanager
    def device(d):
        events.append(("enter", d))
        yield
        events.append(("exit", d))

    monkeypatch.setattr(torch.cuda, "device", device)
    f, i = _elsewhere(torch.zeros(2)), _elsewhere(torch.zeros(2, dtype=torch.int32))
    logits = _elsewhere(torch.zeros((2, 10)))
    q.sample(logits, f, i, f, f, f, i, stream=0)
    assert events == [] and len(q._LIB.calls) == 1
    monkeypatch.setattr(q, "_CURRENT_DEVICE", lambda: 1)
    monkeypatch.setattr(q._LIB, "calls", events)   # in one list with the calls
    q.sample(logits, f, i, f, f, f, i, stream=0)
    assert [e[0] for e in events] == ["enter", logits.data_ptr(), "exit"] and events[0][1] == 3


@pytest.mark.parametrize("change", [{"kv_heads": 0}, {"kv_heads": -3}, {"q_heads": 0}, {"head_dim": 0}, {"head_dim": 96},
                                    {"page_size": 24}, {"max_rows": 17}])
def test_argument_checks_refuse_a_descriptor_that_is_not_valid(change):
    """As the check of the descriptor does, whatever the arguments, and without a division by its fields."""
    from bit_affine_quantized_group_gb300 import _build
    _build.build()
    import bit_affine_quantized_group_gb300 as q
    d = q.make_kv_desc(HQ, HKV, D, PAGE, SEQS, 4, MAX_PAGES)
    for name, value in change.items():
        setattr(d, name, value)
    want = q.kv_validate_desc(d)
    assert want != q.QMM_OK
    cache, attend, append = q.QmmKvCache(), q.QmmAttentionArgs(), q.QmmAppendArgs()
    assert q.lib.qmm_check_attention_args(ctypes.byref(d), ctypes.byref(cache), ctypes.byref(attend)) == want
    assert q.lib.qmm_check_qk_norm_rope_args(ctypes.byref(d), ctypes.byref(cache), ctypes.byref(append)) == want

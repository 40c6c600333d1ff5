"""Log probabilities of given tokens, entropy and alternatives against float64.

Tolerances, from the arithmetic: an exponential is off by at most 2^-22 of its value and, for its argument d = l - max rounded
in float32 and times log2(e), by |d| 2^-22; sums are of float32 terms of one sign, a thread's of at most some hundred and the
rest by trees: 2^-15 covers all of it for the sum and for the sum of e^d d, relative to them. So the log of the sum is off by 2^-15 and
its own rounding, and the entropy, log s - t / s, by 2^-14 (1 + t / s). Differences l - max are rounded once (2^-24)."""
from __future__ import annotations

import numpy as np
import pytest

pytestmark = pytest.mark.gpu

DEV = "cuda"


@pytest.fixture(scope="module")
def q():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from bit_affine_quantized_group_gb300 import _build
    _build.build()
    import bit_affine_quantized_group_gb300 as q
    return q


def _run(q, logits, tokens, top):
    import torch
    M = logits.shape[0]
    full = lambda *s, t=torch.float32: torch.full(s, 77, dtype=t, device=DEV)  # noqa: E731
    lp, h, tt, tl = full(M), full(M), full(M, top, t=torch.int32), full(M, top)
    q.logprobs(logits, torch.tensor(tokens, dtype=torch.int32, device=DEV), lp, h, tt if top else None, tl if top else None)
    torch.cuda.synchronize()
    return [t.cpu().numpy() for t in (lp, h, tt, tl)]


def _check(q, logits, tokens, top):
    """logits: a tensor on the device of finite numbers, infinities and NaN."""
    import torch
    lp, h, tt, tl = _run(q, logits, tokens, top)
    l = logits.float().cpu().numpy().astype(np.float64)
    l = np.where(np.isnan(l), -np.inf, np.minimum(l, float(np.finfo(np.float32).max)))
    M, V = l.shape
    for m in range(M):
        best = l[m].max()
        if best == -np.inf:
            assert lp[m] == -np.inf and h[m] == 0
            want = np.full(V, -np.inf)
        else:
            d = l[m] - best
            w = np.exp(d)
            s = w.sum()
            want = d - np.log(s)
            t = -np.sum(w[w > 0] * d[w > 0]) / s
            assert abs(h[m] - (np.log(s) + t)) <= 2.0 ** -14 * (1 + t) + 2.0 ** -23 * np.log(s)
            if 0 <= tokens[m] < V and want[tokens[m]] > -np.inf:
                assert abs(lp[m] - want[tokens[m]]) <= 2.0 ** -15 + 2.0 ** -22 * abs(want[tokens[m]])
            else:
                assert lp[m] == -np.inf
        order = np.argsort(-l[m], kind="stable")[:top]
        assert list(tt[m, :len(order)]) == list(order)
        assert (tt[m, len(order):] == -1).all() and (tl[m, len(order):] == -np.inf).all()
        for i, j in enumerate(order):
            if want[j] == -np.inf:
                assert tl[m, i] == -np.inf
            else:
                assert abs(tl[m, i] - want[j]) <= 2.0 ** -15 + 2.0 ** -22 * abs(want[j])


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
@pytest.mark.parametrize("M,V,top", [(1, 1, 1), (1, 2, 5), (2, 7, 3), (1, 31, 32), (3, 100, 20), (1, 513, 5), (5, 4097, 32),
                                     (1, 32000, 1), (2, 151936, 5), (9, 50257, 20), (40, 33000, 8), (20, 100277, 0),
                                     (160, 8193, 4), (400, 3001, 32), (1, 393216, 32)])
def test_shapes(q, dtype, M, V, top):
    """Many equal logits among those of bfloat16."""
    import torch
    gen = torch.Generator(device=DEV).manual_seed(M + V)
    l = (3.0 * torch.randn((M, V), generator=gen, device=DEV)).to(getattr(torch, dtype))
    tokens = torch.randint(V, (M,), generator=gen, device=DEV).tolist()
    _check(q, l, tokens, top)


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
@pytest.mark.parametrize("M", [1, 3, 12, 320])
def test_orders_and_ties(q, dtype, M):
    """Rising and falling logits, all equal ones, few levels, and rows that differ by one element."""
    import torch
    V = 20011
    i = torch.arange(V, dtype=torch.float32, device=DEV)
    rows = [i * 1e-3, -i * 1e-3, 0 * i + 2.5, (i % 3), torch.where(i == V - 1, 5.0, 0.0), torch.where(i == 0, -5.0, 0.0),
            torch.floor(i / 7000), -0.0 * (i % 2 - 0.5)]
    l = torch.stack([rows[m % len(rows)] for m in range(M)]).to(getattr(torch, dtype))
    for top in (1, 5, 32):
        _check(q, l, [(m * 7919) % V for m in range(M)], top)
        for r in range(min(M, 3)):
            _check(q, l[r:r + 1], [V - 1], top)


@pytest.mark.parametrize("M", [1, 3, 12, 320])
def test_every_order_alone(q, M):
    """The same row in every place of a call."""
    import torch
    V = 20011
    i = torch.arange(V, dtype=torch.float32, device=DEV)
    for row in (i * 1e-3, (i * 1e-3 % 1.0), torch.floor(i / 7000), 0 * i, (i % 512) * 1.0, torch.where(i % 512 == 77, i, 0 * i)):
        l = row.expand(M, V).contiguous()
        lp, h, tt, tl = _run(q, l, [3] * M, 32)
        assert (tt == tt[:1]).all()
        # V is odd, so that the 16-byte chunks that a thread takes begin at other logits in the next row, and float32 sums of
        # other parts differ in their last bits: by twice what each is off by. Every fourth row is cut alike.
        for g in (lp, h, tl):
            assert (g[::4] == g[:1]).all()
            assert (np.abs(g - g[:1]) <= 2 * (2.0 ** -14 + 2.0 ** -14 * np.abs(g[:1]))).all()
        _check(q, l[:1], [3], 32)


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
@pytest.mark.parametrize("V", [40, 5000, 70001])
def test_masked_logits(q, dtype, V):
    import torch
    inf = float("inf")
    gen = torch.Generator(device=DEV).manual_seed(V)
    l = torch.randn((9, V), generator=gen, device=DEV)
    l[0] = -inf
    l[1] = float("nan")
    l[2, 1:] = -inf
    l[3, :-1] = -inf
    l[4, ::2] = float("nan")
    l[5, 7] = inf
    l[6, 3:9] = inf
    l[7] = torch.finfo(torch.float32).min
    l[8] = torch.where(torch.arange(V, device=DEV) % 97 == 5, l[8], -inf)
    l = l.to(getattr(torch, dtype))
    tokens = [0, 1, 0, V - 1, 2, 7, 4, 0, 5]
    for top in (1, 4, 32):
        _check(q, l, tokens, top)
        for m in range(9):
            _check(q, l[m:m + 1], tokens[m:m + 1], top)


def test_near_certain_tokens(q):
    import torch
    l = torch.zeros((3, 1000), device=DEV)
    l[0, 5], l[1, 5], l[2, 5] = 20.0, 60.0, 1e30
    _check(q, l, [5, 5, 5], 3)
    _check(q, l, [6, 6, 6], 3)


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
def test_strided_rows_and_odd_places(q, dtype):
    import torch
    wide = torch.randn((7, 9001), device=DEV).to(getattr(torch, dtype))
    for a in range(9):
        l = wide[:, a:a + 8191]
        _check(q, l, [0, 8190, 5, 6, 7, 8, 9], 6)


def test_tokens_outside_and_parts_alone(q):
    import torch
    l = torch.randn((4, 3000), device=DEV)
    _check(q, l, [-1, 3000, 2 ** 31 - 1, -2 ** 31], 2)
    lp, h, tt, tl = _run(q, l, [1, 2, 3, 4], 3)
    only = torch.empty(4, device=DEV)
    q.logprobs(l, torch.tensor([1, 2, 3, 4], dtype=torch.int32, device=DEV), only)
    assert (only.cpu().numpy() == lp).all()
    q.logprobs(l, None, None, only)
    assert (only.cpu().numpy() == h).all()
    t, v = torch.empty((4, 3), dtype=torch.int32, device=DEV), torch.empty((4, 3), device=DEV)
    q.logprobs(l, None, None, None, t, v)
    assert (t.cpu().numpy() == tt).all() and (v.cpu().numpy() == tl).all()
    q.logprobs(l[:0], t[:0, 0].contiguous(), only[:0])


def test_after_sampling_in_a_graph(q):
    """A drawn token's log probability is that of sampling without limits, replayed with other logits."""
    import torch
    M, V = 6, 32000
    gen = torch.Generator(device=DEV).manual_seed(0)
    l = torch.randn((M, V), generator=gen, device=DEV)
    f = lambda v, t=torch.float32: torch.full((M,), v, dtype=t, device=DEV)  # noqa: E731
    one, zero, k = f(1.0), f(0.0), f(0, torch.int32)
    u = torch.rand(M, generator=gen, device=DEV)
    tokens, probs, lp, h = f(0, torch.int32), f(0.0), f(0.0), f(0.0)

    def step():
        q.sample(l, one, k, one, zero, u, tokens, probs)
        q.logprobs(l, tokens, lp, h)

    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        step()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=stream):
            step()
        for turn in range(3):
            l.copy_(torch.randn((M, V), generator=gen, device=DEV) * (1 + turn))
            g.replay()
            stream.synchronize()
            # weights of sampling are whole numbers of 2^-40, at most 2^-40 V short of the sum, and 2^-20 of it in all
            assert torch.allclose(lp.exp(), probs, rtol=1e-4, atol=0)

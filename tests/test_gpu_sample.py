"""Sampling against the definition in float64. Every expected token is exact: the random numbers lie in the middle of
a kept token's share of the mass, and top_p in the middle of a token's share of the ranking, so float32 rounding of the
weights cannot decide. The probability is a ratio of float32 weights: off by at most 2^-18 of itself (the exponent's
rounding at 40 units, the exponential's own and two conversions)."""
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


def _masses(l, T):
    """Order (value falling, index rising) and whole-number weights of one row of float64 logits."""
    l = np.where(np.isnan(l), -np.inf, l)
    order = np.lexsort((np.arange(len(l)), -l))
    top = l[order[0]]
    w = np.zeros(len(l))
    fin = l > -np.inf
    w[fin] = np.where(l[fin] == top, 1.0, np.exp((l[fin] - top) / T))
    return order, w, np.floor(w * 2.0 ** 40)


def _kept(l, T, k, p, min_p):
    """Kept mass by index (zeros elsewhere)."""
    order, w, m = _masses(l, T)
    keep = np.zeros(len(l), bool)
    n = k if 0 < k < len(l) else len(l)
    ranked = m[order][:n]
    before = np.cumsum(ranked) - ranked
    ok = np.ones(n, bool) if not p < 1 else before < p * ranked.sum()
    ok &= ~(w[order][:n] < min_p)
    ok[0] = True
    keep[order[:n][ok]] = True
    return np.where(keep, m, 0.0)


def _top_p_between(l, T, k, want):
    """A top_p that keeps `want` tokens of the top k, in the middle of the last one's share."""
    order, _, m = _masses(l, T)
    n = k if 0 < k < len(l) else len(l)
    c = np.cumsum(m[order][:n]) / m[order][:n].sum()
    i = min(want, n) - 1
    return float(np.float32((c[i] + (c[i - 1] if i else 0.0)) / 2))


def _run(q, torch, logits, T, k, p, min_p, u, stride=None, offset=0):
    M, V = logits.shape
    buf = torch.full((M, (stride or V) + offset), 1e30, dtype=logits.dtype)
    buf[:, offset:offset + V] = logits
    dev = buf.to(DEV)[:, offset:offset + V]
    f = lambda a, t: torch.tensor(np.asarray(a), dtype=t).to(DEV)  # noqa: E731
    tokens = torch.full((M,), -9, dtype=torch.int32, device=DEV)
    probs = torch.full((M,), -9.0, device=DEV)
    q.sample(dev, f(T, torch.float32), f(k, torch.int32), f(p, torch.float32), f(min_p, torch.float32), f(u, torch.float32),
             tokens, probs)
    torch.cuda.synchronize()
    again = torch.empty_like(tokens)
    q.sample(dev, f(T, torch.float32), f(k, torch.int32), f(p, torch.float32), f(min_p, torch.float32), f(u, torch.float32), again)
    assert torch.equal(tokens, again)
    return tokens.cpu().numpy(), probs.double().cpu().numpy()


def _check(q, torch, logits, T, k, p, min_p, seed, **kw):
    """Rows of logits, each with its parameters; several draws a row, each aimed at a kept token of its own."""
    rng = np.random.default_rng(seed)
    M, V = logits.shape
    l64 = logits.double().numpy()
    for _ in range(3):
        u, want, prob = np.zeros(M), np.zeros(M, int), np.zeros(M)
        for r in range(M):
            m = _kept(l64[r], np.float64(np.float32(T[r])), k[r], np.float64(np.float32(p[r])), np.float64(np.float32(min_p[r])))
            c = np.cumsum(m)
            heavy = np.nonzero(m > 3e-6 * c[-1])[0]
            want[r] = rng.choice(heavy)
            u[r] = (c[want[r]] - 0.5 * m[want[r]]) / c[-1]
            prob[r] = m[want[r]] / c[-1]
        tokens, probs = _run(q, torch, logits, T, k, p, min_p, u, **kw)
        assert (tokens == want).all(), (tokens, want)
        assert (np.abs(probs - prob) <= 2.0 ** -18 * prob).all()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("V", [1, 2, 31, 1000, 4097, 40003, 151936])
@pytest.mark.parametrize("mode", ["plain", "top_k", "top_p", "both", "min_p", "all"])
def test_modes(q, dtype, V, mode):
    import torch
    gen = torch.Generator().manual_seed(V + len(mode))
    M = 3
    logits = (torch.randn((M, V), generator=gen) * 2.5).to(torch.float32 if dtype == "f32" else torch.bfloat16)
    T = [0.7, 1.0, 1.6]
    k = [0, 0, 0] if mode not in ("top_k", "both", "all") else [2, 50, 1500]
    p, min_p = [1.0] * M, [0.0] * M
    if mode in ("top_p", "both", "all"):
        want = [1, 30, 700]
        p = [_top_p_between(logits[r].double().numpy(), np.float64(np.float32(T[r])), k[r], want[r]) for r in range(M)]
    if mode in ("min_p", "all"):
        min_p = [0.5, 0.0137, 1e-4]
    _check(q, torch, logits, T, k, p, min_p, V)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("M", [1, 2, 10, 17, 40])
def test_rows(q, dtype, M):
    """One row and many: the number of rows decides how many CTAs share one."""
    import torch
    gen = torch.Generator().manual_seed(M)
    logits = (torch.randn((M, 50021), generator=gen) * 2.5).to(torch.float32 if dtype == "f32" else torch.bfloat16)
    l = logits.double().numpy()
    k = [(0, 30)[r % 2] for r in range(M)]
    p = [_top_p_between(l[r], 1.0, k[r], (900, 12)[r % 2]) for r in range(M)]
    _check(q, torch, logits, [1.0] * M, k, p, [0.0] * M, M)


@pytest.mark.parametrize("V", [5000, 30001])
@pytest.mark.parametrize("spread", [0.0, 1e-6, 0.01, 0.3])
def test_flat_rows(q, V, spread):
    """More members of one bin than are ranked one by one: equal logits, and ones that differ in their last bits."""
    import torch
    gen = torch.Generator().manual_seed(V)
    base = torch.randn((1, V), generator=gen)
    logits = (3.0 + spread * base).float().repeat(4, 1)
    T, k = [1.0] * 4, [0, 2500, 0, 4000]
    l = logits[0].double().numpy()
    p = [_top_p_between(l, 1.0, 0, 2000), 1.0, _top_p_between(l, 1.0, 0, V - 7), _top_p_between(l, 1.0, 4000, 1700)]
    _check(q, torch, logits, T, k, p, [0.0] * 4, V)


def test_ties_go_to_the_lowest_index(q):
    import torch
    logits = torch.zeros((4, 9000))
    logits[:, 100::7] = 2.0   # 1272 equal largest ones
    logits[1] = -logits[1]    # and 0 against -0
    logits[1, ::2] = 0.0
    k = [5, 3, 0, 1272]
    _check(q, torch, logits, [0.01, 0.01, 0.01, 1.0], k, [1.0, 1.0, 0.5004, 1.0], [0.0] * 4, 5)
    tokens, probs = _run(q, torch, logits, [0.0, 0.0, -1.0, 1.0], [0, 0, 0, 1], [1.0] * 4, [0.0] * 4, [0.9] * 4)
    first = [int(np.argmax(r.double().numpy())) for r in logits]
    assert (tokens == first).all() and (probs == 1.0).all()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("stride,offset", [(1007, 0), (1008, 1), (1009, 3), (1003, 7)])
def test_strides_and_alignment(q, dtype, stride, offset):
    import torch
    gen = torch.Generator().manual_seed(stride)
    logits = (torch.randn((5, 1003), generator=gen) * 2).to(torch.float32 if dtype == "f32" else torch.bfloat16)
    l = logits.double().numpy()
    p = [_top_p_between(l[r], 1.0, 40, 9) for r in range(5)]
    _check(q, torch, logits, [1.0] * 5, [40] * 5, p, [0.0] * 5, stride, stride=stride, offset=offset)


def test_masked_rows(q):
    """Rows that a grammar leaves one token, few or none; the type's lowest value and NaN in place of masked logits."""
    import torch
    gen = torch.Generator().manual_seed(6)
    V = 20000
    logits = torch.randn((6, V), generator=gen)
    logits[0] = -float("inf")
    logits[1] = float("nan")
    logits[2, :] = -float("inf")
    logits[2, 17777] = -3.0
    logits[3, 5:] = torch.finfo(torch.float32).min
    logits[4, ::2] = float("nan")
    logits[5, 1:] = -float("inf")
    logits[5, 0] = torch.finfo(torch.float32).min
    T, k, p = [1.0] * 6, [0, 7, 50, 0, 20, 3], [0.9, 1.0, 0.9, 0.999, 1.0, 0.5]
    u = [0.3] * 6
    tokens, probs = _run(q, torch, logits, T, k, p, [0.0] * 6, u)
    assert tokens[0] == -1 and tokens[1] == -1 and probs[0] == 0 and probs[1] == 0
    assert tokens[2] == 17777 and probs[2] == 1 and tokens[5] == 0 and probs[5] == 1
    assert 0 <= tokens[3] < 5 and tokens[4] % 2 == 1
    _check(q, torch, logits[2:], T[2:], k[2:], [0.9, 1.0, 1.0, 0.5], [0.0] * 4, 7)


def test_infinite_logits_share_the_mass(q):
    import torch
    logits = torch.zeros((2, 3000))
    logits[:, [7, 2999]] = float("inf")
    tokens, probs = _run(q, torch, logits, [1.0, 1.0], [0, 50], [1.0, 0.9], [0.0, 0.0], [0.2, 0.8])
    assert list(tokens) == [7, 2999] and (probs == 0.5).all()


def test_parameters_at_their_ends(q):
    import torch
    gen = torch.Generator().manual_seed(8)
    logits = torch.randn((8, 5001), generator=gen) * 3
    top = logits.argmax(1).numpy()
    nan = float("nan")
    # top_p of 0 or less, min_p above 1, T of 0 or NaN, top_k = 1: the largest one
    tokens, probs = _run(q, torch, logits, [1, 1, 0, nan, 1, 1, 1, 1], [0, 0, 0, 0, 1, 0, -5, 9999], [0.0, 1, 1, 1, 1, -1, nan, 2],
                         [0, 1.5, 0, 0, 0, 0, 0, nan], [0.7] * 8)
    assert (tokens[:6] == top[:6]).all() and (probs[:6] == 1).all()
    # u at and outside the ends of [0, 1): the first and the last kept index
    m = _kept(logits[0].double().numpy(), 1.0, 30, 1.0, 0.0)
    ends = np.nonzero(m)[0][[0, -1]]
    same = logits[:1].repeat(5, 1)
    tokens, _ = _run(q, torch, same, [1] * 5, [30] * 5, [1] * 5, [0] * 5, [0.0, -1.0, 1.0, 7.0, nan])
    assert list(tokens) == [ends[0], ends[0], ends[1], ends[1], ends[0]]
    # extreme temperatures
    tokens, probs = _run(q, torch, same, [1e-30, 1e30, float("inf"), 1e-45, 1.0], [3] * 5, [1] * 5, [0] * 5, [0.5] * 5)
    order = np.argsort(-logits[0].numpy())[:3]
    assert tokens[0] == top[0] and tokens[3] == top[0] and tokens[1] == tokens[2] == np.sort(order)[1]


def test_largest_vocabulary(q):
    import torch
    gen = torch.Generator().manual_seed(9)
    logits = torch.randn((2, q.SAMPLE_MAX_VOCAB), generator=gen) * 2
    l = logits.double().numpy()
    p = [_top_p_between(l[r], 0.8, 0, 600) for r in range(2)]
    _check(q, torch, logits, [np.float32(0.8)] * 2, [0, 0], [1.0, 1.0], [0.0, 1e-5], 9)
    p = [_top_p_between(l[r], np.float64(np.float32(0.8)), 0, 600) for r in range(2)]
    _check(q, torch, logits, [0.8] * 2, [0, 0], p, [0.0, 0.0], 10, offset=1)


def test_shares_of_the_draws(q):
    """4096 draws of one row fall on its tokens in proportion: a chi-square within its 1e-6 tail."""
    import torch
    logits = torch.tensor([[0.0, 1.0, 2.0, -1.0, 0.5]]).repeat(4096, 1)
    u = (np.arange(4096) + 0.5) / 4096
    tokens, _ = _run(q, torch, logits, [1.0] * 4096, [0] * 4096, [1.0] * 4096, [0.0] * 4096, u)
    want = np.exp([0.0, 1.0, 2.0, -1.0, 0.5])
    want = want / want.sum() * 4096
    assert (np.abs(np.bincount(tokens, minlength=5) - want) <= 1.0).all()   # evenly spaced numbers


def test_graph_and_stream(q):
    import torch
    gen = torch.Generator().manual_seed(10)
    logits = (torch.randn((4, 50000), generator=gen) * 2).to(DEV)
    f = lambda v, t=torch.float32: torch.full((4,), v, dtype=t, device=DEV)  # noqa: E731
    args = (f(0.9), f(40, torch.int32), f(0.95), f(0.0))
    u, tokens, probs = torch.rand(4, generator=gen).to(DEV), f(0, torch.int32), f(0.0)
    q.sample(logits, *args, u, tokens, probs)
    torch.cuda.synchronize()
    eager = tokens.clone(), probs.clone()
    stream = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        q.sample(logits, *args, u, tokens, probs)
    tokens.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(tokens, eager[0]) and torch.equal(probs, eager[1])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("V", [1003, 33001])
@pytest.mark.parametrize("M", [39, 80, 153, 310])
def test_batches_agree(q, dtype, V, M):
    """A row's token and probability do not depend on how many rows share the call: the masses are whole numbers, and their
    sums the same for one CTA as for sixteen. Rows of every kind, next to one another."""
    import torch
    gen = torch.Generator().manual_seed(V + M)
    R = 22
    base = torch.randn((R, V + 3), generator=gen) * 2.2
    base[1] = 1.5                                    # equal logits
    base[2, ::2] = -float("inf")
    base[3] = torch.round(base[3])                   # many ties
    base[4] = -float("inf")                          # nothing to draw from
    base[5, 17:] = -float("inf")
    base[6] *= 1e-5
    base[7, 40] = float("nan")
    base[8, :V // 3] += 9.0                          # the likely ones in one part of the row
    base = base.to(torch.float32 if dtype == "f32" else torch.bfloat16).to(DEV)[:, 1:V + 1]
    T = [(1.0, 0.7, 1.3)[r % 3] for r in range(R)]
    k = [(0, 50, 0, 1000, 3)[r % 5] for r in range(R)]
    p = [(1.0, 0.9, 0.6, 1.0)[r % 4] for r in range(R)]
    min_p = [(0.0, 0.0, 0.02)[r % 3] for r in range(R)]
    T[9], k[10] = 0.0, 1
    u = torch.rand(M, generator=gen).tolist()
    rows = [r % R for r in range(M)]
    col = lambda v, t: torch.tensor([v[r] for r in rows], dtype=t).to(DEV)  # noqa: E731
    args = [col(T, torch.float32), col(k, torch.int32), col(p, torch.float32), col(min_p, torch.float32), torch.tensor(u).to(DEV)]
    logits = base[torch.tensor(rows).to(DEV)]
    tokens, probs = torch.full((M,), -9, dtype=torch.int32, device=DEV), torch.full((M,), -9.0, device=DEV)
    q.sample(logits, *args, tokens, probs)
    for i in range(0, M, 5):
        few = slice(i, min(i + 5, M))
        t, pr = torch.full((M,), -9, dtype=torch.int32, device=DEV)[few], torch.full((M,), -9.0, device=DEV)[few]
        q.sample(logits[few], *(a[few] for a in args), t, pr)
        assert torch.equal(t, tokens[few]), (i, t, tokens[few])
        assert torch.equal(pr, probs[few])

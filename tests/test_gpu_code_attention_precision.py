"""Attention over a cache of codes where terms of an output cancel, so that the precision of weights and sums shows.

Keys have the scale 0, so that a score is its position's bias: the products' sums are exact, and a weight is off by the rounding
of its exponent (|score| 2^-23, and 2^-24 of 15 for the power that weights are held at) and by ex2.approx (2^-22), 2^-18 in all
for scores down to -10. With weights P relative to the largest a position's share of an output of up to 16 rows is off by
    (2^-19 P + 2^-37) (|s| top + |b|) + 2^-30
with top = 255 or 15: the weight's two binary16 terms (2^-21 of it, or 2^-24 where the largest weight is 2^15 or, of 4 bits, 2^13),
its product with the scale in two terms (2^-21 and three roundings of subnormal numbers, 2^-25 each, times a code), and products
that the tensor cores cut at 2^-24 of the largest of 16, codes being subnormal numbers. The output is rounded once (2^-8)."""
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


def _run(q, bits, d, group, scores, code, scale, bias, page=64):
    """One token of every sequence, with `group` equal query heads of ones. scores: [seqs, n, heads]; code, scale, bias: of the
    values, [seqs, n, heads, d / 64], the same for all 64 columns of a group. Returns the outputs [seqs, heads, group, d / 64]
    of the groups, and what they should be, and by how much they may be off."""
    import torch
    S, n, H = scores.shape
    G, pages = d // 64, -(-n // page)
    half = lambda x: x.astype(np.float16)  # noqa: E731
    scores, scale, bias = half(scores), half(scale), half(bias)

    def paged(x):   # [seqs, n, heads, ...] to pages
        y = np.zeros((S, pages * page, *x.shape[2:]), x.dtype)
        y[:, :n] = x
        return torch.from_numpy(np.ascontiguousarray(y.reshape(S * pages, page, *x.shape[2:]).swapaxes(1, 2))).to(DEV)

    byte = (code if bits == 8 else code | code << 4).astype(np.uint8)
    k = torch.zeros((S * pages, H, page, d * bits // 8), dtype=torch.uint8, device=DEV)
    v = paged(np.repeat(byte, 64 * bits // 8, 3))
    ka = paged(np.stack((np.zeros((S, n, H, G), np.float16), np.repeat(scores[..., None], G, 3)), 4))
    va = paged(np.stack((scale, bias), 4))
    plan = q.KVPlan(H * group, H, d, page, max_seqs=S, max_rows=1, max_pages=pages, rot_dim=0, scale=1.0 / d)
    cache = q.QuantKVCache(k, v, ka, va, bits)
    table = torch.arange(S * pages, dtype=torch.int32, device=DEV).view(S, pages)
    out = torch.empty((S, H * group, d), dtype=torch.bfloat16, device=DEV)
    q.attention(plan, torch.ones_like(out), cache, table, torch.full((S,), n, dtype=torch.int32, device=DEV), out)
    torch.cuda.synchronize()
    assert plan.error_flags() == 0
    got = out.double().cpu().numpy().reshape(S, H, group, G, 64)
    assert (got == got[..., :1]).all()
    a = scores.astype(np.float64)
    P = np.exp(a - a.max(1, keepdims=True))[..., None]
    s, b, top = scale.astype(np.float64), bias.astype(np.float64), 2 ** bits - 1
    L = P.sum(1)
    want = (P * (s * code + b)).sum(1) / L
    size = np.abs(s) * top + np.abs(b)
    off = (2.0 ** -17 * (P * np.abs(s * code + b)).sum(1) + ((2.0 ** -19 * P + 2.0 ** -37) * size + 2.0 ** -30).sum(1)) / L
    return got[..., 0], want[:, :, None], (off + 2.0 ** -8 * np.abs(want))[:, :, None]


@pytest.mark.parametrize("bits", [8, 4])
@pytest.mark.parametrize("d,group", [(64, 1), (128, 4), (128, 12), (256, 8), (256, 16), (64, 16)])
def test_weights_keep_more_bits_than_the_output(q, bits, d, group):
    """The last of three positions takes off what the first two add, to 11 bits: what is left is 2^-11 of the terms, and weights
    of one binary16 number would be off by as much."""
    rng = np.random.default_rng(bits + d + group)
    S, H, G, top = 24, 4, d // 64, 2 ** bits - 1
    scores = -8.0 * rng.random((S, 3, H))
    scores[:, 2] = -1.0 * rng.random((S, H))
    code = rng.integers(0, top + 1, (S, 3, H, G))
    scale = (0.2 + rng.random((S, 3, H, G))) * 4 / top
    bias = -2.0 + rng.random((S, 3, H, G))
    scale[:, 2] = 0
    a = scores.astype(np.float16).astype(np.float64)[..., None]
    v = scale.astype(np.float16).astype(np.float64) * code + bias.astype(np.float16)
    bias[:, 2] = -(np.exp(a[:, :2] - a[:, 2:]) * v[:, :2]).sum(1)
    got, want, off = _run(q, bits, d, group, scores, code, scale, bias)
    assert (np.abs(got - want) <= off).all(), np.max(np.abs(got - want) / off)


@pytest.mark.parametrize("bits", [8, 4])
@pytest.mark.parametrize("d,group", [(64, 2), (128, 4), (128, 16), (256, 1)])
def test_small_weights_on_large_values(q, bits, d, group):
    """The likeliest position has the value 0, the others weights down to 2^-45 of its and values of up to 65,000."""
    rng = np.random.default_rng(bits * d + group)
    S, n, H, G, top = 8, 7, 3, d // 64, 2 ** bits - 1
    scores = -31.0 * rng.random((S, n, H))
    code = rng.integers(0, top + 1, (S, n, H, G))
    scale = np.where(rng.random((S, n, H, G)) < 0.5, 0.0, (1.0 if bits == 8 else 7.0) * rng.random((S, n, H, G)))
    bias = 6.0e4 * rng.random((S, n, H, G))
    scores[:, 0], code[:, 0], scale[:, 0], bias[:, 0] = 0.0, 0, 0.0, 0.0
    got, want, off = _run(q, bits, d, group, scores, code, scale, bias)
    # (scores down to -31: their exponents round to |score| 2^-23 more)
    assert (np.abs(got - want) <= off + 2.0 ** -18 * np.abs(want)).all(), np.max(np.abs(got - want) / off)


@pytest.mark.parametrize("bits", [8, 4])
@pytest.mark.parametrize("d,group,n", [(128, 4, 4000), (64, 4, 4000), (256, 4, 4000), (128, 12, 3000)])
def test_long_sums_of_codes_and_biases(q, bits, d, group, n):
    """Equal weights, and values whose code and bias cancel: their sums are as long as a sequence, and the outputs hundreds of
    times smaller. The tensor cores cut what they add at 2^-24 of their largest term, always to the same side: of a step's 32
    positions that is 2^-20 of a code's share at most, of sums over all steps it grew with them."""
    rng = np.random.default_rng(bits + d + n)
    S, H, G, top = 80, 4, d // 64, 2 ** bits - 1
    code = rng.integers(top // 2, top + 1, (S, n, H, G))
    scale = np.full((S, n, H, G), (1.5 if bits == 8 else 6.0) * 2.0 / top)
    bias = -scale * code * (1.0 + 2.0 ** -6 * (rng.random((S, n, H, G)) - 0.5))
    got, want, off = _run(q, bits, d, group, np.zeros((S, n, H)), code, scale, bias)
    size = 2 * np.abs(bias).mean(1)[:, :, None]   # weights are powers of two, exact
    assert (np.abs(got - want) <= 2.0 ** -20 * size + 2.0 ** -8 * np.abs(want)).all(), np.max(np.abs(got - want) / size) * 2.0 ** 20


@pytest.mark.parametrize("bits", [8, 4])
@pytest.mark.parametrize("d,group", [(64, 20), (128, 32), (256, 17), (128, 64)])
def test_more_rows_round_keys_and_values_once(q, bits, d, group):
    """Of more than 16 rows s c + b is a binary16 number, and so is the weight: each rounded once (2^-11), whatever the group's
    middle: values of groups far from zero, in which small ones stand out."""
    rng = np.random.default_rng(bits + d + group)
    S, n, H, G, top = 8, 1, 3, d // 64, 2 ** bits - 1
    code = rng.integers(0, 2, (S, n, H, G))
    scale = (0.5 + rng.random((S, n, H, G))) * 60 / top
    bias = 2.0 ** -7 * (0.1 + rng.random((S, n, H, G)))
    got, want, _ = _run(q, bits, d, group, np.zeros((S, n, H)), code, scale, bias)
    assert (np.abs(got - want) <= (2.0 ** -8 + 2.0 ** -11 + 2.0 ** -19) * np.abs(want)).all(), np.max(np.abs(got - want) / np.abs(want))


@pytest.mark.parametrize("bits", [8, 4])
@pytest.mark.parametrize("d,group,rows", [(64, 5, 1), (128, 4, 4), (128, 10, 2), (128, 8, 8), (64, 16, 4), (256, 6, 4), (256, 8, 8)])
@pytest.mark.parametrize("q_shift,k_shift", [(0.0, 0.0), (2.0, 4.0), (0.0, 8.0)])
def test_keys_far_from_zero(q, bits, d, group, rows, q_shift, k_shift):
    """Keys whose groups lie far from zero, of which scores have only the differences. Over all outputs roundings to bfloat16 come to
    2^-7 / sqrt(12) of the numbers' powers of two, 0.0017 of the norm; of more than 16 rows weights and values are binary16
    numbers besides (2^-11 / sqrt(3) each): 2^-9 in all, and no more where keys are shifted, for they are not rounded."""
    import torch
    from tests._codes import quantise, pack, values
    gen = torch.Generator().manual_seed(bits + d + group)
    S, H, page, n = 2, 2, 64, 700
    pages = -(-n // page)
    shift = k_shift * torch.sign(torch.randn(d, generator=gen))
    parts = []
    for off in (shift, torch.zeros(d)):
        parts.append(quantise(torch.randn((S * pages, H, page, d), generator=gen) + off, bits))
    (kc, ka), (vc, va) = parts
    cache = q.QuantKVCache(*(t.to(DEV) for t in (pack(kc, bits), pack(vc, bits), ka, va)), bits)
    plan = q.KVPlan(H * group, H, d, page, max_seqs=S, max_rows=rows, max_pages=pages, rot_dim=0)
    x = (1.5 * torch.randn((S * rows, H * group, d), generator=gen) + q_shift * torch.sign(shift + 0.5)).to(torch.bfloat16)
    out = torch.empty_like(x, device=DEV)
    table = torch.arange(S * pages, dtype=torch.int32, device=DEV).view(S, pages)
    q.attention(plan, x.to(DEV), cache, table, torch.full((S,), n, dtype=torch.int32, device=DEV), out)
    k, v = (values(c, a).view(S, pages, H, page, d).transpose(2, 3).reshape(S, pages * page, H, d)[:, :n] for c, a in parts)
    xx = x.double().view(S, rows, H, group, d)
    a = torch.einsum("srhgd,sjhd->srhgj", xx, k) * d ** -0.5
    seen = torch.arange(n)[None] <= (n - rows + torch.arange(rows))[:, None]
    a = a.masked_fill(~seen[None, :, None, None], float("-inf"))
    want = torch.einsum("srhgj,sjhd->srhgd", torch.softmax(a, 4), v).reshape(S * rows, H * group, d)
    error = float((out.double().cpu() - want).norm() / want.norm())
    assert plan.error_flags() == 0
    assert error <= 2.0 ** -9, error

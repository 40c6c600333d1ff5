"""The terms that the adapters' first products enter the second ones in: three bfloat16 terms for float32 outputs, within 2^-26,
and two for bfloat16 ones, within 2^-17.

Sums of three products with 24 bits in all, 8 of them from each, and columns of B with a single 1: an output is one first
product. The tensor cores cut each of the two sums at 2^-23 of it at most (three products, and three terms, in one product of 16
or in two), the scale is a power of two, and the output is rounded once (2^-24): 2^-21 in all for float32."""
from __future__ import annotations

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


def _terms(v, n):
    """v as the sum of n bfloat16 terms, in float64."""
    import torch
    total, rest = torch.zeros_like(v, dtype=torch.float64), v.float()
    for _ in range(n):
        h = rest.to(torch.bfloat16).float()
        total += h.double()
        rest = rest - h
    return total


@pytest.mark.parametrize("rows,N,rank,adapters", [(1, 8, 8, 1), (5, 40, 24, 2), (33, 100, 32, 3), (64, 64, 64, 4), (70, 333, 72, 5),
                                                  (200, 1031, 128, 3)])
@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
def test_first_products_keep_their_bits(q, dtype, rows, N, rank, adapters):
    import torch
    gen = torch.Generator().manual_seed(rows + N)
    K, dt = 64, getattr(torch, dtype)
    # x: elements of 8 bits in [1, 1.9) with signs; A: of each column of rank, three elements 1, 2^-8 and 2^-16
    x = ((1.0 + 0.9 * torch.rand((rows, K), generator=gen)) * (1 - 2 * torch.randint(2, (rows, K), generator=gen))).to(torch.bfloat16)
    a = torch.zeros((adapters, rank, K))
    for i in range(adapters):
        for r in range(rank):
            at = torch.randperm(K, generator=gen)[:3]
            a[i, r, at] = torch.tensor([1.0, 2.0 ** -8, 2.0 ** -16])
    b = torch.zeros((adapters, N, rank))
    n = torch.arange(N)
    b[:, n, (n * 7) % rank] = 1.0
    scale = 2.0 ** torch.randint(-3, 4, (adapters,), generator=gen).float()
    ids = torch.randint(adapters, (rows,), generator=gen).int()
    plan = q.AdapterPlan(K, N, rank, adapters, rows, out_dtype=dt)
    y = torch.zeros((rows, N), dtype=dt, device=DEV)
    out = torch.empty_like(y)
    q.add_adapters(plan, x.to(DEV), a.to(torch.bfloat16).to(DEV), b.to(torch.bfloat16).to(DEV), scale.to(DEV), ids.to(DEV), y, out)
    low = torch.einsum("mk,mrk->mr", x.double(), a.double()[ids.long()]) * scale.double()[ids.long()][:, None]
    want = low[:, (n * 7) % rank]
    error = (out.double().cpu() - want).abs() / want.abs()
    bound = 2.0 ** -21 if dtype == "float32" else 2.0 ** -8 + 2.0 ** -17 + 2.0 ** -21
    assert float(error.max()) <= bound, float(error.max())
    if dtype == "float32":   # terms that are lost would be seen
        for terms in (1, 2):
            assert float(((_terms(want, terms) - want).abs() / want.abs()).max()) > 2 * bound
    assert plan.error_flags() == 0

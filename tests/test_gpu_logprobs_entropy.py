"""Entropies of rows that are nearly certain, whose likeliest token comes after a likely one where one thread reads them.

A row has the logit 0, one of r, and others of -25 or less, whose share in all is below e^-30. With e = e^-r the entropy is
log(1 + e) + r e / (1 + e). Sums are held to a logit of the row that the largest lies less than 6 above. For r above that the
largest is the reference, the sum 1 + e is rounded once (2^-24), and the rest are roundings of e's share: 2^-19 of the entropy.
Below, r e^r comes and goes, rounded to 2^-24 of r, twice, and the sum's rounding: (2 r + 2) 2^-24."""
from __future__ import annotations

import math

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


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
@pytest.mark.parametrize("M", [24, 320])
@pytest.mark.parametrize("falling", [False, True])
def test_entropy_of_nearly_certain_rows(q, dtype, M, falling):
    """A thread reads every 512th (256th of more than 304 rows) chunk of 16 bytes."""
    import torch
    gen = torch.Generator().manual_seed(M)
    rises = [0.5, 2.0, 3.75, 5.0, 5.9375, 6.0625, 6.5, 7.0, 8.0, 9.0, 10.0, 11.0, 11.9375, 12.5, 13.0, 13.75, 14.0, 14.25, 14.5, 15.0, 15.25,
             15.5, 15.9375, 20.0]
    step = (512 if M <= 304 else 256) * (4 if dtype == "float32" else 8)
    V = 8 * step
    l = torch.full((M, V), -25.0) - 30.0 * torch.rand((M, V), generator=gen)
    r = [rises[m % len(rises)] for m in range(M)]
    for m in range(M):
        first = (m * 37) % step
        at = (first, first + step * (1 + m % 6))
        l[m, at[falling]], l[m, at[not falling]] = 0.0, r[m]
    entropy = torch.full((M,), 77.0, device=DEV)
    q.logprobs(l.to(getattr(torch, dtype)).to(DEV), None, None, entropy)
    got = entropy.cpu().numpy().astype(np.float64)
    for m in range(M):
        e = math.exp(-r[m])
        want = math.log1p(e) + r[m] * e / (1 + e)
        bound = 2.0 ** -19 * want + (2.0 ** -23 if r[m] > 6 else (2 * r[m] + 2) * 2.0 ** -24)
        assert abs(got[m] - want) <= bound, (r[m], got[m], want)
        assert got[m] >= 0

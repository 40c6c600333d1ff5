"""Attention over a cache of codes: infinite queries, and keys that are not finite, in calls of few and of many rows. A row that does
not see them, or is not theirs, has the bits that it has without them."""
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


def _setup(q, bits, d, group, rows, n, window=0, change=None):
    import torch
    from tests._codes import Pool
    gen = torch.Generator().manual_seed(d + group + rows)
    pool = Pool([n], 1, 16, d, bits, gen)
    if change:
        change(pool)
    cache, table = pool.device(q)
    x = torch.randn((rows, group, d), generator=gen).to(torch.bfloat16)
    plan = q.KVPlan(group, 1, d, 16, max_seqs=1, max_rows=rows, max_pages=pool.max_pages, window=window)
    lens = torch.tensor([n], dtype=torch.int32, device=DEV)

    def run(x):
        out = torch.full_like(x, 7.0, device=DEV)
        q.attention(plan, x.to(DEV), cache, table, lens, out)
        torch.cuda.synchronize()
        assert plan.error_flags() == 0
        return out.cpu()

    return x, run


@pytest.mark.parametrize("bits", [8, 4])
@pytest.mark.parametrize("d,group,rows", [(128, 4, 1), (64, 3, 5), (256, 8, 2), (128, 20, 1), (64, 9, 7), (256, 33, 1), (128, 16, 4)])
@pytest.mark.parametrize("value", [float("inf"), float("nan")])
def test_a_query_that_is_not_finite_spoils_its_own_row_alone(q, bits, d, group, rows, value):
    import torch
    x, run = _setup(q, bits, d, group, rows, 150)
    clean = run(x)
    at = (rows - 1, group // 2)
    x[at[0], at[1], 7] = value
    out = run(x)
    assert torch.isnan(out[at]).all()
    others = torch.ones((rows, group), dtype=torch.bool)
    others[at] = False
    assert torch.equal(out[others], clean[others]) and torch.isfinite(clean).all()


@pytest.mark.parametrize("bits", [8, 4])
@pytest.mark.parametrize("d,group", [(64, 2), (128, 2), (256, 2), (128, 4), (64, 8), (256, 8)])
@pytest.mark.parametrize("what", ["scale_inf", "scale_nan", "bias_inf", "bias_nan"])
def test_keys_that_are_not_finite_reach_no_row_that_does_not_see_them(q, bits, d, group, what):
    import torch
    n, rows, window = 150, 6, 40
    side, value = what.split("_")

    def change(pool):
        for j in (147, n - rows - window + 2):   # seen by rows 3 to 5, and by rows 0 and 1
            page, slot = pool.place(0, j)
            pool.ka[page, 0, slot, 0, 0 if side == "scale" else 1] = float(value)

    x, run = _setup(q, bits, d, group, rows, n, window)
    clean = run(x)
    x, run = _setup(q, bits, d, group, rows, n, window, change)
    out = run(x)
    assert torch.equal(out[2], clean[2])
    if value == "nan":
        for r in (0, 1, 3, 4, 5):
            assert torch.isnan(out[r]).all()

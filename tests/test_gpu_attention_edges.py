"""Attention where values are not finite, where a window or the sinks end between drafted tokens, and where a length is past
the page table, against plain float64 computations.

Tolerances, from the arithmetic: outputs are rounded once to bfloat16 (at most 2^-8 of the value between neighbours); a
score's float32 sum of products is off by at most 2^-19 of the sum of their magnitudes, and the weights and their sums by
2^-15, which move an output by that share of the largest value in sight."""
from __future__ import annotations

import numpy as np
import pytest

pytestmark = pytest.mark.gpu

DEV = "cuda"
PAGE = 16


@pytest.fixture(scope="module")
def q():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from bit_affine_quantized_group_gb300 import _build
    _build.build()
    import bit_affine_quantized_group_gb300 as q
    return q


class Sequence:
    """One sequence's cache of shuffled pages, and its keys and values as float64 [positions, heads, d]."""

    def __init__(self, torch, positions, hkv, d, seed, key_size=1.0):
        gen = torch.Generator().manual_seed(seed)
        self.torch, self.pages = torch, -(-positions // PAGE)
        self.table = torch.randperm(self.pages, generator=gen).int()[None]
        self.k, self.v = (torch.full((self.pages, hkv, PAGE, d), float("nan"), dtype=torch.bfloat16) for _ in range(2))
        a, b = (torch.randn((positions, hkv, d), generator=gen) for _ in range(2))
        a, b = (a * key_size).to(torch.bfloat16), b.to(torch.bfloat16)
        j = torch.arange(positions)
        self.k[self.table[0, j // PAGE].long(), :, j % PAGE] = a
        self.v[self.table[0, j // PAGE].long(), :, j % PAGE] = b
        self.keys, self.values = a.double().numpy(), b.double().numpy()
        self.gen = gen

    def put(self, side, j, head, d, value):
        """A value at position j, of the tensors alone: the float64 copies keep what was there."""
        side[self.table[0, j // PAGE].long(), head, j % PAGE, d] = value

    def attend(self, q, qs, hkv, rows, length, window=0, sinks=0):
        torch = self.torch
        hq, d = qs.shape[1:]
        plan = q.KVPlan(hq, hkv, d, PAGE, max_seqs=1, max_rows=rows, max_pages=self.pages, window=window, sinks=sinks)
        out = torch.full(qs.shape, 77.0, dtype=torch.bfloat16, device=DEV)
        q.attention(plan, qs.to(DEV), q.KVCache(self.k.to(DEV), self.v.to(DEV)), self.table.to(DEV),
                    torch.tensor([length], dtype=torch.int32, device=DEV), out)
        torch.cuda.synchronize()
        return out.double().cpu().numpy(), plan.error_flags()

    def expected(self, qs, rows, length, window=0, sinks=0):
        """Outputs, tolerances, and which positions of the table each row sees."""
        hq, d = qs.shape[1:]
        group = hq // self.keys.shape[1]
        x = qs.double().numpy()
        out, tol = np.zeros(qs.shape), np.zeros(qs.shape)
        seen = np.zeros((rows, len(self.keys)), bool)
        j = np.arange(len(self.keys))
        for r in range(rows):
            pos = length - rows + r
            see = j <= pos
            if window:
                see &= (pos - j < window) | (j < sinks)
            seen[r] = see
            if not see.any():
                continue
            for h in range(hq):
                kk, vv = self.keys[see, h // group], self.values[see, h // group]
                a = kk @ x[r, h] * d ** -0.5
                e = np.exp(a - a.max())
                out[r, h] = (e / e.sum()) @ vv
                size = np.max(np.abs(kk) @ np.abs(x[r, h])) * d ** -0.5
                tol[r, h] = 2.0 ** -8 * np.abs(out[r, h]) + (2.0 ** -15 + 2.0 ** -19 * size) * np.max(np.abs(vv))
        return out, tol, seen

    def queries(self, rows, hq, d):
        return self.torch.randn((rows, hq, d), generator=self.gen).to(self.torch.bfloat16)


def _near(got, want, tol):
    return (np.abs(got - want) <= tol).all()


@pytest.mark.parametrize("key_size", [0.0, 1.0])   # equal weights of 1, and others
@pytest.mark.parametrize("d,hq,hkv,rows", [(64, 4, 2, 1), (128, 4, 2, 1), (256, 2, 1, 1), (128, 8, 2, 4), (64, 8, 1, 4), (128, 8, 1, 8),
                                           (256, 8, 1, 4), (256, 8, 1, 8)])
@pytest.mark.parametrize("length", [1, 200, 9000])
def test_a_visible_infinity_is_the_output(q, key_size, d, hq, hkv, rows, length):
    """A weight above 0 of an infinite value is infinite, whatever the weight; other columns and heads do not notice."""
    import torch
    s = Sequence(torch, length, hkv, d, seed=length + d, key_size=key_size)
    qs = s.queries(rows, hq, d)
    at = [(length // 3, 0, 3, float("inf")), (length // 2, hkv - 1, d - 1, -float("inf"))]
    for j, head, col, value in at:
        s.put(s.v, j, head, col, value)
    got, flags = s.attend(q, qs, hkv, rows, length)
    want, tol, seen = s.expected(qs, rows, length)
    assert flags == 0
    for j, head, col, value in at:
        heads = slice(head * (hq // hkv), (head + 1) * (hq // hkv))
        want[seen[:, j], heads, col] = value
        same = got[:, heads, col] == want[:, heads, col]
        assert same[seen[:, j]].all(), (got[:, heads, col], want[:, heads, col])
        got[:, heads, col][same] = want[:, heads, col][same] = 0.0
    assert _near(got, want, tol)


@pytest.mark.parametrize("d,hq,hkv,rows", [(64, 4, 2, 4), (128, 8, 1, 4), (128, 8, 1, 7), (256, 2, 1, 3)])
@pytest.mark.parametrize("window,sinks", [(40, 0), (40, 5), (40, 109), (64, 70), (0, 0)])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_strange_values_reach_the_rows_that_see_them(q, d, hq, hkv, rows, window, sinks, bad):
    """Around the ends of the rows' windows, of the sinks and of the sequence, one position after the other."""
    import torch
    length = 150
    first = length - rows
    edges = {first - 1, first, first + 1, length - 2, length - 1}
    if window:
        low = first - window + 1
        edges |= {low - 1, low, low + 1, low + rows - 2, low + rows - 1, sinks - 1, sinks, sinks + 1}
    for j in sorted(e for e in edges if 0 <= e < length):
        for keys in (False, True):
            if keys and bad == bad:
                continue   # an infinite key is a score of either sign
            s = Sequence(torch, length, hkv, d, seed=7 * j + d)
            qs = s.queries(rows, hq, d)
            s.put(s.k if keys else s.v, j, 0, slice(None), bad)
            got, flags = s.attend(q, qs, hkv, rows, length, window, sinks)
            want, tol, seen = s.expected(qs, rows, length, window, sinks)
            assert flags == 0
            see, own = seen[:, j], slice(0, hq // hkv)
            rest = np.ones(got.shape[:2], bool)
            rest[see, own] = False
            assert _near(got[rest], want[rest], tol[rest]), (j, keys)
            mine = got[see, own]
            assert (np.isnan(mine) if bad != bad else mine == bad).all(), (j, keys, mine)


@pytest.mark.parametrize("rows,hq", [(2, 1), (3, 8)])
def test_a_window_of_many_millions(q, rows, hq):
    """Offsets of positions from a window's ends that pass 32 bits when they are multiplied by a row's size. All pages of the
    table are the same one, so that a score's share of the softmax is the number of times that the window shows its slot."""
    import torch
    d, page, pages, window = 256, 1024, 65600, (1 << 26) + 1000
    gen = torch.Generator().manual_seed(23)
    k, v = (torch.randn((1, 1, page, d), generator=gen).to(torch.bfloat16) for _ in range(2))
    qs = torch.randn((rows, hq, d), generator=gen).to(torch.bfloat16)
    length = pages * page - 5
    plan = q.KVPlan(hq, 1, d, page, max_seqs=1, max_rows=rows, max_pages=pages, window=window)
    out = torch.full(qs.shape, 77.0, dtype=torch.bfloat16, device=DEV)
    q.attention(plan, qs.to(DEV), q.KVCache(k.to(DEV), v.to(DEV)), torch.zeros((1, pages), dtype=torch.int32, device=DEV),
                torch.tensor([length], dtype=torch.int32, device=DEV), out)
    got = out.double().cpu().numpy()
    assert plan.error_flags() == 0
    keys, values = k[0, 0].double().numpy(), v[0, 0].double().numpy()
    slot = np.arange(page)
    upto = lambda n: n // page + (slot < n % page)   # times that each slot lies before position n   # noqa: E731
    for r in range(rows):
        pos = length - rows + r
        times = upto(pos + 1) - upto(pos + 1 - window)
        for h in range(hq):
            x = qs[r, h].double().numpy()
            a = keys @ x * d ** -0.5
            e = np.exp(a - a.max()) * times
            want = (e / e.sum()) @ values
            size = np.max(np.abs(keys) @ np.abs(x)) * d ** -0.5
            # float32 sums over the 7,000 steps of a share, two additions each
            tol = 2.0 ** -8 * np.abs(want) + (2.0 ** -15 + 2.0 ** -19 * size + 2.0 ** -24 * 2 ** 14) * np.max(np.abs(values))
            assert _near(got[r, h], want, tol)


@pytest.mark.parametrize("rows,hq,hkv,d", [(1, 2, 1, 64), (8, 4, 2, 128), (8, 8, 1, 128), (5, 2, 1, 256)])
@pytest.mark.parametrize("window,sinks", [(0, 0), (20, 0), (20, 3), (70, 100), (2 ** 31 - 2, 0)])
@pytest.mark.parametrize("over", [0, 1, 3, 7, 25, 200, 2 ** 31 - 1 - 128])
def test_lengths_past_the_page_table(q, rows, hq, hkv, d, window, sinks, over):
    """Rows stand where the length says, and see what the table holds."""
    import torch
    s = Sequence(torch, 128, hkv, d, seed=rows + d)
    qs = s.queries(rows, hq, d)
    got, flags = s.attend(q, qs, hkv, rows, 128 + over, window, sinks)
    want, tol, _ = s.expected(qs, rows, 128 + over, window, sinks)
    assert flags == (q.KV_BAD_LENGTH if over else 0)
    assert _near(got, want, tol)


@pytest.mark.parametrize("rows", [1, 3])
def test_negative_lengths_are_padding(q, rows):
    """However far below 0, in the append and in attention; the sequence between them is whole."""
    import torch
    lengths, hq, hkv, d = [-2 ** 31, 20, -1, -2 ** 31 + 2], 4, 2, 64
    gen = torch.Generator().manual_seed(24)
    k, v = (torch.full((8, hkv, PAGE, d), 3.0, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    cache = q.KVCache(k, v)
    table = torch.arange(8, dtype=torch.int32, device=DEV).view(4, 2)
    lens = torch.tensor(lengths, dtype=torch.int32, device=DEV)
    x = torch.randn((4 * rows, (hq + 2 * hkv) * d), generator=gen).to(torch.bfloat16).to(DEV)
    rope = torch.zeros((32, d), device=DEV)
    rope[:, :d // 2] = 1.0   # turns nothing
    plan = q.KVPlan(hq, hkv, d, PAGE, max_seqs=4, max_rows=rows, max_pages=2)
    queries, out = (torch.full((4 * rows, hq, d), 9.0, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    q.qk_norm_rope(plan, x[:, :hq * d], x[:, hq * d:(hq + hkv) * d], x[:, (hq + hkv) * d:], None, None, rope, lens, table, cache, queries)
    q.attention(plan, queries, cache, table, lens, out)
    assert plan.error_flags() == 0
    whole = torch.arange(4 * rows, device=DEV) // rows == 1
    assert (queries[~whole] == 0).all() and (out[~whole] == 0).all()
    assert torch.equal(queries[whole].view(rows, -1), x[whole, :hq * d])
    written = (k != 3.0).any(3).any(1).cpu()   # [page, slot]
    at = torch.zeros_like(written)
    for pos in range(20 - rows, 20):
        at[2 + pos // PAGE, pos % PAGE] = True
    assert torch.equal(written, at) and torch.isfinite(out.float()).all()

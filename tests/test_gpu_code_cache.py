"""The cache of 8- and 4-bit codes: its append, its read-back and attention over it, against float64 and against the
definition's float32 operations.

Tolerances, from the arithmetic. Appended values that pass no arithmetic are quantised bit for bit as defined. Normed and
rotated keys are off by at most 2^-19 of the head's largest value before they are quantised, and a stored element by half a
step, 2^-11 of the bias and the scale's own rounding (2^-17 at most). Attention: a score's sum of 64 products of a query and
1024 + code is off by at most 64 * 2^-24 = 2^-18 of the sum of their magnitudes; values and weights are rounded to binary16
(2^-11 of the value, of the group's middle, of the weight, and the sum of the weights 2^-12), which moves an output by that
share of the largest value in sight; the output is rounded once to bfloat16 (2^-8)."""
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


def _int32(x):
    import torch
    return torch.tensor(x, dtype=torch.int32, device=DEV)


# ---- read-back ----

def _read(q, pool, starts, rows, dtype, lengths=None, plan=None, layout=None):
    import torch
    cache, table = pool.device(q)
    S, H, D = len(pool.lengths), pool.heads, pool.d
    plan = plan or q.KVPlan(H, H, D, pool.page, max_seqs=S, max_rows=1, max_pages=pool.max_pages)
    if layout == "strided":   # rows apart, sequences inside
        k, v = (torch.full((rows, S, H + 1, D), 7.0, dtype=dtype, device=DEV)[:, :, :H].transpose(0, 1) for _ in range(2))
    else:
        k, v = (torch.full((S, rows, H, D), 7.0, dtype=dtype, device=DEV) for _ in range(2))
    q.kv_read(plan, cache, table, _int32(lengths or pool.lengths), k, v, None if starts is None else _int32(starts))
    torch.cuda.synchronize()
    return plan, k.cpu(), v.cpu()


def _expect_read(pool, side, starts, rows, dtype):
    import torch
    from tests._codes import values
    want = torch.full((len(pool.lengths), rows, pool.heads, pool.d), 7.0, dtype=dtype)
    for s, n in enumerate(pool.lengths):
        x = values(*pool.parts[s][side]).float().to(dtype)
        for j in range(rows):
            pos = (starts[s] if starts else 0) + j
            if 0 <= pos < n:
                want[s, j] = x[pos]
    return want


@pytest.mark.parametrize("bits", [8, 4])
@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
@pytest.mark.parametrize("heads,d,page", [(1, 64, 16), (3, 128, 1), (8, 128, 64), (2, 256, 8), (5, 64, 1024)])
def test_read(q, bits, dtype, heads, d, page):
    """Exact, and rows before position 0 and behind the length are left as they were."""
    import torch
    from tests._codes import Pool
    dt = getattr(torch, dtype)
    pool = Pool([1, 0, 77, 150], heads, page, d, bits, torch.Generator().manual_seed(bits + d))
    for starts, rows in ((None, 160), ([0, 0, 70, -3], 9), ([-2 ** 31, 5, 2 ** 31 - 2, 149], 33)):
        plan, k, v = _read(q, pool, starts, rows, dt, layout="strided" if rows == 9 else None)
        assert torch.equal(k, _expect_read(pool, 0, starts, rows, dt))
        assert torch.equal(v, _expect_read(pool, 1, starts, rows, dt))
        assert plan.error_flags() == 0


def test_read_of_bad_pages_and_lengths(q):
    import torch
    from tests._codes import Pool
    pool = Pool([40, 20], 2, 16, 64, 8, torch.Generator().manual_seed(1), extra=0)
    want = _expect_read(pool, 0, None, 60, torch.float32)
    pool.table[0, 1] = pool.pages   # out of range
    want[0, 16:32] = 0.0
    plan, k, _ = _read(q, pool, None, 60, torch.float32, lengths=[40, 1000])
    # a length past the table: positions 20 to 31 are slots that nothing was written to, and page 2 is out of range already
    assert torch.isnan(k[1, 20:32]).all()
    want[1, 32:48] = 0.0
    k[1, 20:32] = want[1, 20:32]
    assert torch.equal(k, want)
    assert plan.error_flags() == q.KV_BAD_PAGE | q.KV_BAD_LENGTH
    assert plan.error_flags() == 0


def test_read_far_into_a_large_pool(q):
    """Codes that lie past 2^32 bytes."""
    import torch
    H, D, page = 8, 256, 1024
    pages = 2200   # 2 MB each
    k = torch.zeros((pages, H, page, D), dtype=torch.uint8, device=DEV)
    a = torch.zeros((pages, H, page, 4, 2), dtype=torch.float16, device=DEV)
    k[-1] = torch.arange(D, device=DEV).to(torch.uint8)
    a[-1, ..., 0] = 0.5
    a[-1, ..., 1] = -3.0
    plan = q.KVPlan(H, H, D, page, max_seqs=1, max_rows=1, max_pages=1)
    out = torch.zeros((1, 5, H, D), device=DEV)
    cache = q.QuantKVCache(k, k, a, a, 8)
    q.kv_read(plan, cache, _int32([[pages - 1]]), _int32([1000]), out, out.clone(), _int32([500]))
    want = (0.5 * torch.arange(D, device=DEV) - 3.0).expand(1, 5, H, D)
    assert torch.equal(out, want)
    queries = torch.ones((1, H, D), dtype=torch.bfloat16, device=DEV)
    att = torch.empty_like(queries)
    q.attention(plan, queries, cache, _int32([[pages - 1]]), _int32([1000]), att)
    assert torch.equal(att, want[:, 0].to(torch.bfloat16))   # all positions are alike, and the values binary16 numbers
    assert plan.error_flags() == 0


# ---- append ----

def _rope(positions, rot):
    import torch
    i = torch.arange(rot // 2, dtype=torch.float64)
    a = torch.arange(positions, dtype=torch.float64)[:, None] * 10000.0 ** (-2.0 * i / max(rot, 1))
    return torch.cat((a.cos(), a.sin()), 1).float()


def _append(q, lengths, rows, hq, hkv, d, page, bits, rot, interleaved, dtype, norm=True, layout="hnd", seed=0, change=None):
    import torch
    from tests._codes import Pool
    gen = torch.Generator().manual_seed(seed)
    pool = Pool(lengths, hkv, page, d, bits, gen, layout)
    T = len(lengths) * rows
    x = torch.randn((T, (hq + 2 * hkv) * d), generator=gen).to(dtype)
    if change:
        change(x)
    weights = [1 + 0.1 * torch.randn(d, generator=gen) for _ in range(2)] if norm else [None, None]
    rope = _rope(max(max(lengths), 1), rot) if rot else None
    plan = q.KVPlan(hq, hkv, d, page, max_seqs=len(lengths), max_rows=1, max_pages=pool.max_pages, rot_dim=rot,
                    interleaved=interleaved)
    cache, table = pool.device(q)
    out = torch.full((T, hq * d), 7.0, dtype=torch.bfloat16, device=DEV)
    dx = x.to(DEV)
    cut = [dx[:, :hq * d], dx[:, hq * d:(hq + hkv) * d], dx[:, (hq + hkv) * d:]]
    q.qk_norm_rope(plan, *cut, *(w if w is None else w.to(DEV) for w in weights), None if rope is None else rope.to(DEV),
                   _int32(lengths), table, cache, out)
    torch.cuda.synchronize()

    def turned(t, heads, weight):
        t = t.double().view(T, heads, d)
        if weight is not None:
            t = t * torch.rsqrt((t * t).mean(2, keepdim=True) + 1e-6) * weight.double()
        if rot:
            pos = torch.cat([torch.arange(n - rows, n) for n in lengths]).clamp(min=0)
            c, s = (rope[pos][:, None, i * rot // 2:(i + 1) * rot // 2].double() for i in (0, 1))
            a, b = (t[..., 0:rot:2], t[..., 1:rot:2]) if interleaved else (t[..., :rot // 2], t[..., rot // 2:rot])
            a, b = a * c - b * s, b * c + a * s
            t = torch.cat(((torch.stack((a, b), 3).flatten(2) if interleaved else torch.cat((a, b), 2)), t[..., rot:]), 2)
        return t

    keys = turned(x[:, hq * d:(hq + hkv) * d], hkv, weights[1])
    vals = x[:, (hq + hkv) * d:].float().view(T, hkv, d)
    queries = turned(x[:, :hq * d], hq, weights[0])
    return plan, pool, out.view(T, hq, d).cpu(), queries, keys, vals


def _check_append(pool, rows, keys, vals, exact_keys):
    """Every slot of the pool: new tokens' codes, and all others as they were."""
    import torch
    from tests._codes import pack, quantise, unpack, values
    k, v = ([c, a] for c, a in pool.back())
    want = [(unpack(pool.k, pool.bits).clone(), pool.ka.clone()), (unpack(pool.v, pool.bits).clone(), pool.va.clone())]
    at = []
    for s, n in enumerate(pool.lengths):
        for r in range(rows):
            if n - rows + r >= 0:
                at.append((s * rows + r, *pool.place(s, n - rows + r)))
    if at:
        t, page, slot = (torch.tensor([int(a[i]) for a in at]) for i in range(3))
        want[1][0][page, :, slot], want[1][1][page, :, slot] = quantise(vals[t], pool.bits)
        if exact_keys:
            want[0][0][page, :, slot], want[0][1][page, :, slot] = quantise(keys[t].float(), pool.bits)
        else:
            code, affine = k[0][page, :, slot], k[1][page, :, slot]
            x = keys[t]
            g = x.unflatten(-1, (-1, 64))
            lo, hi = g.amin(-1), g.amax(-1)
            off = 2.0 ** -19 * x.abs().amax(-1, keepdim=True)
            scale, bias = affine[..., 0].double(), affine[..., 1].double()
            top = 2 ** pool.bits - 1
            assert ((bias - lo).abs() <= off + 2.0 ** -11 * lo.abs() + 2.0 ** -25).all()
            assert ((scale - (hi - lo) / top).abs() <= (2 * off) / top + 2.0 ** -11 * (hi - lo) / top + 2.0 ** -25).all()
            step = scale[..., None].expand(g.shape).flatten(-2)
            low = lo.abs()[..., None].expand(g.shape).flatten(-2)
            err = (values(code, affine) - x).abs()
            # (the code's own float32 arithmetic: 2^-20 of 255 steps)
            assert (err <= (0.5 + 2.0 ** -12) * step + 2 * off + 2.0 ** -11 * low + 2.0 ** -17).all()
            want[0][0][page, :, slot], want[0][1][page, :, slot] = code, affine
    for got, expect in zip((k, v), want):
        assert torch.equal(got[0], expect[0])
        assert torch.equal(got[1].view(torch.int16), expect[1].view(torch.int16))


@pytest.mark.parametrize("bits", [8, 4])
@pytest.mark.parametrize("hq,hkv,d,rot,interleaved,rows,page", [
    (4, 2, 64, 64, False, 1, 16), (3, 1, 64, 32, True, 5, 4), (8, 8, 128, 128, False, 3, 16), (2, 2, 128, 128, True, 1, 64),
    (5, 1, 128, 48, False, 2, 16), (6, 2, 256, 256, False, 4, 16), (2, 1, 256, 64, False, 40, 16), (4, 4, 256, 80, True, 2, 1),
    (1, 1, 64, 16, False, 70, 32), (7, 7, 64, 0, False, 2, 16), (32, 8, 128, 128, False, 1, 16)])
@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
def test_append(q, bits, hq, hkv, d, rot, interleaved, rows, page, dtype):
    """Lengths below `rows` leave padding, whose queries are zeros."""
    import torch
    lengths = [rows, 3 * rows + 70, 0, max(0, rows - 1), 1]
    plan, pool, out, queries, keys, vals = _append(q, lengths, rows, hq, hkv, d, page, bits, rot, interleaved,
                                                   getattr(torch, dtype), seed=d + rot + rows,
                                                   layout="nhd" if rows == 2 else "hnd")
    _check_append(pool, rows, keys, vals, exact_keys=False)
    pad = torch.tensor([n - rows + r < 0 for n in lengths for r in range(rows)])
    assert (out[pad] == 0).all()
    want = queries[~pad]
    assert ((out[~pad].double() - want).abs() <= 2.0 ** -8 * want.abs() + 2.0 ** -19 * want.abs().amax(-1, keepdim=True)).all()
    assert plan.error_flags() == 0


@pytest.mark.parametrize("bits", [8, 4])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_append_without_arithmetic_is_as_defined(q, bits, d):
    """No norm, no rotation: keys too. Groups that are constant, zero, tiny, huge, one-sided and far from zero."""
    import torch

    def change(x):
        g = x.view(x.shape[0], -1, 64)
        g[0] = 0.0
        g[1] = 3.25
        g[2] = -1e-30
        g[3] *= 1e-9
        g[4] *= 3e-4
        g[5] = 1000.0 + g[5]
        g[6] *= 1e6
        g[7, :, :5] = 65280.0
        g[8] = g[8].abs()
        g[9] = torch.arange(64.0) - 20.0   # halves of steps in places
        g[10] = (torch.arange(64) % 16).float() * 0.5

    plan, pool, out, queries, keys, vals = _append(q, [13], 13, 2, 2, d, 16, bits, 0, False, torch.float32, norm=False, seed=d,
                                                   change=change)
    _check_append(pool, 13, keys, vals, exact_keys=True)
    assert plan.error_flags() == 0


@pytest.mark.parametrize("value,bit", [(float("nan"), True), (float("inf"), True), (-float("inf"), True), (3e38, False)])
def test_append_of_values_that_codes_cannot_hold(q, value, bit):
    import torch

    def change(x):
        x[1, 4 * 128 + 3] = value          # a key
        x[2, (4 + 2) * 128 + 127] = value  # a value

    plan, pool, out, queries, keys, vals = _append(q, [3], 3, 4, 2, 128, 16, 8, 0, False, torch.float32, norm=False,
                                                   change=change)
    _check_append(pool, 3, keys, vals, exact_keys=True)
    assert plan.error_flags() == (q.KV_NOT_FINITE if bit else 0)
    for _, affine in pool.back():
        page, slot = pool.place(0, torch.arange(3))
        assert torch.isfinite(affine[page, :, slot]).all()


def test_append_to_bad_places(q):
    """A page out of range, and a length past the table: nothing is written, and the queries come out all the same."""
    import torch
    from tests._codes import Pool
    pool = Pool([20, 30], 1, 16, 64, 8, torch.Generator().manual_seed(0), extra=0)
    pool.table[0, 1] = -1
    cache, table = pool.device(q)
    before = pool.back()
    plan = q.KVPlan(1, 1, 64, 16, max_seqs=2, max_rows=1, max_pages=pool.max_pages, rot_dim=0)
    x = torch.randn((2, 64), device=DEV).to(torch.bfloat16)
    out = torch.empty_like(x)
    q.qk_norm_rope(plan, x, x, x, None, None, None, _int32([20, 33]), table, cache, out)
    assert plan.error_flags() == q.KV_BAD_PAGE | q.KV_BAD_LENGTH
    assert torch.equal(out, x)
    for (c0, a0), (c1, a1) in zip(before, pool.back()):
        assert torch.equal(c0, c1) and torch.equal(a0.view(torch.int16), a1.view(torch.int16))


# ---- attention ----

def _reference(qs, pool, lengths, rows, window, sinks, scale):
    from tests._codes import values
    hq, d = qs.shape[1:]
    group = hq // pool.heads
    out, tol = np.zeros(qs.shape), np.zeros(qs.shape[:2] + (1,))
    for s, n in enumerate(lengths):
        if n <= 0:
            continue
        k, v = (values(c, a).numpy() for c, a in pool.parts[s])
        step = np.repeat(np.abs(pool.parts[s][0][1][..., 0].double().numpy()), 64, 2)   # of every key element
        for r in range(rows):
            pos = n - rows + r
            j = np.arange(len(k))
            see = j <= pos
            if window:
                see &= (pos - j < window) | (j < sinks)
            j = j[see]
            if pos < 0 or not len(j):
                continue
            for h in range(hq):
                x, kk, vv = qs[s * rows + r, h], k[j, h // group], v[j, h // group]
                a = kk @ x * scale
                e = np.exp(a - a.max())
                out[s * rows + r, h] = (e / e.sum()) @ vv
                size = np.max(step[j, h // group] @ np.abs(x)) * 1279 * abs(scale)
                tol[s * rows + r, h] = (4 * 2.0 ** -11 + 2.0 ** -17 * size) * np.max(np.abs(vv))
    return out, tol + 2.0 ** -8 * np.abs(out)


def _attend(q, lengths, hq, hkv, d, bits, rows=1, page=16, window=0, sinks=0, seed=0, layout="hnd", scale=None, q_size=1.5,
            max_rows=None, change=None, told=None, size=1.0, extra=1):
    import torch
    from tests._codes import Pool
    gen = torch.Generator().manual_seed(seed)
    pool = Pool(lengths, hkv, page, d, bits, gen, layout, size=size, extra=extra)
    if change:
        change(pool)
    cache, table = pool.device(q)
    qt = (q_size * torch.randn((len(lengths) * rows, hq, d), generator=gen)).to(torch.bfloat16)
    plan = q.KVPlan(hq, hkv, d, page, max_seqs=len(lengths), max_rows=max_rows or rows, max_pages=pool.max_pages,
                    window=window, sinks=sinks, scale=scale)
    out = torch.full((len(lengths) * rows, hq, d), 77.0, dtype=torch.bfloat16, device=DEV)
    call = lambda: q.attention(plan, qt.to(DEV), cache, table, _int32(told or lengths), out)  # noqa: E731
    call()
    torch.cuda.synchronize()
    flags = plan.error_flags()
    got = out.double().cpu().numpy()
    want, tol = _reference(qt.double().numpy(), pool, lengths, rows, window, sinks, d ** -0.5 if scale is None else scale)
    return got, want, tol, flags, (pool, qt, call, out)


def _fits(got, want, tol, flags):
    assert flags == 0
    assert np.isfinite(got).all()
    assert (np.abs(got - want) <= tol).all(), np.max(np.abs(got - want) / np.maximum(tol, 1e-30))
    # over all outputs: roundings to bfloat16 (2^-8 at most), of values and weights in sums that keep their shares (2^-9)
    assert np.linalg.norm(got - want) <= 1.5 * 2.0 ** -8 * np.linalg.norm(want)


@pytest.mark.parametrize("bits", [8, 4])
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("lengths", [[1], [0], [2, 0, 1], [15, 16, 17], [63, 64, 65, 129], [1000], [300, 1, 0, 77, 513]])
def test_lengths(q, bits, d, lengths):
    _fits(*_attend(q, lengths, 8, 2, d, bits, seed=len(lengths) * d)[:4])


@pytest.mark.parametrize("bits", [8, 4])
@pytest.mark.parametrize("page", [1, 2, 4, 8, 16, 32, 128, 1024])
def test_page_sizes(q, bits, page):
    _fits(*_attend(q, [1, 37, 250], 4, 2, 128, bits, page=page, seed=page)[:4])


@pytest.mark.parametrize("bits", [8, 4])
@pytest.mark.parametrize("hq,hkv,rows,d", [(1, 1, 1, 64), (5, 1, 3, 128), (14, 2, 1, 128), (16, 1, 1, 256), (17, 1, 1, 64),
                                           (8, 1, 4, 128), (12, 3, 16, 64), (64, 1, 2, 128), (33, 1, 1, 256), (8, 2, 16, 256),
                                           (32, 2, 5, 128), (7, 7, 2, 64), (40, 8, 8, 128)])
@pytest.mark.parametrize("lengths", [[40, 333], [16, 2, 900]])
def test_heads_and_rows(q, bits, hq, hkv, rows, d, lengths):
    _fits(*_attend(q, lengths, hq, hkv, d, bits, rows=rows, seed=hq + rows)[:4])


@pytest.mark.parametrize("bits", [8, 4])
@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 4), (17, 1), (100, 33), (500, 16), (10000, 4), (128, 10000),
                                          (2 ** 31 - 1, 2 ** 31 - 1)])
@pytest.mark.parametrize("rows,d", [(1, 128), (5, 64), (16, 128), (3, 256)])
def test_window_and_sinks(q, bits, window, sinks, rows, d):
    _fits(*_attend(q, [700, 5, 101, 0, 116], 4, 2, d, bits, rows=rows, window=window, sinks=sinks, seed=window % 1000 + sinks)[:4])


@pytest.mark.parametrize("bits,d,hq,rows,n", [(8, 128, 8, 1, 30000), (4, 128, 8, 1, 30000), (8, 64, 4, 16, 9000),
                                               (4, 256, 4, 9, 9000), (8, 256, 2, 1, 20000), (4, 128, 16, 4, 12000)])
def test_long_sequences_are_cut_and_joined(q, bits, d, hq, rows, n):
    got, want, tol, flags, (pool, qt, call, out) = _attend(q, [n, 200], hq, 1, d, bits, rows=rows, seed=n)
    _fits(got, want, tol, flags)
    import torch
    first = out.clone()
    for _ in range(3):
        out.fill_(5.0)
        call()
        assert torch.equal(out, first)


@pytest.mark.parametrize("bits", [8, 4])
def test_many_sequences(q, bits):
    rng = np.random.default_rng(3)
    lengths = [int(n) for n in rng.integers(0, 200, 75)] + [2000]
    _fits(*_attend(q, lengths, 4, 2, 64, bits, seed=8)[:4])
    _fits(*_attend(q, lengths[:33], 6, 1, 128, bits, rows=2, window=64, sinks=2, seed=9)[:4])


@pytest.mark.parametrize("bits", [8, 4])
@pytest.mark.parametrize("scale,q_size", [(-0.1, 1.0), (0.0, 1.0), (0.5, 1e-3), (1e-6, 1e6), (1e-33, 1e33), (1e30, 1e-31), (0.09, 0.0)])
def test_scales_and_sizes_of_queries(q, bits, scale, q_size):
    _fits(*_attend(q, [130, 30], 4, 1, 128, bits, rows=2, scale=scale, q_size=q_size, seed=4)[:4])


@pytest.mark.parametrize("bits", [8, 4])
@pytest.mark.parametrize("d,rows", [(64, 1), (128, 3), (256, 2), (128, 9)])
@pytest.mark.parametrize("q_size", [1e7, 3e7, 1e8, 1e10])
def test_scores_whose_steps_are_larger_than_one(q, bits, d, rows, q_size):
    """Scores of 1e7 to 1e11, whose roundings are larger than the exponents of weights. No output leaves the values' range, and a
    row takes the value of its best key where that leads the others by more than the scores' error."""
    from tests._codes import values
    got, want, tol, flags, (pool, qt, *_) = _attend(q, [200, 70], 4, 1, d, bits, rows=rows, q_size=q_size, seed=d + rows)
    assert flags == 0 and np.isfinite(got).all()
    x, led = qt.double().numpy(), 0
    for s, n in enumerate((200, 70)):
        k, v = (values(c, a).numpy()[:, 0] for c, a in pool.parts[s])
        step = float(pool.parts[s][0][1][..., 0].max())
        most = np.abs(v).max()
        assert (np.abs(got[s * rows:(s + 1) * rows]) <= most * (1 + 2.0 ** -7)).all()
        for r in range(s * rows, (s + 1) * rows):
            for h in range(4):
                scores = np.sort((k[:n - rows + 1 + r - s * rows] @ x[r, h]) * d ** -0.5)
                error = 2.0 ** -17 * 1279 * step * np.abs(x[r, h]).sum() * d ** -0.5   # of a score
                if scores[-1] - scores[-2] > 2 * error + 40:   # e^-40 of 200 keys is nothing
                    led += 1
                    assert (np.abs(got[r, h] - want[r, h]) <= 2.0 ** -8 * np.abs(want[r, h]) + 2.0 ** -10 * most).all()
    assert led >= 1


@pytest.mark.parametrize("bits", [8, 4])
@pytest.mark.parametrize("d,rows", [(64, 1), (128, 1), (128, 3), (256, 2), (128, 9)])
@pytest.mark.parametrize("size", [1e-6, 1e-3, 300.0, 15000.0])
def test_sizes_of_keys_and_values(q, bits, d, rows, size):
    """Scales that are no normal binary16 numbers, and scales whose multiples leave binary16. The scores stay small: their
    tolerance grows with what is summed."""
    got, want, tol, flags, (pool, *_) = _attend(q, [150, 70], 4, 1, d, bits, rows=rows, q_size=1.0 / size, size=size, seed=d + rows)
    if size < 1e-3:   # values are multiples of 2^-24, and so held in binary16, but the weights' products round as ever
        tol = tol + 2.0 ** -24
        assert flags == 0 and (np.abs(got - want) <= tol).all()
    else:
        _fits(got, want, tol, flags)


@pytest.mark.parametrize("bits", [8, 4])
@pytest.mark.parametrize("d,rows", [(64, 2), (128, 1), (128, 9), (256, 3)])
@pytest.mark.parametrize("size", [12.0, 20.0, 28.0, 60.0, 80.0, 100.0])
def test_sizes_of_values_about_the_largest_scales_of_weights(q, bits, d, rows, size):
    """Scales on both sides of 2 and 8, some of each in a step."""
    _fits(*_attend(q, [150, 70], 4, 1, d, bits, rows=rows, q_size=1.0 / size, size=size, seed=d + rows + 1)[:4])


@pytest.mark.parametrize("bits", [8, 4])
@pytest.mark.parametrize("scale", [0x3FFF, 0x4000, 0x47FF, 0x4800, 0xBFFF, 0xC000, 0xC7FF, 0xC800, 0x0001, 0x8001])
@pytest.mark.parametrize("n,d,rows", [(1, 128, 1), (2, 64, 2), (40, 256, 1), (9, 128, 4)])
def test_scales_at_the_edges_of_binary16(q, bits, scale, n, d, rows):
    """The largest scales that weights are multiplied by, the next ones, negative ones and the smallest: the last position's."""
    import torch
    of = torch.tensor([scale], dtype=torch.int32).to(torch.int16).view(torch.float16)

    def change(pool):
        page, slot = pool.place(0, n - 1)
        pool.va[page, :, slot, :, 0] = of
        pool.parts[0][1][1][n - 1, :, :, 0] = of

    got, want, tol, flags, _ = _attend(q, [n], 4, 1, d, bits, rows=rows, seed=n + d, change=change)
    assert flags == 0 and np.isfinite(got).all()
    assert (np.abs(got - want) <= tol + 2.0 ** -10 * abs(float(of)) * 2 ** bits).all()


@pytest.mark.parametrize("bits", [8, 4])
@pytest.mark.parametrize("rows,window,told", [(1, 0, 100), (3, 0, 98), (3, 20, 100), (2, 0, 5000)])
def test_lengths_past_the_page_table(q, bits, rows, window, told):
    """Rows stand where the length says; what is past the table is not seen."""
    from tests._codes import values
    n, d, hq = 96, 128, 4
    got, _, _, flags, (pool, qt, *_) = _attend(q, [n], hq, 1, d, bits, rows=rows, window=window, told=[told], extra=0)
    assert flags == q.KV_BAD_LENGTH
    k, v = (values(c, a).numpy()[:, 0] for c, a in pool.parts[0])
    x = qt.double().numpy()
    for r in range(rows):
        pos = told - rows + r
        j = np.arange(n)
        j = j[(j <= pos) & ((pos - j < window) if window else True)]
        for h in range(hq):
            if not len(j):
                assert (got[r, h] == 0).all()
                continue
            a = k[j] @ x[r, h] * d ** -0.5
            e = np.exp(a - a.max())
            want = e / e.sum() @ v[j]
            size = np.abs(x[r, h]).sum() * 1279 * d ** -0.5 * float(pool.parts[0][0][1][..., 0].max())
            assert (np.abs(got[r, h] - want) <= 2.0 ** -8 * np.abs(want) + (2.0 ** -9 + 2.0 ** -17 * size) * np.abs(v).max()).all()


@pytest.mark.parametrize("bits", [8, 4])
def test_two_threads_share_a_plan(q, bits):
    """Host threads that launch attention of many rows, whose joins are launches of their own, on one stream."""
    import threading

    import torch
    runs = [_attend(q, [9000], 8, 1, 128, bits, rows=4, seed=s)[4] for s in (1, 2)]
    want = [out.clone() for *_, out in runs]
    plan = q.KVPlan(8, 1, 128, 16, max_seqs=1, max_rows=4, max_pages=runs[0][0].max_pages)
    stream = torch.cuda.Stream()
    outs = [[torch.empty_like(want[i]) for _ in range(20)] for i in range(2)]
    args = [(qt.to(DEV), pool.cache, pool.table.cuda(), _int32([9000])) for pool, qt, *_ in runs]
    torch.cuda.synchronize()

    def work(i):
        x, cache, table, lens = args[i]
        for out in outs[i]:
            q.attention(plan, x, cache, table, lens, out, stream=stream)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(out, want[i]) for out in outs[i])


@pytest.mark.parametrize("bits", [8, 4])
def test_queries_of_very_different_elements(q, bits):
    """A row's largest element is 2^20 times another row's, and within a row."""
    import torch
    from tests._codes import Pool
    gen = torch.Generator().manual_seed(2)
    pool = Pool([200], 1, 16, 128, bits, gen)
    cache, table = pool.device(q)
    qt = torch.randn((1, 4, 128), generator=gen) * torch.tensor([1e-6, 1.0, 1e-3, 0.5])[None, :, None]
    qt[0, 1, ::3] *= 1e-6
    qt = qt.to(torch.bfloat16)
    plan = q.KVPlan(4, 1, 128, 16, max_seqs=1, max_rows=1, max_pages=pool.max_pages, scale=0.3)
    out = torch.empty((1, 4, 128), dtype=torch.bfloat16, device=DEV)
    q.attention(plan, qt.to(DEV), cache, table, _int32([200]), out)
    want, tol = _reference(qt.double().numpy(), pool, [200], 1, 0, 0, 0.3)
    _fits(out.double().cpu().numpy(), want, tol, plan.error_flags())


def test_an_infinite_query_spoils_its_own_row_alone(q):
    import torch
    from tests._codes import Pool
    pool = Pool([100], 1, 16, 128, 8, torch.Generator().manual_seed(5))
    cache, table = pool.device(q)
    qt = torch.randn((1, 4, 128)).to(torch.bfloat16)
    plan = q.KVPlan(4, 1, 128, 16, max_seqs=1, max_rows=1, max_pages=pool.max_pages)
    clean, out = torch.empty_like(qt, device=DEV), torch.empty_like(qt, device=DEV)
    q.attention(plan, qt.to(DEV), cache, table, _int32([100]), clean)
    qt[0, 2, 7] = float("inf")
    q.attention(plan, qt.to(DEV), cache, table, _int32([100]), out)
    assert torch.isnan(out[0, 2]).all()
    assert torch.equal(out[0, [0, 1, 3]], clean[0, [0, 1, 3]])


@pytest.mark.parametrize("bits", [8, 4])
@pytest.mark.parametrize("d,hq", [(64, 2), (128, 2), (128, 8), (256, 2), (256, 8)])
@pytest.mark.parametrize("what", ["bias_nan", "scale_inf", "large"])
def test_strange_values_reach_no_row_that_does_not_see_them(q, bits, d, hq, what):
    """Positions that only later rows see, and that only earlier rows' windows see."""
    import torch
    n, rows, window = 150, 6, 40

    def change(pool):
        for j in (147, n - rows - window + 2):   # seen by rows 3 to 5, and by rows 0 and 1
            page, slot = pool.place(0, j)
            if what == "bias_nan":
                pool.va[page, 0, slot, 0, 1] = float("nan")
            elif what == "scale_inf":
                pool.va[page, 0, slot, -1, 0] = float("inf")
            else:   # finite, but some codes' values are not in binary16
                pool.va[page, 0, slot] = 65000.0

    got, want, tol, flags, _ = _attend(q, [n], hq, 1, d, bits, rows=rows, window=window, seed=d, change=change)
    assert flags == 0
    got, want, tol = (t.reshape(rows, hq, -1) for t in (got, want, tol))
    assert np.isfinite(got[2]).all()
    assert (np.abs(got[2] - want[2]) <= tol[2]).all()
    if what != "large":
        cols = slice(0, 64) if what == "bias_nan" else slice(d - 64, d)
        for r in (0, 1, 3, 4, 5):
            assert not np.isfinite(got[r][:, cols]).any()
            others = np.delete(np.arange(d), np.arange(d)[cols])
            assert (np.abs(got[r] - want[r])[:, others] <= np.broadcast_to(tol[r], got[r].shape)[:, others]).all()


def test_bad_pages_and_lengths(q):
    """A page out of range reads as zeros; a length past the table leaves rows standing where it says."""
    import torch
    from tests._codes import Pool
    pool = Pool([40], 1, 16, 64, 8, torch.Generator().manual_seed(0), extra=0)
    cache, table = pool.device(q)
    plan = q.KVPlan(2, 1, 64, 16, max_seqs=1, max_rows=1, max_pages=pool.max_pages)
    qt = torch.zeros((1, 2, 64), dtype=torch.bfloat16, device=DEV)
    out = torch.empty_like(qt)
    from tests._codes import values
    v = values(*pool.parts[0][1])[:, 0]
    table[0, 1] = pool.pages + 9
    q.attention(plan, qt, cache, table, _int32([40]), out)   # all weights are equal
    want = (v[:16].sum(0) + v[32:].sum(0)) / 40
    assert plan.error_flags() == q.KV_BAD_PAGE
    assert ((out[0].double().cpu() - want).abs() <= 2.0 ** -8 * want.abs() + 2.0 ** -9 * v.abs().max()).all()


@pytest.mark.parametrize("bits", [8, 4])
def test_views_of_wider_tensors(q, bits):
    """Rows of queries and outputs, and heads of the pool, with gaps between them."""
    import torch
    from tests._codes import Pool
    gen = torch.Generator().manual_seed(6)
    pool = Pool([90, 33], 2, 16, 128, bits, gen, layout="nhd")
    cache, table = pool.device(q)
    wide = [torch.cat((t, t), 1)[:, :2] for t in (cache.k, cache.v, cache.k_affine, cache.v_affine)]
    other = q.QuantKVCache(*wide, bits)
    qt = torch.randn((2, 3 * 4 * 128), generator=gen).to(torch.bfloat16).to(DEV)
    plan = q.KVPlan(4, 2, 128, 16, max_seqs=2, max_rows=1, max_pages=pool.max_pages)
    lens = _int32([90, 33])
    a, b = torch.empty((2, 512), dtype=torch.bfloat16, device=DEV), torch.zeros((2, 2048), dtype=torch.bfloat16, device=DEV)
    q.attention(plan, qt[:, 512:1024], cache, table, lens, a)
    q.attention(plan, qt[:, 512:1024].contiguous(), other, table, lens, b[:, 1024:1536])
    assert torch.equal(a, b[:, 1024:1536])
    assert (b[:, :1024] == 0).all() and (b[:, 1536:] == 0).all()


@pytest.mark.parametrize("bits", [8, 4])
def test_step_in_a_graph_on_another_stream(q, bits):
    """Append, attention and read-back, captured once and replayed as lengths grow, with two plans' graphs side by side."""
    import torch
    from tests._codes import Pool
    H, D, page, S = 2, 128, 16, 3
    runs = []
    for seed in (1, 2):
        gen = torch.Generator().manual_seed(seed)
        pool = Pool([64] * S, H, page, D, bits, gen, extra=0)
        cache, table = pool.device(q)
        plan = q.KVPlan(4, H, D, page, max_seqs=S, max_rows=1, max_pages=pool.max_pages, rot_dim=0)
        x = [torch.randn((S, h * D), generator=gen).to(torch.bfloat16).to(DEV) for h in (4, H, H)]
        lens = _int32([0] * S)
        out, att = torch.empty_like(x[0]), torch.empty_like(x[0])
        back = [torch.zeros((S, 64, H, D), device=DEV) for _ in range(2)]

        def step(plan=plan, x=x, lens=lens, table=table, cache=cache, out=out, att=att, back=back):
            lens.add_(1)
            q.qk_norm_rope(plan, *x, None, None, None, lens, table, cache, out)
            q.attention(plan, out, cache, table, lens, att)
            q.kv_read(plan, cache, table, lens, *back)
            x[1].mul_(-0.5)

        runs.append((step, x, lens, out, att, back, plan))
    results = []
    for graph in (False, True):
        got = []
        for step, x, lens, out, att, back, plan in runs:
            start = [t.clone() for t in x]
            stream = torch.cuda.Stream()
            stream.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(stream):
                run = step
                if graph:
                    step()
                    captured = torch.cuda.CUDAGraph()
                    with torch.cuda.graph(captured, stream=stream):
                        step()
                    run = captured.replay
                lens.zero_()
                for t, u in zip(x, start):
                    t.copy_(u)
                for t in back:
                    t.zero_()
                for _ in range(20):
                    run()
                got.append([t.clone() for t in (att, *back)])
                lens.zero_()
                for t, u in zip(x, start):
                    t.copy_(u)
                stream.synchronize()
            assert plan.error_flags() == 0
        results.append(got)
    for eager, replayed in zip(*results):
        for a, b in zip(eager, replayed):
            assert torch.equal(a, b)
        assert (eager[1][:, 20:] == 0).all() and eager[1][:, :20].abs().sum() > 0

"""Cache append and attention against plain float64 computations: lengths from none to many, pages that end inside
tiles, windows and sinks, rows that see nothing, strange values wherever no row looks, strides and large offsets.

Tolerances, from the arithmetic: outputs are rounded once to bfloat16 (at most 2^-8 of the value between neighbours);
a score's float32 sum of products is off by at most 2^-19 of the sum of their magnitudes, and the weights and their
sums by 2^-15, which move an output by that share of the largest value in sight."""
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


def _pool(torch, gen, lengths, hkv, page, d, layout="hnd", poison=float("nan"), spare=3):
    """Cache tensors full of `poison`, a shuffled page table with garbage in unused entries, and the used values as
    float64 [len, hkv, d] per sequence."""
    used = [max(0, -(-n // page)) for n in lengths]
    max_pages, pages = max(1, max(used)) + 1, sum(used) + spare
    order = torch.randperm(pages, generator=gen)
    table = torch.full((len(lengths), max_pages), -7, dtype=torch.int32)
    table[:, -1] = 1 << 30
    shape = (pages, hkv, page, d) if layout == "hnd" else (pages, page, hkv, d)
    k, v = (torch.full(shape, poison, dtype=torch.bfloat16) for _ in range(2))
    kt, vt = (t if layout == "hnd" else t.transpose(1, 2) for t in (k, v))
    ks, vs, at = [], [], 0
    for i, n in enumerate(lengths):
        own = order[at:at + used[i]]
        at += used[i]
        table[i, :used[i]] = own.int()
        a, b = (torch.randn((max(n, 0), hkv, d), generator=gen).to(torch.bfloat16) for _ in range(2))
        j = torch.arange(max(n, 0))
        kt[own[j // page], :, j % page] = a
        vt[own[j // page], :, j % page] = b
        ks.append(a.double().numpy())
        vs.append(b.double().numpy())
    k, v = k.to(DEV), v.to(DEV)
    if layout != "hnd":
        k, v = k.transpose(1, 2), v.transpose(1, 2)
    return k, v, table.to(DEV), ks, vs, max_pages


def _reference(qs, ks, vs, lengths, rows, window, sinks, scale):
    """float64 outputs [tokens, hq, d] and the largest magnitudes that the tolerance needs."""
    hq, d = qs.shape[1:]
    out = np.zeros(qs.shape)
    tol = np.zeros(qs.shape[:2] + (1,))
    for s, n in enumerate(lengths):
        for r in range(rows):
            pos = n - rows + r
            j = np.arange(max(n, 0))
            see = j <= pos
            if window:
                see &= (pos - j < window) | (j < sinks)
            j = j[see]
            if pos < 0 or not len(j):
                continue
            for h in range(hq):
                kk, vv = ks[s][j, h // (hq // ks[s].shape[1])], vs[s][j, h // (hq // ks[s].shape[1])]
                x = qs[s * rows + r, h]
                a = kk @ x * scale
                e = np.exp(a - a.max())
                out[s * rows + r, h] = (e / e.sum()) @ vv
                size = np.max(np.abs(kk) @ np.abs(x)) * abs(scale)
                tol[s * rows + r, h] = (2.0 ** -15 + 2.0 ** -19 * size) * np.max(np.abs(vv))
    return out, tol + 2.0 ** -8 * np.abs(out)


def _attend(q, torch, lengths, hq, hkv, d, rows=1, page=16, window=0, sinks=0, seed=0, layout="hnd", scale=None,
            q_size=1.5, max_rows=None):
    gen = torch.Generator().manual_seed(seed)
    k, v, table, ks, vs, max_pages = _pool(torch, gen, lengths, hkv, page, d, layout)
    qt = (q_size * torch.randn((len(lengths) * rows, hq, d), generator=gen)).to(torch.bfloat16)
    plan = q.KVPlan(hq, hkv, d, page, max_seqs=len(lengths), max_rows=max_rows or rows, max_pages=max_pages, window=window,
                    sinks=sinks, scale=scale)
    lens = torch.tensor(lengths, dtype=torch.int32, device=DEV)
    out = torch.full((len(lengths) * rows, hq, d), 77.0, dtype=torch.bfloat16, device=DEV)
    q.attention(plan, qt.to(DEV), q.KVCache(k, v), table, lens, out)
    torch.cuda.synchronize()
    assert plan.error_flags() == 0
    want, tol = _reference(qt.double().numpy(), ks, vs, lengths, rows, window, sinks, scale if scale is not None else d ** -0.5)
    got = out.double().cpu().numpy()
    assert np.isfinite(got).all()
    assert (np.abs(got - want) <= tol).all(), np.max(np.abs(got - want) / np.maximum(tol, 1e-30))
    return plan, qt, k, v, table, lens, out


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("lengths", [[1], [0], [2, 0, 1], [15, 16, 17], [63, 64, 65, 129], [1000], [300, 1, 0, 77, 513]])
def test_lengths(q, d, lengths):
    import torch
    _attend(q, torch, lengths, 8, 2, d, seed=len(lengths) * d)


@pytest.mark.parametrize("page", [1, 2, 4, 8, 16, 32, 128, 1024])
def test_page_sizes(q, page):
    import torch
    _attend(q, torch, [1, 37, 250], 4, 2, 128, page=page, seed=page)


@pytest.mark.parametrize("hq,hkv,rows,d", [(1, 1, 1, 64), (5, 1, 3, 128), (14, 2, 1, 128), (16, 1, 1, 256), (17, 1, 1, 64),
                                           (8, 1, 4, 128), (12, 3, 16, 64), (64, 1, 2, 128), (33, 1, 1, 256), (8, 2, 16, 256),
                                           (32, 2, 5, 128), (7, 7, 2, 64), (40, 8, 8, 128)])
@pytest.mark.parametrize("lengths", [[40, 333], [16, 2, 900]])
def test_heads_and_rows(q, hq, hkv, rows, d, lengths):
    """Groups and drafted tokens that fill, overfill and leave odd rests of the row tiles; lengths below `rows` leave
    rows before the first position."""
    import torch
    _attend(q, torch, lengths, hq, hkv, d, rows=rows, seed=hq + rows)


@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 4), (16, 0), (17, 1), (100, 4), (100, 33), (500, 16), (10000, 4),
                                          (128, 10000), (2 ** 31 - 1, 2 ** 31 - 1)])
@pytest.mark.parametrize("rows,d", [(1, 128), (5, 64), (16, 128), (3, 256)])
def test_window_and_sinks(q, window, sinks, rows, d):
    import torch
    _attend(q, torch, [700, 5, 101, 0, 116], 4, 2, d, rows=rows, window=window, sinks=sinks, seed=window % 1000 + sinks % 1000)


def test_many_sequences(q):
    import torch
    rng = np.random.default_rng(3)
    lengths = [int(n) for n in rng.integers(0, 200, 75)] + [2000]
    _attend(q, torch, lengths, 4, 2, 64, seed=8)
    _attend(q, torch, lengths[:33], 6, 1, 128, rows=2, window=64, sinks=2, seed=9)


def test_one_long_sequence(q):
    import torch
    _attend(q, torch, [20011], 4, 1, 128, seed=10)
    _attend(q, torch, [9001, 20000], 2, 1, 256, rows=3, seed=11)


@pytest.mark.parametrize("scale,q_size", [(1.0, 3.0), (-0.3, 1.0), (0.0, 1.0), (0.2, 1e4)])
def test_scales(q, scale, q_size):
    """Scores of thousands, of the other sign, and all alike."""
    import torch
    _attend(q, torch, [5, 400], 4, 2, 128, scale=scale, q_size=q_size, seed=12)


def test_position_major_pages_and_row_strides(q):
    """A pool laid out [pages, page_size, heads, d], queries and outputs inside wider rows, fewer rows than planned."""
    import torch
    plan, qt, k, v, table, lens, out = _attend(q, torch, [100, 31], 8, 2, 128, rows=2, layout="nhd", seed=13, max_rows=16)
    wide_q = torch.full((4, 8 * 128 + 64), float("nan"), dtype=torch.bfloat16, device=DEV)
    wide_q[:, 64:] = qt.view(4, -1).to(DEV)
    wide_o = torch.full((4, 8 * 128 + 8), 5.0, dtype=torch.bfloat16, device=DEV)
    q.attention(plan, wide_q[:, 64:], q.KVCache(k, v), table, lens, wide_o[:, :1024])
    torch.cuda.synchronize()
    assert torch.equal(wide_o[:, :1024].reshape(4, 8, 128), out)
    assert (wide_o[:, 1024:] == 5.0).all()


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("d,rows", [(64, 4), (128, 16), (256, 2)])
def test_values_that_only_later_rows_see(q, bad, d, rows):
    """Keys and values at the drafted positions that are not finite reach the rows that see them and no others."""
    import torch
    gen = torch.Generator().manual_seed(14)
    lengths, hq, hkv = [50 + rows], 4, 2
    k, v, table, ks, vs, max_pages = _pool(torch, gen, lengths, hkv, 16, d)
    n = lengths[0]
    for t, side in ((k, ks), (v, vs)):
        page = table[0, (n - 1) // 16]
        t[page, :, (n - 1) % 16] = bad   # the last position: only the last row sees it
    qt = torch.randn((rows, hq, d), generator=gen).to(torch.bfloat16)
    plan = q.KVPlan(hq, hkv, d, 16, max_seqs=1, max_rows=rows, max_pages=max_pages)
    out = torch.empty((rows, hq, d), dtype=torch.bfloat16, device=DEV)
    q.attention(plan, qt.to(DEV), q.KVCache(k, v), table, torch.tensor(lengths, dtype=torch.int32, device=DEV), out)
    want, tol = _reference(qt.double().numpy(), ks, vs, lengths, rows, 0, 0, d ** -0.5)
    got = out.double().cpu().numpy()
    assert (np.abs(got - want) <= tol)[:-1].all()
    if bad != bad:
        assert np.isnan(got[-1]).all()


def test_infinite_query_stays_in_its_row(q):
    import torch
    gen = torch.Generator().manual_seed(15)
    k, v, table, ks, vs, max_pages = _pool(torch, gen, [90], 1, 16, 128)
    qt = torch.randn((1, 4, 128), generator=gen).to(torch.bfloat16)
    bad = qt.clone()
    bad[0, 2, 5] = float("nan")
    plan = q.KVPlan(4, 1, 128, 16, max_seqs=1, max_rows=1, max_pages=max_pages)
    lens = torch.tensor([90], dtype=torch.int32, device=DEV)
    outs = []
    for x in (qt, bad):
        out = torch.empty((1, 4, 128), dtype=torch.bfloat16, device=DEV)
        q.attention(plan, x.to(DEV), q.KVCache(k, v), table, lens, out)
        outs.append(out.cpu())
    assert torch.equal(outs[0][0, [0, 1, 3]], outs[1][0, [0, 1, 3]])
    assert torch.isnan(outs[1][0, 2].float()).all()


def test_offsets_past_32_bits(q):
    """A pool of more than 2^31 elements whose last pages hold the sequence."""
    import torch
    gen = torch.Generator().manual_seed(16)
    k, v, table, ks, vs, max_pages = _pool(torch, gen, [75], 2, 16, 128, spare=0)
    n = (1 << 31) // (2 * 16 * 128) + 64
    big_k, big_v = (torch.empty((n, 2, 16, 128), dtype=torch.bfloat16, device=DEV) for _ in range(2))
    big_k[-5:], big_v[-5:] = k, v
    far = table.clone()
    far[:, :5] += n - 5
    qt = torch.randn((1, 4, 128), generator=gen).to(torch.bfloat16).to(DEV)
    plan = q.KVPlan(4, 2, 128, 16, max_seqs=1, max_rows=1, max_pages=max_pages)
    lens = torch.tensor([75], dtype=torch.int32, device=DEV)
    near_out, far_out = (torch.empty((1, 4, 128), dtype=torch.bfloat16, device=DEV) for _ in range(2))
    q.attention(plan, qt, q.KVCache(k, v), table, lens, near_out)
    q.attention(plan, qt, q.KVCache(big_k, big_v), far, lens, far_out)
    torch.cuda.synchronize()
    assert plan.error_flags() == 0
    assert torch.equal(near_out, far_out)
    # the append writes there too
    x = torch.randn((1, 128 * 8), generator=gen).to(torch.bfloat16).to(DEV)
    nope = q.KVPlan(4, 2, 128, 16, max_seqs=1, max_rows=1, max_pages=max_pages, rot_dim=0)
    q.qk_norm_rope(nope, x[:, :512], x[:, 512:768], x[:, 768:], None, None, None, lens, far, q.KVCache(big_k, big_v), near_out)
    page = far[0, 74 // 16]
    assert torch.equal(big_k[page, :, 74 % 16].reshape(-1), x[0, 512:768])
    assert torch.equal(big_v[page, :, 74 % 16].reshape(-1), x[0, 768:])


def test_bad_pages_and_lengths_are_recorded(q):
    """What the page table or a length says wrongly is left out and shows in the error word; other sequences are whole."""
    import torch
    plan, qt, k, v, table, lens, out = _attend(q, torch, [100, 90], 4, 2, 128, seed=17)
    wrong = table.clone()
    wrong[0, 2] = k.shape[0]
    got = torch.empty_like(out)
    q.attention(plan, qt.to(DEV), q.KVCache(k, v), wrong, lens, got)
    torch.cuda.synchronize()
    assert plan.error_flags() == q.KV_BAD_PAGE and plan.error_flags() == 0
    assert torch.isfinite(got.float()).all()
    assert torch.allclose(got[1].float(), out[1].float(), rtol=2 ** -7, atol=2 ** -10)
    long = torch.tensor([plan.max_pages * 16 + 1, 90], dtype=torch.int32, device=DEV)
    q.attention(plan, qt.to(DEV), q.KVCache(k, v), torch.clamp(table, 0, k.shape[0] - 1).int(), long, got)
    assert plan.error_flags() == q.KV_BAD_LENGTH
    # the append leaves them out as well
    x = torch.randn((2, 128 * 8), device=DEV).to(torch.bfloat16)
    before = k.clone()
    nope = q.KVPlan(4, 2, 128, 16, max_seqs=2, max_rows=1, max_pages=plan.max_pages, rot_dim=0)
    wrong = torch.full_like(table, -1)
    q.qk_norm_rope(nope, x[:, :512], x[:, 512:768], x[:, 768:], None, None, None, long, wrong, q.KVCache(k, v), got)
    assert nope.error_flags() == q.KV_BAD_PAGE | q.KV_BAD_LENGTH
    assert torch.equal(k.view(torch.int16), before.view(torch.int16))


def test_same_bits_every_time_streams_and_graphs(q):
    """Repeated calls, a stream of its own and a captured graph give the same bits, with the joins of cut heads."""
    import torch
    plan, qt, k, v, table, lens, out = _attend(q, torch, [4000, 17, 2500], 8, 2, 128, rows=2, seed=18)
    qd, cache = qt.to(DEV), q.KVCache(k, v)
    for _ in range(20):
        got = torch.zeros_like(out)
        q.attention(plan, qd, cache, table, lens, got)
        assert torch.equal(got, out)
    stream = torch.cuda.Stream()
    got = torch.zeros_like(out)
    torch.cuda.synchronize()
    q.attention(plan, qd, cache, table, lens, got, stream=stream)
    stream.synchronize()
    assert torch.equal(got, out)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        for _ in range(3):
            q.attention(plan, qd, cache, table, lens, got)
    # lengths are read when the graph runs
    for n in ([4000, 17, 2500], [3, 11, 2500]):   # each within its pages
        lens.copy_(torch.tensor(n, dtype=torch.int32))
        got.zero_()
        graph.replay()
        torch.cuda.synchronize()
        eager = torch.zeros_like(out)
        q.attention(plan, qd, cache, table, lens, eager)
        assert torch.equal(got, eager)
        if n[0] == 4000:
            assert torch.equal(got, out)
    assert plan.error_flags() == 0


def test_library_owned_workspace_and_empty_calls(q):
    import torch
    plan, qt, k, v, table, lens, out = _attend(q, torch, [600], 4, 2, 64, seed=19)
    own = q.KVPlan(4, 2, 64, 16, max_seqs=1, max_rows=1, max_pages=plan.max_pages, torch_workspace=False)
    got = torch.zeros_like(out)
    q.attention(own, qt.to(DEV), q.KVCache(k, v), table, lens, got)
    assert torch.equal(got, out)
    q.attention(own, qt[:0].to(DEV), q.KVCache(k, v), table[:0], lens[:0], got[:0])
    assert own.error_flags() == 0
    own.close()
    with pytest.raises(q.QmmError):   # more rows than planned
        q.attention(plan, torch.cat([qt, qt]).to(DEV), q.KVCache(k, v), table, lens, torch.cat([got, got]))


# ---- append ------------------------------------------------------------------------------------------------------


def _append_reference(x, w, eps, rope, pos, rot, interleaved):
    """x float64 [tokens, heads, d]: normalised and rotated."""
    y = x.copy()
    if w is not None:
        y = y / np.sqrt(np.mean(y * y, axis=2, keepdims=True) + eps) * w
    if rot:
        c, s = rope[pos, :rot // 2][:, None], rope[pos, rot // 2:][:, None]
        a, b = (y[..., 0:rot:2], y[..., 1:rot:2]) if interleaved else (y[..., :rot // 2], y[..., rot // 2:rot])
        a, b = a * c - b * s, b * c + a * s
        if interleaved:
            y[..., 0:rot:2], y[..., 1:rot:2] = a, b
        else:
            y[..., :rot // 2], y[..., rot // 2:rot] = a, b
    return y


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("d,hq,hkv,rot,interleaved,norm,layout", [
    (128, 8, 2, 128, False, True, "hnd"), (128, 5, 1, 128, True, True, "nhd"), (64, 7, 7, 32, False, True, "hnd"),
    (64, 2, 1, 16, True, False, "nhd"), (256, 4, 2, 64, False, True, "nhd"), (256, 3, 1, 256, True, True, "hnd"),
    (128, 8, 4, 96, False, True, "hnd"), (128, 1, 1, 0, False, True, "hnd"), (64, 16, 2, 48, False, False, "hnd"),
])
@pytest.mark.parametrize("lengths,rows", [([1], 1), ([0, 17, 400], 1), ([7, 3, 64], 5), ([130], 130)])
def test_append(q, dtype, d, hq, hkv, rot, interleaved, norm, layout, lengths, rows):
    """Queries, cache slots and everything around them; lengths below `rows` begin with padding rows."""
    import torch
    gen = torch.Generator().manual_seed(d + rot + rows)
    k, v, table, ks, vs, max_pages = _pool(torch, gen, lengths, hkv, 16, d, layout, poison=3.0)
    tokens = len(lengths) * rows
    tdt = torch.float32 if dtype == "f32" else torch.bfloat16
    qkv = (torch.randn((tokens, (hq + 2 * hkv) * d + 8), generator=gen) * 2).to(tdt)
    wq, wk = (torch.rand(d, generator=gen) + 0.5 for _ in range(2)) if norm else (None, None)
    n_rope = max(max(lengths), 1)
    angle = torch.rand((n_rope, max(rot // 2, 1)), generator=gen).double() * 6.3
    rope = torch.cat([angle.cos(), angle.sin()], 1).float()
    plan = q.KVPlan(hq, hkv, d, 16, max_seqs=len(lengths), max_rows=1, max_pages=max_pages, rot_dim=rot, interleaved=interleaved)
    dev = qkv.to(DEV)
    cut = [0, hq * d, (hq + hkv) * d, (hq + 2 * hkv) * d]
    parts = [dev[:, a:b] for a, b in zip(cut, cut[1:])]
    out = torch.full((tokens, hq, d), 9.0, dtype=torch.bfloat16, device=DEV)
    k0, v0 = k.clone(), v.clone()
    q.qk_norm_rope(plan, *parts, None if wq is None else wq.to(DEV), None if wk is None else wk.to(DEV), rope.to(DEV) if rot else None,
                   torch.tensor(lengths, dtype=torch.int32, device=DEV), table, q.KVCache(k, v), out)
    torch.cuda.synchronize()
    assert plan.error_flags() == 0
    x = [qkv[:, a:b].double().numpy().reshape(tokens, -1, d) for a, b in zip(cut, cut[1:])]
    pos = np.array([n - rows + r for n in lengths for r in range(rows)])
    at = np.maximum(pos, 0)
    r64 = rope.double().numpy()
    yq = _append_reference(x[0], None if wq is None else wq.double().numpy(), 1e-6, r64, at, rot, interleaved)
    yk = _append_reference(x[1], None if wk is None else wk.double().numpy(), 1e-6, r64, at, rot, interleaved)

    def near(got, want):
        # one rounding to bfloat16, and float32 sums and products of a pair below 2^-20 of its larger element
        size = np.max(np.abs(want), axis=-1, keepdims=True)
        return np.abs(got - want) <= 2.0 ** -8 * np.abs(want) + 2.0 ** -20 * size

    got_q = out.double().cpu().numpy()
    assert near(got_q[pos >= 0], yq[pos >= 0]).all()
    assert (got_q[pos < 0] == 0).all()
    kc, vc, tab = k.cpu(), v.cpu(), table.cpu()
    touched = torch.zeros(k.shape[0], 16, dtype=torch.bool)
    for t in np.nonzero(pos >= 0)[0]:
        page, slot = int(tab[t // rows, pos[t] // 16]), int(pos[t] % 16)
        touched[page, slot] = True
        assert near(kc[page, :, slot].double().numpy(), yk[t]).all()
        assert torch.equal(vc[page, :, slot], qkv[t, cut[2]:cut[3]].view(hkv, d).to(torch.bfloat16))
    keep = ~touched[:, None, :, None].expand(k.shape)
    assert torch.equal(kc[keep], k0.cpu()[keep]) and torch.equal(vc[keep], v0.cpu()[keep])


def test_append_positions_of_their_own(q):
    """Rotation by given positions; one outside the table leaves its row unrotated and shows in the error word."""
    import torch
    gen = torch.Generator().manual_seed(21)
    k, v, table, ks, vs, max_pages = _pool(torch, gen, [20, 30], 1, 16, 64)
    x = torch.randn((2, 4 * 64), generator=gen)
    rope = torch.randn((10, 64), generator=gen)
    plan = q.KVPlan(2, 1, 64, 16, max_seqs=2, max_rows=1, max_pages=max_pages)
    lens = torch.tensor([20, 30], dtype=torch.int32, device=DEV)
    out = torch.empty((2, 2, 64), dtype=torch.bfloat16, device=DEV)
    for given, flags in (([9, 0], 0), ([3, 10], q.KV_BAD_POSITION), ([-1, 4], q.KV_BAD_POSITION)):
        xd = x.to(DEV)
        q.qk_norm_rope(plan, xd[:, :128], xd[:, 128:192], xd[:, 192:], None, None, rope.to(DEV), lens, table,
                       q.KVCache(k, v), out, positions=torch.tensor(given, dtype=torch.int32, device=DEV))
        assert plan.error_flags() == flags
        for t, at in enumerate(given):
            ok = 0 <= at < 10
            want = _append_reference(x[t:t + 1, :128].double().numpy().reshape(1, 2, 64), None, 0.0, rope.double().numpy(),
                                     np.array([at if ok else 0]), 64 if ok else 0, False)
            size = np.max(np.abs(want))
            assert (np.abs(out[t:t + 1].double().cpu().numpy() - want) <= 2.0 ** -8 * np.abs(want) + 2.0 ** -20 * size).all()


def test_append_then_attend(q):
    """Token by token into an empty cache, each attending to what was appended before, against one call of all rows."""
    import torch
    gen = torch.Generator().manual_seed(22)
    hq, hkv, d, n = 4, 2, 128, 12
    k, v = (torch.full((2, hkv, 16, d), float("nan"), dtype=torch.bfloat16, device=DEV) for _ in range(2))
    cache = q.KVCache(k, v)
    table = torch.tensor([[1, 0]], dtype=torch.int32, device=DEV)
    qkv = torch.randn((n, (hq + 2 * hkv) * d), generator=gen).to(torch.bfloat16).to(DEV)
    w = torch.ones(d, device=DEV)
    angle = torch.arange(n).double()[:, None] * 100.0 ** -(torch.arange(64).double() / 64)
    rope = torch.cat([angle.cos(), angle.sin()], 1).float().to(DEV)
    plan = q.KVPlan(hq, hkv, d, 16, max_seqs=1, max_rows=n, max_pages=2)

    def step(first, rows, out):
        x = qkv[first:first + rows]
        lens = torch.tensor([first + rows], dtype=torch.int32, device=DEV)
        rot = torch.empty((rows, hq, d), dtype=torch.bfloat16, device=DEV)
        q.qk_norm_rope(plan, x[:, :hq * d], x[:, hq * d:(hq + hkv) * d], x[:, (hq + hkv) * d:], w, w, rope, lens, table, cache, rot)
        q.attention(plan, rot, cache, table, lens, out[first:first + rows])

    one = torch.empty((n, hq, d), dtype=torch.bfloat16, device=DEV)
    for t in range(n):
        step(t, 1, one)
    k1 = k.clone()
    k.fill_(float("nan"))
    v.fill_(float("nan"))
    whole = torch.empty_like(one)
    step(0, n, whole)
    torch.cuda.synchronize()
    assert plan.error_flags() == 0
    assert torch.equal(k.view(torch.int16), k1.view(torch.int16))
    assert torch.allclose(one.float(), whole.float(), rtol=2 ** -7, atol=2 ** -12)


def test_long_neighbours_joined_in_runs(q):
    """Two long sequences among many short ones, which a GPU of 152 SMs cuts into 49 and 216 parts that meet in one CTA: the
    49th part of the first is a run of its own there, where the second's first run begins."""
    import torch
    lengths = [388 * 64, 1724 * 64] + [1] * 320
    plan, qt, k, v, table, lens, out = _attend(q, torch, lengths, 2, 1, 64, page=128, seed=5)
    dev, cache = qt.to(DEV), q.KVCache(k, v)
    for _ in range(30):
        again = torch.full_like(out, 77.0)
        q.attention(plan, dev, cache, table, lens, again)
        assert torch.equal(again, out)
    assert plan.error_flags() == 0

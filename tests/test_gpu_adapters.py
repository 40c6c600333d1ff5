"""Low-rank adapters of many requests against float64.

Tolerances, from the arithmetic: x A^T is a float32 sum of K products (off by at most K 2^-24 of the sum of their magnitudes,
and more where the tensor cores cut sums short: 2^-22 a product of 16 is taken) times the scale (2^-24), held within 2^-17;
the second sum is of 2 rank + 1 terms in float32. All of it moves an output by that share of the sum of magnitudes of its
terms; the output is rounded once (float32 2^-24, bfloat16 2^-8)."""
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


class Case:
    def __init__(self, q, rows, K, N, rank, adapters, dtype, ids=None, seed=0, scale=True, max_rows=None, plan=None):
        import torch
        gen = torch.Generator().manual_seed(seed)
        self.dtype = getattr(torch, dtype)
        normal = lambda *s: torch.randn(s, generator=gen)  # noqa: E731
        self.x = normal(rows, K).to(torch.bfloat16)
        self.a = (normal(adapters, rank, K) * K ** -0.5).to(torch.bfloat16)
        self.b = (normal(adapters, N, rank) * rank ** -0.5).to(torch.bfloat16)
        self.y = normal(rows, N).to(self.dtype)
        self.scale = (0.5 + torch.rand(adapters, generator=gen)) if scale else None
        self.ids = torch.randint(-1, adapters, (rows,), generator=gen).int() if ids is None else torch.tensor(ids, dtype=torch.int32)
        self.plan = plan or q.AdapterPlan(K, N, rank, adapters, max_rows or rows, out_dtype=self.dtype)
        self.q = q

    def tensors(self):
        return [None if t is None else t.to(DEV) for t in (self.x, self.a, self.b, self.scale, self.ids)]

    def run(self, out=None, y=None):
        import torch
        y = self.y.to(DEV) if y is None else y
        out = torch.full_like(y, 7.0) if out is None else out
        self.q.add_adapters(self.plan, *self.tensors(), y, out)
        torch.cuda.synchronize()
        return out

    def check(self, out):
        import torch
        K, rank = self.x.shape[1], self.a.shape[1]
        want, size = self.y.double(), self.y.double().abs()
        for i in range(self.a.shape[0]):
            m = (self.ids == i).nonzero()[:, 0]
            s = float(self.scale[i]) if self.scale is not None else 1.0
            x, a, b = self.x[m].double(), self.a[i].double(), self.b[i].double()
            want[m] += s * (x @ a.T) @ b.T
            size[m] += s * (x.abs() @ a.abs().T) @ b.abs().T
        rounding = 2.0 ** -24 if self.dtype == torch.float32 else 2.0 ** -8
        bound = rounding * want.abs() + (K / 16 * 2.0 ** -22 + 2.0 ** -17 + 2.0 ** -23 + (2 * rank + 1) / 16 * 2.0 ** -22) * size
        err = (out.double().cpu() - want).abs()
        assert (err <= bound).all(), float((err / bound).max())
        # over all outputs roundings do not all fall the same way
        assert float(err.norm()) <= (4e-6 if self.dtype == torch.float32 else 2.0 ** -8) * float(want.norm())


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
@pytest.mark.parametrize("rows,K,N,rank,adapters", [
    (1, 64, 1, 8, 1), (1, 2048, 2048, 16, 4), (3, 128, 33, 24, 2), (16, 4096, 1000, 16, 16), (17, 320, 517, 40, 5),
    (64, 1024, 640, 64, 32), (65, 64, 255, 8, 3), (130, 576, 100, 128, 7), (300, 256, 96, 72, 2), (1000, 192, 64, 16, 64)])
def test_shapes(q, dtype, rows, K, N, rank, adapters):
    c = Case(q, rows, K, N, rank, adapters, dtype, seed=rows + N, scale=rows != 17)
    c.check(c.run())
    assert c.plan.error_flags() == 0


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
@pytest.mark.parametrize("N,rank", [(1728, 32), (1704, 32), (1701, 64), (1728, 64), (1728, 128), (1704, 128), (1703, 104), (1696, 40)])
def test_many_columns_of_a_warp(q, dtype, N, rank):
    """So many rows that each warp has several units of 32 columns, whole and cut short, of one tile and of two."""
    gen = np.random.default_rng(N + rank)
    ids = np.repeat(gen.integers(-1, 9, 64), gen.integers(1, 80, 64))[:2100].tolist()
    c = Case(q, len(ids), 64, N, rank, 9, dtype, ids=ids, seed=N)
    c.check(c.run())


@pytest.mark.parametrize("ids", [[-1] * 70, [2] * 70, [0, 1] * 35, list(range(35)) * 2, [34] * 16 + [-1] * 16 + [3] * 38,
                                 [3] * 17 + [5] * 15 + [3] * 38, [-1] * 69 + [0]])
def test_orders_of_adapters(q, ids):
    c = Case(q, 70, 128, 80, 16, 35, "float32", ids=ids, seed=1)
    c.check(c.run())


def test_rows_without_an_adapter_are_copied(q):
    import torch
    c = Case(q, 20, 64, 50, 8, 2, "bfloat16", ids=[-1, 1] * 10)
    out = c.run()
    assert torch.equal(out[0::2].cpu(), c.y[0::2])
    c.check(out)


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
@pytest.mark.parametrize("N", [64, 83])
def test_in_place(q, dtype, N):
    import torch
    c = Case(q, 40, 128, N, 16, 6, dtype)
    apart, y = c.run(), c.y.to(DEV)
    assert torch.equal(c.run(out=y, y=y), apart)
    c.check(y)


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
def test_strided_rows(q, dtype):
    """Rows inside wider tensors, at places that are not 16-byte aligned; what lies between them stays."""
    import torch
    c = Case(q, 19, 128, 70, 16, 4, dtype)
    want = c.run()
    for shift in (0, 1, 8):
        wide_x = torch.zeros((19, 400), dtype=torch.bfloat16, device=DEV)
        wide_x[:, 64:192] = c.x.to(DEV)
        wide_y, wide_out = (torch.full((19, 90 + k), 3.0, dtype=c.dtype, device=DEV) for k in (0, 6))
        y, out = wide_y[:, shift:shift + 70], wide_out[:, shift:shift + 70]
        y.copy_(c.y)
        t = c.tensors()
        c.q.add_adapters(c.plan, wide_x[:, 64:192], *t[1:], y, out)
        assert torch.equal(out, want)
        assert (wide_out[:, :shift] == 3.0).all() and (wide_out[:, shift + 70:] == 3.0).all()


def test_ids_out_of_range(q):
    import torch
    c = Case(q, 6, 64, 32, 8, 3, "float32", ids=[0, 3, -2, 2, 2 ** 31 - 1, -2 ** 31])
    out = c.run()
    assert c.plan.error_flags() == q.ADAPTER_BAD_ID
    assert c.plan.error_flags() == 0
    c.ids = torch.where((c.ids < 0) | (c.ids >= 3), -1, c.ids)
    c.check(out)


def test_strange_values_stay_in_their_rows(q):
    import torch
    c = Case(q, 8, 64, 32, 8, 2, "float32", ids=[0, 1] * 4)
    clean = c.run()
    c.x[2, 5], c.x[3, 9] = float("inf"), float("nan")
    out = c.run()
    rest = [0, 1, 4, 5, 6, 7]
    assert torch.equal(out[rest], clean[rest])
    assert torch.isnan(out[3]).all()
    assert not torch.isfinite(out[2]).all()
    # an infinite product keeps its sign where nothing cancels it: one column of A and B
    c.a[0].zero_()
    c.b[0].zero_()
    c.a[0, 0], c.b[0, :, 0] = 1.0, 1.0
    c.x[2] = c.x[2].abs()
    out = c.run()
    assert not torch.isfinite(out[2]).any()


def test_fewer_rows_than_the_plan_and_the_same_bits(q):
    """A plan for many rows; a call's bits do not depend on what was called before."""
    import torch
    big = Case(q, 200, 256, 128, 32, 8, "bfloat16", seed=3)
    small = Case(q, 5, 256, 128, 32, 8, "bfloat16", seed=4, plan=big.plan)
    first = small.run()
    big.check(big.run())
    assert torch.equal(small.run(), first)
    small.check(first)
    empty = torch.empty((0, 128), dtype=torch.bfloat16, device=DEV)
    t = big.tensors()
    q.add_adapters(big.plan, t[0][:0], t[1], t[2], t[3], t[4][:0], empty, empty)


def test_beside_a_projection_in_a_graph(q):
    """y = projection(x) with its adapters, captured on a stream and replayed with other rows, and two plans at once."""
    import torch
    K, N, M = 1024, 512, 12
    gen = torch.Generator(device=DEV).manual_seed(0)
    words = torch.randint(-2 ** 31, 2 ** 31, (N, K * 4 // 32), generator=gen, device=DEV, dtype=torch.int32)
    scales = torch.full((N, K // 64), 0.01, dtype=torch.float16, device=DEV)
    plan = q.Plan(K, N, 4, 64, max_M=M, out_dtype="bf16")
    runs = []
    for seed in (1, 2):
        c = Case(q, M, K, N, 16, 5, "bfloat16", seed=seed)
        t = c.tensors()
        y, out = (torch.empty((M, N), dtype=torch.bfloat16, device=DEV) for _ in range(2))

        def step(c=c, t=t, y=y, out=out):
            q.forward(plan, t[0], words, scales, -7.5 * scales, y)
            q.add_adapters(c.plan, *t, y, out)

        runs.append((c, t, y, out, step))
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        graphs = []
        for *_, step in runs:
            step()
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=stream):
                step()
            graphs.append(g)
        for turn in range(3):
            for (c, t, y, out, step), g in zip(runs, graphs):
                t[0].copy_(c.x.roll(turn, 0))
                t[4].copy_(c.ids.roll(turn, 0))
                g.replay()
            for c, t, y, out, step in runs:
                stream.synchronize()
                now = Case(q, M, K, N, 16, 5, "bfloat16", plan=c.plan)
                now.x, now.a, now.b, now.scale, now.ids, now.y = c.x.roll(turn, 0), c.a, c.b, c.scale, c.ids.roll(turn, 0), y.cpu()
                now.check(out)


def test_two_threads_share_a_plan(q):
    """Host threads that launch on one stream: no call's two kernels have another's between them."""
    import threading

    import torch
    a = Case(q, 40, 256, 128, 16, 6, "bfloat16", seed=1)
    b = Case(q, 33, 256, 128, 16, 6, "bfloat16", seed=2, plan=a.plan)
    want = [c.run() for c in (a, b)]
    stream = torch.cuda.Stream()
    work = [(c.tensors(), c.y.to(DEV), [torch.empty_like(w) for _ in range(50)]) for c, w in zip((a, b), want)]
    torch.cuda.synchronize()

    def launch(t, y, outs):
        for out in outs:
            q.add_adapters(a.plan, *t, y, out, stream=stream)

    threads = [threading.Thread(target=launch, args=w) for w in work]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    for w, (_, _, outs) in zip(want, work):
        assert all(torch.equal(out, w) for out in outs)


def test_y_is_the_kernel_before_and_out_the_one_after(q):
    """y, x and ids written just before the call on the stream, out read just after, many times in a row."""
    import torch
    c = Case(q, 50, 512, 300, 32, 5, "bfloat16")
    x, a, b, scale, ids = c.tensors()
    want = c.run()
    xs, ys, idss, out, seen = torch.zeros_like(x), torch.zeros_like(c.y.to(DEV)), torch.full_like(ids, -1), c.y.to(DEV), []
    y = c.y.to(DEV)
    for i in range(30):
        for t in (xs, ys, idss):
            t.fill_(0)
        xs.copy_(x)
        idss.copy_(ids)
        ys.copy_(y)
        q.add_adapters(c.plan, xs, a, b, scale, idss, ys, ys if i % 2 else out)
        seen.append((ys if i % 2 else out).clone())
    assert all(torch.equal(s, want) for s in seen)


def test_far_into_large_tensors(q):
    """Adapters that lie past 2^32 bytes."""
    import torch
    K, N, rank, n = 8192, 8192, 128, 2100
    a = torch.zeros((n, rank, K), dtype=torch.bfloat16, device=DEV)
    b = torch.zeros((n, N, rank), dtype=torch.bfloat16, device=DEV)
    a[-1, 3] = 1.0
    b[-1, :, 3] = 0.5
    x = torch.ones((2, K), dtype=torch.bfloat16, device=DEV)
    y = torch.ones((2, N), device=DEV)
    plan = q.AdapterPlan(K, N, rank, n, 2, out_dtype="f32")
    out = torch.empty_like(y)
    q.add_adapters(plan, x, a, b, None, torch.tensor([n - 1, 0], dtype=torch.int32, device=DEV), y, out)
    assert (out[0] == 1 + K / 2).all() and (out[1] == 1).all()

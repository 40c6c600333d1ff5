"""Plans of caches of codes and of adapters next to other work on the GPU, and calls of nothing."""
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


@pytest.mark.parametrize("rows", [1, 3, 12])
def test_one_plan_for_caches_of_every_kind(q, rows):
    """Heads that are cut and joined, by the last CTA of each or by a launch of its own, of caches of 16, 8 and 4 bits in turn."""
    import torch
    from tests._codes import Pool
    n, page = 9000, 16
    pools = [Pool([n], 2, page, 128, bits, torch.Generator().manual_seed(bits)) for bits in (8, 4)]
    calls = [pool.device(q) for pool in pools]
    dense = torch.randn((2, pools[0].pages, 2, page, 128), generator=torch.Generator().manual_seed(5)).to(DEV, torch.bfloat16)
    calls.append((q.KVCache(dense[0], dense[1]), calls[0][1]))
    x = torch.randn((rows, 8, 128), generator=torch.Generator().manual_seed(6)).to(DEV, torch.bfloat16)
    lengths = torch.tensor([n], dtype=torch.int32, device=DEV)
    make = lambda: q.KVPlan(8, 2, 128, page, max_seqs=1, max_rows=rows, max_pages=pools[0].max_pages)  # noqa: E731

    def run(plan, cache, table):
        out = torch.full_like(x, 7.0)
        q.attention(plan, x, cache, table, lengths, out)
        return out

    plans = [make() for _ in calls]
    want = [run(plan, *call) for plan, call in zip(plans, calls)]
    shared = make()
    got = [[run(shared, *call) for call in calls] for _ in range(8)]
    assert shared.error_flags() == 0
    for some in got:
        assert all(torch.equal(a, b) for a, b in zip(some, want))


class Adapters:
    def __init__(self, q, torch, rows=40, K=512, N=700, rank=16, adapters=5):
        gen = torch.Generator(device=DEV).manual_seed(1)
        normal = lambda *s: torch.randn(s, generator=gen, device=DEV).to(torch.bfloat16)  # noqa: E731
        self.q, self.make = q, lambda **kw: q.AdapterPlan(K, N, rank, adapters, rows, **kw)
        self.x, self.a, self.b, self.y = normal(rows, K), normal(adapters, rank, K), normal(adapters, N, rank), normal(rows, N)
        self.scale = torch.rand(adapters, generator=gen, device=DEV)
        self.ids = torch.randint(-1, adapters, (rows,), generator=gen, device=DEV).int()

    def __call__(self, plan, ids=None):
        import torch
        out = torch.empty_like(self.y)
        self.q.add_adapters(plan, self.x, self.a, self.b, self.scale, self.ids if ids is None else ids, self.y, out)
        return out


def test_an_adapter_plan_made_behind_a_late_write_to_its_block(q):
    """On a side stream, whose freed blocks are given out again at once."""
    import torch
    step = Adapters(q, torch)
    want = step(step.make())
    nbytes = step.make().workspace.numel()
    torch.cuda.synchronize()
    room = torch.empty(1 << 31, dtype=torch.uint8, device=DEV)
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        block = torch.empty(nbytes, dtype=torch.uint8, device=DEV)
        at = block.data_ptr()
        for i in range(40):
            room.fill_(i)
        block.fill_(255)
        del block
        plan = step.make()
        out = step(plan)
        flags = plan.error_flags()
    assert plan.workspace.data_ptr() == at
    assert flags == 0 and torch.equal(out, want)


def test_error_flags_of_adapters_wait_and_are_cleared(q):
    import torch
    step = Adapters(q, torch)
    plan = step.make()
    bad = step.ids.clone()
    bad[7] = 99
    room = torch.empty(1 << 31, dtype=torch.uint8, device=DEV)
    with torch.cuda.stream(torch.cuda.Stream()):
        for i in range(40):
            room.fill_(i)
        step(plan, bad)
    assert plan.error_flags() == q.ADAPTER_BAD_ID
    assert plan.error_flags() == 0


def test_workspace_of_the_library(q):
    import torch
    step = Adapters(q, torch)
    plan = step.make(torch_workspace=False)
    assert plan.workspace is None and torch.equal(step(plan), step(step.make()))
    plan.close()


def test_two_graphs_of_one_adapter_plan(q):
    """Replayed one after the other, in either order."""
    import torch
    step = Adapters(q, torch)
    plan = step.make()
    other = (step.ids + 2) % 6 - 1
    want = [step(plan), step(plan, other.int())]
    outs = [torch.empty_like(step.y) for _ in range(2)]
    stream = torch.cuda.Stream()
    graphs = []
    with torch.cuda.stream(stream):
        for out, ids in zip(outs, (step.ids, other.int())):
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=stream):
                q.add_adapters(plan, step.x, step.a, step.b, step.scale, ids, step.y, out)
            graphs.append(g)
        for order in ((0, 1), (1, 0), (0, 0, 1)):
            for out in outs:
                out.fill_(0)
            for i in order:
                graphs[i].replay()
            stream.synchronize()
            assert all(torch.equal(o, w) for o, w in zip(outs, want))


def test_calls_of_nothing(q):
    import torch
    from tests._codes import Pool
    step = Adapters(q, torch)
    plan = step.make()
    none = torch.empty(0, dtype=torch.int32, device=DEV)
    q.add_adapters(plan, step.x[:0], step.a, step.b, None, none, step.y[:0], step.y[:0])
    q.logprobs(step.y[:0], none, none.float(), none.float(), torch.empty((0, 3), dtype=torch.int32, device=DEV),
               torch.empty((0, 3), device=DEV))
    pool = Pool([20], 1, 16, 64, 8, torch.Generator().manual_seed(0))
    cache, table = pool.device(q)
    kv = q.KVPlan(1, 1, 64, 16, max_seqs=2, max_rows=1, max_pages=pool.max_pages)
    kept = torch.full((2, 1, 4, 1, 64), 7.0, device=DEV)
    q.kv_read(kv, cache, table[:0], none, kept[0, :0], kept[1, :0])
    lengths = torch.tensor([20], dtype=torch.int32, device=DEV)
    q.kv_read(kv, cache, table, lengths, kept[0, :, :0], kept[1, :, :0])
    q.kv_read(kv, cache, table, torch.zeros_like(lengths), kept[0], kept[1])
    q.attention(kv, step.x[:0, :64], cache, table[:0], none, torch.empty((0, 1, 64), dtype=torch.bfloat16, device=DEV))
    torch.cuda.synchronize()
    assert (kept == 7.0).all() and plan.error_flags() == 0 and kv.error_flags() == 0

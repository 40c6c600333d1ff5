"""Plans next to other work on the GPU."""
from __future__ import annotations

import pytest

pytestmark = pytest.mark.gpu

DEV = "cuda"
PAGE, MAX_PAGES = 16, 600


@pytest.fixture(scope="module")
def q():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from bit_affine_quantized_group_gb300 import _build
    _build.build()
    import bit_affine_quantized_group_gb300 as q
    return q


def _busy(torch, n=80):
    """Some tens of milliseconds of work on the current stream."""
    room = torch.empty(1 << 31, dtype=torch.uint8, device=DEV)
    for i in range(n):
        room.fill_(i)


class Step:
    """Heads that are cut and joined: one sequence over all SMs."""

    def __init__(self, q, torch, rows=1, seed=0):
        self.q, self.torch = q, torch
        gen = torch.Generator(device=DEV).manual_seed(seed)
        normal = lambda *s: torch.randn(s, generator=gen, device=DEV).to(torch.bfloat16)  # noqa: E731
        self.rows = rows
        self.queries = normal(rows, 8, 128)
        self.cache = q.KVCache(normal(MAX_PAGES, 2, PAGE, 128), normal(MAX_PAGES, 2, PAGE, 128))
        self.table = torch.randperm(MAX_PAGES, generator=gen, device=DEV).int()[None]
        self.lengths = torch.tensor([MAX_PAGES * PAGE - 3], dtype=torch.int32, device=DEV)

    def plan(self, **kw):
        return self.q.KVPlan(8, 2, 128, PAGE, max_seqs=1, max_rows=self.rows, max_pages=MAX_PAGES, **kw)

    def __call__(self, plan, table=None):
        out = self.torch.full_like(self.queries, 77.0)
        self.q.attention(plan, self.queries, self.cache, self.table if table is None else table, self.lengths, out)
        return out


@pytest.mark.parametrize("rows", [1, 8])
def test_a_plan_made_behind_a_late_write_to_its_block(q, rows):
    """On a side stream, whose freed blocks are given out again at once."""
    import torch
    step = Step(q, torch, rows)
    want = step(step.plan())
    plan0 = step.plan()
    nbytes = plan0.workspace.numel()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        block = torch.empty(nbytes, dtype=torch.uint8, device=DEV)
        at = block.data_ptr()
        _busy(torch)
        block.fill_(255)
        del block
        plan = step.plan()
        assert plan.workspace.data_ptr() == at   # the same block
        outs = [step(plan) for _ in range(3)]
        side.synchronize()
        assert plan.error_flags() == 0
    for out in outs:
        assert torch.equal(out, want)


def test_a_projection_plan_made_behind_a_late_write_to_its_block(q):
    import torch
    gen = torch.Generator(device=DEV).manual_seed(1)
    K, N, M = 4096, 1024, 8
    x = torch.randn((M, K), generator=gen, device=DEV).to(torch.bfloat16)
    w = torch.randint(-2 ** 31, 2 ** 31, (N, K * 4 // 32), generator=gen, device=DEV, dtype=torch.int32)
    s = torch.full((N, K // 64), 0.01, dtype=torch.float16, device=DEV)
    b = -7.5 * s

    def make():
        return q.Plan(K, N, 4, 64, max_M=M, out_dtype="f32", splits=4)

    def run(plan):
        out = torch.empty((M, N), device=DEV)
        q.forward(plan, x, w, s, b, out)
        return out

    plan0 = make()
    want = run(plan0)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        block = torch.empty(plan0.workspace.numel(), dtype=torch.uint8, device=DEV)
        at = block.data_ptr()
        _busy(torch)
        block.fill_(255)
        del block
        plan = make()
        assert plan.workspace.data_ptr() == at   # the same block
        got = run(plan)
        side.synchronize()
        assert plan.error_flags() == 0
    assert torch.equal(got, want)


def test_error_flags_of_calls_in_flight(q):
    """Asked for while the call with the fault still waits on a side stream, and not lost or kept by the clearing."""
    import torch
    step = Step(q, torch)
    plan = step.plan()
    want = step(plan)
    wrong = step.table.clone()
    wrong[0, 5] = MAX_PAGES
    torch.cuda.synchronize()
    assert plan.error_flags() == 0
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        for _ in range(3):
            _busy(torch, 20)
            step(plan, wrong)
            assert plan.error_flags() == q.KV_BAD_PAGE
            out = step(plan)
            assert plan.error_flags() == 0
            assert torch.equal(out, want)
            step(plan, wrong)   # right behind a clearing
            assert plan.error_flags() == q.KV_BAD_PAGE


def test_error_flags_of_projections_in_flight(q):
    """A bit that is set late, here by a write to the workspace, for no call sets one on purpose."""
    import torch
    plan = q.Plan(1024, 256, 4, 64, max_M=4)
    word = (plan.workspace.data_ptr() + 255) // 256 * 256 - plan.workspace.data_ptr()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        for _ in range(3):
            _busy(torch, 20)
            plan.workspace[word:word + 1].fill_(1)
            assert plan.error_flags() == 1
            plan.workspace[word:word + 1].fill_(2)   # right behind a clearing
            assert plan.error_flags() == 2 and plan.error_flags() == 0


@pytest.mark.parametrize("rows", [1, 8])
def test_threads_share_a_plan_and_a_stream(q, rows):
    """Calls of two threads give the bits of one, with parts that the call's own kernel joins or a second one."""
    import threading

    import torch
    steps = [Step(q, torch, rows, seed=i) for i in range(2)]
    plan = steps[0].plan()
    want = [step(plan) for step in steps]
    n = 200
    outs = [[torch.full_like(w, 77.0) for _ in range(n)] for w in want]
    torch.cuda.synchronize()
    start = threading.Barrier(2)

    def run(step, out):
        start.wait()
        for o in out:
            q.attention(plan, step.queries, step.cache, step.table, step.lengths, o)

    threads = [threading.Thread(target=run, args=a) for a in zip(steps, outs)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert plan.error_flags() == 0
    for w, out in zip(want, outs):
        assert all(torch.equal(o, w) for o in out)

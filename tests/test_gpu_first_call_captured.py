"""The first calls of a process may be captured ones: what a kernel needs before its first launch is done then. And a plan for
bfloat16 caches alone prepares nothing of caches of codes."""
from __future__ import annotations

import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

STEP = """
import sys, torch
sys.path.insert(0, sys.argv[1])
import bit_affine_quantized_group_gb300 as q
bits, rows, d = (int(x) for x in sys.argv[2:5])
H, page, n = 2, 16, 100
w = d * bits // 8
gen = torch.Generator().manual_seed(0)
pool = [torch.zeros((8, H, page, w), dtype=torch.uint8, device="cuda") for _ in range(2)]
pool += [torch.zeros((8, H, page, d // 64, 2), dtype=torch.float16, device="cuda") for _ in range(2)]
plan = q.KVPlan(4 * H, H, d, page, max_seqs=1, max_rows=rows, max_pages=8, rot_dim=0)
adapters = q.AdapterPlan(64, 40, 16, 2, 4, out_dtype="f32")
x = [torch.randn((n, h * d), generator=gen).to(torch.bfloat16).cuda() for h in (4 * H, H, H)]
lens, table = torch.tensor([n], dtype=torch.int32, device="cuda"), torch.arange(8, dtype=torch.int32, device="cuda").view(1, 8)
out = torch.empty_like(x[0])
att = torch.empty((rows, 4 * H, d), dtype=torch.bfloat16, device="cuda")
back = [torch.zeros((1, n, H, d), device="cuda") for _ in range(2)]
ax, aa, ab = (torch.randn(s, generator=gen).to(torch.bfloat16).cuda() for s in ((4, 64), (2, 16, 64), (2, 40, 16)))
ids = torch.tensor([0, 1, -1, 1], dtype=torch.int32, device="cuda")
y, ay = torch.randn((4, 40), generator=gen).cuda(), torch.empty((4, 40), device="cuda")
lp = torch.empty(4, device="cuda")


def step():
    cache = q.QuantKVCache(*pool, bits)
    q.qk_norm_rope(plan, *x, None, None, None, lens, table, cache, out)
    q.attention(plan, out[n - rows:], cache, table, lens, att)
    q.kv_read(plan, cache, table, lens, *back)
    q.add_adapters(adapters, ax, aa, ab, None, ids, y, ay)
    q.logprobs(ay, ids.clamp(min=0), lp)


torch.cuda.synchronize()
stream = torch.cuda.Stream()
with torch.cuda.stream(stream):
    ids.clamp(min=0)   # (torch's own kernel is not the matter)
    stream.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=stream):
        step()
    g.replay()
    stream.synchronize()
    got = [t.clone() for t in (out, att, *back, ay, lp)]
    for t in (out, att, *back, ay, lp):
        t.zero_()
    step()
    stream.synchronize()
assert all(torch.equal(a, b) for a, b in zip(got, (out, att, *back, ay, lp)))
assert att.abs().sum() > 0 and lp.abs().sum() > 0 and plan.error_flags() == 0 and adapters.error_flags() == 0
print("equal")
"""


@pytest.mark.parametrize("bits,rows,d", [(8, 1, 128), (4, 8, 64)])
def test_first_calls_of_a_process_are_captured(bits, rows, d):
    from bit_affine_quantized_group_gb300 import _build
    _build.build()
    r = subprocess.run([sys.executable, "-c", STEP, ROOT, str(bits), str(rows), str(d)], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "equal" in r.stdout, r.stderr[-2000:]

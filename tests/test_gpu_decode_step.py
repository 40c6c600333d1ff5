"""The operators between the projections, together: the example's decode steps, eager and replayed from a graph, and its
attention layers against a float64 computation over everything that was appended."""
from __future__ import annotations

import os
import sys

import numpy as np
import pytest

pytestmark = pytest.mark.gpu

EXAMPLES = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples")


@pytest.fixture(scope="module")
def example():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from bit_affine_quantized_group_gb300 import _build
    _build.build()
    if EXAMPLES not in sys.path:
        sys.path.insert(0, EXAMPLES)
    import decode_step
    return decode_step


SMALL = dict(layers=2, hidden=256, q_heads=4, kv_heads=2, head_dim=64, ffn=512, vocab=1000, max_len=64)


@pytest.mark.parametrize("sequences,window,sinks", [(1, 0, 0), (5, 0, 0), (16, 8, 2)])
def test_eager_and_graph_draw_the_same(example, sequences, window, sinks):
    import torch
    d = example.Decoder(sequences=sequences, window=window, sinks=sinks, **SMALL)
    eager, _ = d.generate(40, graph=False)
    d.restart()
    replayed, _ = d.generate(40, graph=True)
    assert torch.equal(eager, replayed)
    assert ((eager >= 0) & (eager < SMALL["vocab"])).all()
    assert len(torch.unique(eager[:, 0])) > 5   # random weights do not repeat themselves


def test_last_step_against_float64(example):
    """The last layer's attended values from its cache and queries; the drawn token from the last logits."""
    import torch
    d = example.Decoder(sequences=3, **SMALL)
    d.generate(37, graph=False)
    n, S, D, hq, hkv = 37, 3, 64, 4, 2
    page, slot = d.page_table.long()[:, torch.arange(n) // 16], torch.arange(n, device="cuda") % 16
    k = d.caches[-1].k[page, :, slot[None].expand(S, n)].double().cpu().numpy()   # [S, n, hkv, D]
    v = d.caches[-1].v[page, :, slot[None].expand(S, n)].double().cpu().numpy()
    q = d.queries.view(S, hq, D).double().cpu().numpy()
    want = np.zeros((S, hq, D))
    for s in range(S):
        for h in range(hq):
            a = k[s, :, h // (hq // hkv)] @ q[s, h] * D ** -0.5
            e = np.exp(a - a.max())
            want[s, h] = e / e.sum() @ v[s, :, h // (hq // hkv)]
    got = d.attended.view(S, hq, D).double().cpu().numpy()
    # one rounding to bfloat16, and 2^-12 of the largest value for the scores' and weights' float32 arithmetic
    assert (np.abs(got - want) <= 2.0 ** -8 * np.abs(want) + 2.0 ** -12 * np.abs(v).max()).all()
    logits = d.head.out.double().cpu().numpy()
    for s in range(S):
        order = np.argsort(-logits[s], kind="stable")[:40]
        assert int(d.tokens[s]) in order
        assert 0.0 < float(d.probs[s]) <= 1.0

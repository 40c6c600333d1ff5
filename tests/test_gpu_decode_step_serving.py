"""The example's decode steps with a cache of codes, adapters beside the q/k/v projections and log probabilities, eager and
replayed from a graph, and its last step against float64 computations from what the step read."""
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


@pytest.mark.parametrize("sequences,bits,adapters,top,window", [(1, 8, 1, 5, 0), (5, 4, 3, 1, 0), (16, 8, 4, 20, 8), (3, 16, 2, 32, 0)])
def test_eager_and_graph_draw_the_same(example, sequences, bits, adapters, top, window):
    import torch
    d = example.Decoder(sequences=sequences, cache_bits=bits, adapters=adapters, top=top, window=window, sinks=2 if window else 0,
                        rank=8, **SMALL)
    eager, _ = d.generate(40, graph=False)
    scores = [t.clone() for t in d.scores]
    d.restart()
    replayed, _ = d.generate(40, graph=True)
    assert torch.equal(eager, replayed)
    assert all(torch.equal(a, b) for a, b in zip(scores, d.scores))
    assert ((eager >= 0) & (eager < SMALL["vocab"])).all()
    assert len(torch.unique(eager[:, 0])) > 5   # random weights do not repeat themselves


@pytest.mark.parametrize("bits", [8, 4])
def test_last_step_against_float64(example, bits):
    """The last layer's attended values from its codes and queries, and the scores from the last logits."""
    import torch
    from tests._codes import unpack, values
    qmm = example.qmm
    d = example.Decoder(sequences=3, cache_bits=bits, adapters=2, rank=8, top=7, **SMALL)
    d.generate(37, graph=False)
    n, S, D, hq, hkv = 37, 3, 64, 4, 2
    cache = d.caches[-1]
    page, slot = d.page_table.long()[:, torch.arange(n) // 16].cpu(), torch.arange(n)[None].expand(S, n) % 16
    k, v = (values(unpack(c.cpu()[page, :, slot], bits), a.cpu()[page, :, slot]).numpy()
            for c, a in ((cache.k, cache.k_affine), (cache.v, cache.v_affine)))     # [S, n, hkv, D]
    back = [torch.zeros((S, n, hkv, D), device="cuda") for _ in range(2)]
    qmm.kv_read(d.kv, cache, d.page_table, d.lengths, *back)
    assert (back[0].cpu().numpy() == k.astype(np.float32)).all() and (back[1].cpu().numpy() == v.astype(np.float32)).all()
    q = d.queries.view(S, hq, D).double().cpu().numpy()
    step = np.abs(cache.k_affine.double().cpu()[page, :, slot][..., 0].numpy())   # scales [S, n, hkv, 1]
    for s in range(S):
        for h in range(hq):
            kk, vv = k[s, :, h // (hq // hkv)], v[s, :, h // (hq // hkv)]
            a = kk @ q[s, h] * D ** -0.5
            e = np.exp(a - a.max())
            want = e / e.sum() @ vv
            got = d.attended.view(S, hq, D)[s, h].double().cpu().numpy()
            # one rounding to bfloat16; values and weights in binary16 (2^-11 each, of the values' middles too); and the scores'
            # float32 sums of products with numbers of up to 1279 scales
            size = float(np.max(step[s, :, h // (hq // hkv), 0]) * np.abs(q[s, h]).sum() * 1279 * D ** -0.5)
            assert (np.abs(got - want) <= 2.0 ** -8 * np.abs(want) + (2.0 ** -9 + 2.0 ** -17 * size) * np.abs(vv).max()).all()
    logits = d.head.out.double().cpu().numpy()
    lse = np.log(np.exp(logits - logits.max(1, keepdims=True)).sum(1)) + logits.max(1)
    lp, entropy, tokens, lps = (t.cpu().numpy() for t in d.scores)
    drawn = d.tokens.cpu().numpy()
    p = np.exp(logits - lse[:, None])
    for s in range(S):
        assert abs(lp[s] - (logits[s, drawn[s]] - lse[s])) <= 2.0 ** -14
        assert abs(entropy[s] + (p[s] * np.log(p[s])).sum()) <= 2.0 ** -12
        order = np.argsort(-logits[s], kind="stable")[:7]
        assert list(tokens[s]) == list(order)
        assert (np.abs(lps[s] - (logits[s, order] - lse[s])) <= 2.0 ** -14).all()


def test_adapters_change_their_sequences_alone(example):
    """Sequences without an adapter draw what they draw in a decoder that has none."""
    import torch
    plain = example.Decoder(sequences=6, **SMALL)
    with_adapters = example.Decoder(sequences=6, adapters=2, rank=16, **SMALL)
    a, _ = plain.generate(30, graph=False)
    b, _ = with_adapters.generate(30, graph=False)
    none = with_adapters.adapter_ids == -1
    assert 0 < int(none.sum()) < 6
    assert torch.equal(a[:, none], b[:, none])
    for s in (~none).nonzero()[:, 0].tolist():
        assert not torch.equal(a[:, s], b[:, s])

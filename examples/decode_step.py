"""Decode steps of a small decoder with random weights, all of it on this library's operators but the residual norms:

    embedding -> [ norm -> q/k/v projection -> q/k norms, rotation, cache append -> attention -> output projection
                   -> norm -> gate/up projection with SwiGLU -> down projection ] x layers
              -> norm -> output head -> sampling

    python examples/decode_step.py [--sequences 8] [--steps 64] [--cache-bits 16|8|4] [--adapters N] [--top N]

With --cache-bits 8 or 4 keys and values are held as codes; with --adapters each sequence has one of N low-rank adapters beside the
q/k/v projections; with --top the log probabilities of the drawn tokens and of the N likeliest ones are computed too.

A step has no host work that depends on its data (lengths, tokens and random numbers live on the device), so it is
captured once in a CUDA graph and replayed. The cache pages of a sequence are handed out in advance.
"""
from __future__ import annotations

import argparse
import os
import sys
import time

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

import torch

import bit_affine_quantized_group_gb300 as qmm

BITS, GROUP = 4, 64


class Projection:
    """A quantized projection of random codes whose outputs keep their inputs' size."""

    def __init__(self, gen, K, N, rows, out_dtype="bf16", banks=1):
        self.plan = qmm.Plan(K, N, BITS, GROUP, max_M=rows, out_dtype=out_dtype, max_banks=banks)
        self.weights = []
        for _ in range(banks):
            words = torch.randint(-2 ** 31, 2 ** 31, (N, K * BITS // 32), generator=gen, device="cuda", dtype=torch.int32)
            scale = torch.full((N, K // GROUP), 1.0 / (4.6 * K ** 0.5), dtype=torch.float16, device="cuda")
            self.weights.append((words, scale, -7.5 * scale))   # codes 0..15 around zero
        self.out = torch.empty((rows, N), dtype=self.plan.out_dtype, device="cuda")

    def __call__(self, x):
        qmm.forward(self.plan, x, *self.weights[0], self.out)
        return self.out

    def swiglu(self, x):
        qmm.forward_swiglu(self.plan, x, *self.weights[0], *self.weights[1], self.out)
        return self.out


def rms_norm(x):
    x = x.float()
    return (x * torch.rsqrt((x * x).mean(1, keepdim=True) + 1e-6)).to(torch.bfloat16)


class Decoder:
    def __init__(self, sequences=8, layers=2, hidden=2048, q_heads=16, kv_heads=8, head_dim=128, ffn=4096, vocab=32000,
                 max_len=512, page=16, window=0, sinks=0, seed=0, cache_bits=16, adapters=0, rank=16, top=0):
        gen = torch.Generator(device="cuda").manual_seed(seed)
        S, D = sequences, head_dim
        self.cut = (q_heads * D, kv_heads * D, kv_heads * D)
        self.qkv = [Projection(gen, hidden, sum(self.cut), S) for _ in range(layers)]
        self.out = [Projection(gen, q_heads * D, hidden, S) for _ in range(layers)]
        self.up = [Projection(gen, hidden, ffn, S, banks=2) for _ in range(layers)]
        self.down = [Projection(gen, ffn, hidden, S) for _ in range(layers)]
        self.head = Projection(gen, hidden, vocab, S, out_dtype="f32")
        self.embedding = torch.randn((vocab, hidden), generator=gen, device="cuda").to(torch.bfloat16)
        self.q_weight = self.k_weight = torch.ones(D, device="cuda")
        turn = torch.arange(max_len, device="cuda")[:, None] * 10000.0 ** (-2.0 * torch.arange(D // 2, device="cuda") / D)
        self.rope = torch.cat((turn.cos(), turn.sin()), 1).float()

        pages = -(-max_len // page)
        self.kv = qmm.KVPlan(q_heads, kv_heads, D, page, max_seqs=S, max_rows=1, max_pages=pages, window=window, sinks=sinks)
        pool = lambda: torch.zeros((S * pages, kv_heads, page, D), dtype=torch.bfloat16, device="cuda")  # noqa: E731
        if cache_bits == 16:
            self.caches = [qmm.KVCache(pool(), pool()) for _ in range(layers)]
        else:
            codes = lambda: torch.zeros((S * pages, kv_heads, page, D * cache_bits // 8), dtype=torch.uint8, device="cuda")  # noqa: E731
            pairs = lambda: torch.zeros((S * pages, kv_heads, page, D // 64, 2), dtype=torch.float16, device="cuda")  # noqa: E731
            self.caches = [qmm.QuantKVCache(codes(), codes(), pairs(), pairs(), cache_bits) for _ in range(layers)]
        self.page_table = torch.randperm(S * pages, generator=gen, device="cuda").int().view(S, pages)
        self.queries = torch.empty((S, q_heads * D), dtype=torch.bfloat16, device="cuda")
        self.attended = torch.empty_like(self.queries)

        f = lambda v, t=torch.float32: torch.full((S,), v, dtype=t, device="cuda")  # noqa: E731
        self.temperature, self.top_k, self.top_p, self.min_p = f(0.8), f(40, torch.int32), f(0.95), f(0.0)
        self.uniform = torch.rand((max_len, S), generator=gen, device="cuda")
        self.tokens, self.probs, self.lengths = f(1, torch.int32), f(0.0), f(0, torch.int32)

        self.adapters = []   # (plan, A, B) of each layer's q/k/v projection
        if adapters:
            normal = lambda *s: torch.randn(s, generator=gen, device="cuda")  # noqa: E731
            for _ in range(layers):
                a, b = normal(adapters, rank, hidden) * hidden ** -0.5, normal(adapters, sum(self.cut), rank) * rank ** -0.5
                self.adapters.append((qmm.AdapterPlan(hidden, sum(self.cut), rank, adapters, S), a.to(torch.bfloat16), b.to(torch.bfloat16)))
            self.adapter_scale = torch.full((adapters,), 0.5, device="cuda")
            self.adapter_ids = torch.arange(S, device="cuda").int() % (adapters + 1) - 1   # -1: a sequence without one
        self.scores = None   # log probabilities of the drawn tokens, entropy, likeliest tokens and their log probabilities
        if top:
            self.scores = f(0.0), f(0.0), torch.zeros((S, top), dtype=torch.int32, device="cuda"), torch.zeros((S, top), device="cuda")

    def step(self):
        """Appends every sequence's last token to its cache and draws its next."""
        u = self.uniform.index_select(0, self.lengths[:1].long()).view(-1)
        self.lengths += 1
        x = self.embedding[self.tokens.long()].float()
        for i, (qkv, out, up, down, cache) in enumerate(zip(self.qkv, self.out, self.up, self.down, self.caches)):
            h = rms_norm(x)
            qkv_out = qkv(h)
            if self.adapters:
                plan, a, b = self.adapters[i]
                qmm.add_adapters(plan, h, a, b, self.adapter_scale, self.adapter_ids, qkv_out, qkv_out)
            q, k, v = qkv_out.split(self.cut, 1)
            qmm.qk_norm_rope(self.kv, q, k, v, self.q_weight, self.k_weight, self.rope, self.lengths, self.page_table,
                             cache, self.queries)
            qmm.attention(self.kv, self.queries, cache, self.page_table, self.lengths, self.attended)
            x = x + out(self.attended).float()
            x = x + down(up.swiglu(rms_norm(x))).float()
        logits = self.head(rms_norm(x))
        qmm.sample(logits, self.temperature, self.top_k, self.top_p, self.min_p, u, self.tokens, self.probs)
        if self.scores is not None:
            qmm.logprobs(logits, self.tokens, *self.scores)

    def restart(self):
        self.lengths.zero_()
        self.tokens.fill_(1)

    def generate(self, steps, graph=True):
        """The tokens [steps, sequences] that follow token 1, and the seconds that the steps took."""
        drawn = torch.empty((steps, len(self.tokens)), dtype=torch.int32, device="cuda")
        stream = torch.cuda.Stream()
        stream.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(stream):
            run = self.step
            if graph:
                self.step()   # everything is loaded before the capture
                captured = torch.cuda.CUDAGraph()
                with torch.cuda.graph(captured, stream=stream):
                    self.step()
                run = captured.replay
            self.restart()
            stream.synchronize()
            t = time.perf_counter()
            for i in range(steps):
                run()
                drawn[i].copy_(self.tokens)
            stream.synchronize()
            seconds = time.perf_counter() - t
        if self.kv.error_flags() != 0:
            raise RuntimeError("a cache operator met a bad page, length or position, or a value that is not finite")
        if any(plan.error_flags() for plan, _, _ in self.adapters):
            raise RuntimeError("a row names an adapter that is not there")
        return drawn, seconds


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--sequences", type=int, default=8)
    ap.add_argument("--steps", type=int, default=64)
    ap.add_argument("--cache-bits", type=int, default=16, choices=(16, 8, 4))
    ap.add_argument("--adapters", type=int, default=0)
    ap.add_argument("--top", type=int, default=0)
    a = ap.parse_args()
    decoder = Decoder(sequences=a.sequences, max_len=max(512, a.steps + 1), cache_bits=a.cache_bits, adapters=a.adapters, top=a.top)
    tokens, seconds = decoder.generate(a.steps)
    print(f"{a.sequences} sequences, {a.steps} steps: {seconds / a.steps * 1e6:.1f} us a step")
    print("first sequence:", tokens[:16, 0].tolist())
    if decoder.scores is not None:
        print("its last token: log probability %.3f, entropy %.3f, likeliest %s" % (
            float(decoder.scores[0][0]), float(decoder.scores[1][0]), decoder.scores[2][0].tolist()))


if __name__ == "__main__":
    main()

"""Cases of the operators that stand between two quantized projections of a decode or verification step:
`qk_norm_rope` (norms of queries and keys, rotation, append to the paged cache), `attention` (new tokens over the paged
cache) and `sample` (temperature, top-k, top-p, min-p from given random numbers).

`run` computes an operator in its plain form, or, with `own`, by the calls that a user makes. Row r of sequence s has the
cache position lengths[s] - rows + r; the lengths count the new tokens.
"""
import math
import random
from types import SimpleNamespace

import torch

own = False

EPS = 1e-6
WEIGHT_ONE = float(1 << 40)  # the fixed-point weight of the largest logit


def listed():
    return [
        # the append of one decoded token: the smallest call of a step
        dict(name="append_1x1", op="append", seqs=1, rows=1, q_heads=32, kv_heads=8, head_dim=128, page=16, min_len=700,
             max_len=700, rot=128, fused=True, interleaved=False, dtype="bf16"),
        # verification of 16 drafted tokens behind an f32 projection, 5120 wide
        dict(name="append_1x16_f32", op="append", seqs=1, rows=16, q_heads=40, kv_heads=8, head_dim=128, page=16,
             min_len=4099, max_len=4099, rot=128, fused=False, interleaved=True, dtype="f32"),
        # a serving batch of a model with wide heads that rotates a quarter of each
        dict(name="append_96x1_partial", op="append", seqs=96, rows=1, q_heads=16, kv_heads=2, head_dim=256, page=64,
             min_len=5, max_len=2500, rot=64, fused=True, interleaved=False,
             dtype="bf16"),
        # prompts of several thousand tokens written to the cache
        dict(name="append_4x2048", op="append", seqs=4, rows=2048, q_heads=32, kv_heads=8, head_dim=128, page=64,
             min_len=2048, max_len=2100, rot=128, fused=True, interleaved=False, dtype="bf16"),
        # the first tokens of a conversation
        dict(name="attn_1x1_257", op="attn", seqs=1, rows=1, q_heads=32, kv_heads=8, head_dim=128, page=16, min_len=257,
             max_len=257, window=0, sinks=0),
        # one user with a long document
        dict(name="attn_1x1_131072", op="attn", seqs=1, rows=1, q_heads=32, kv_heads=8, head_dim=128, page=16,
             min_len=131072, max_len=131072, window=0, sinks=0),
        # a serving batch with ragged lengths: the largest
        dict(name="attn_64x1_ragged", op="attn", seqs=64, rows=1, q_heads=40, kv_heads=8, head_dim=128, page=64, min_len=1,
             max_len=8191, window=0, sinks=0),
        # verification of 8 drafted tokens by four users, 8 query heads to a cache head
        dict(name="attn_4x8_verify", op="attn", seqs=4, rows=8, q_heads=32, kv_heads=4, head_dim=128, page=32, min_len=1500,
             max_len=16001, window=0, sinks=0),
        # layers with a sliding window that keep the first tokens
        dict(name="attn_24x1_window", op="attn", seqs=24, rows=1, q_heads=16, kv_heads=2, head_dim=256, page=64, min_len=90,
             max_len=20000, window=4096, sinks=4),
        # one user's next token over the repository's lm_head
        dict(name="sample_1_151936", op="sample", rows=1, vocab=151936, top_k=20, top_p=0.95, min_p=0.0, temperature=0.7,
             spread=3.0, dtype="f32"),
        # 16 verified rows of bf16 logits, cut by the largest probability and by mass
        dict(name="sample_16_bf16", op="sample", rows=16, vocab=151936, top_k=0, top_p=0.9, min_p=0.02, temperature=1.0,
             spread=2.5, dtype="bf16"),
        # a large serving batch with an odd vocabulary
        dict(name="sample_256_odd", op="sample", rows=256, vocab=100277, top_k=50, top_p=0.9, min_p=0.0, temperature=0.8,
             spread=2.0, dtype="f32"),
    ]


def _spread(rng, lo, hi):
    """A whole number between lo and hi, even over the logarithm."""
    return _uneven(max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))))


def _uneven(n):
    """n, or the next one for a multiple of 1024: a drawn length ends inside a tile or page."""
    return n + (n % 1024 == 0)


def draw(rng):
    op = rng.choice(("append", "attn", "attn", "sample"))
    if op == "sample":
        rows, vocab = _spread(rng, 1, 256), _spread(rng, 1000, 200000)
        while rows * vocab > 25_600_000:
            rows = max(1, rows // 2)
        return dict(op=op, rows=rows, vocab=vocab, top_k=rng.choice((0, 1, 20, 50, 1000)), top_p=rng.choice((1.0, 0.95, 0.8, 0.5)),
                    min_p=rng.choice((0.0, 0.0, 0.05)), temperature=rng.choice((0.0, 0.6, 0.8, 1.0, 1.3)),
                    spread=round(rng.uniform(1.0, 4.0), 2), dtype=rng.choice(("f32", "bf16")))
    head_dim = rng.choice((64, 128, 128, 256))
    kv_heads = rng.choice((1, 2, 4, 8))
    case = dict(op=op, q_heads=kv_heads * rng.choice((1, 2, 4, 5, 7, 8, 16)), kv_heads=kv_heads, head_dim=head_dim,
                page=rng.choice((16, 32, 64, 128)))
    if op == "append":
        seqs = _spread(rng, 1, 128)
        rows = _spread(rng, 1, 16) if rng.random() < 0.6 else _spread(rng, 17, 2048)
        while seqs * rows * (case["q_heads"] + 2 * kv_heads) * head_dim > 48_000_000:
            seqs, rows = (seqs // 2, rows) if seqs > 1 else (1, rows // 2)
        longest = _spread(rng, rows, rows + 2500)
        case.update(seqs=seqs, rows=rows, min_len=_uneven(rng.randint(rows, longest)), max_len=longest + 1, fused=False,
                    rot=rng.choice((head_dim, head_dim // 2, head_dim // 4)), interleaved=rng.random() < 0.4,
                    dtype=rng.choice(("bf16", "f32")))
        return case
    seqs, rows = _spread(rng, 1, 64), rng.choice((1, 1, 1, 2, 4, 5, 8, 16))
    longest = _spread(rng, 16, 131072)
    while seqs * longest * kv_heads * head_dim > 250_000_000 or seqs * longest * case["q_heads"] * rows > 150_000_000:
        seqs, longest = (seqs // 2, longest) if seqs > 1 else (1, _uneven(longest * 3 // 4))
    case.update(seqs=seqs, rows=rows, min_len=_uneven(rng.randint(rows, max(rows, longest))), max_len=max(rows, longest) + 1,
                window=rng.choice((0, 0, 128, 1000, 4096)), sinks=rng.choice((0, 4, 16)))
    return case


def _lengths(case):
    rng = random.Random("%(seqs)d %(min_len)d %(max_len)d" % case)
    n = [rng.randint(case["min_len"], case["max_len"]) for _ in range(case["seqs"])]
    n[-1] = case["max_len"]
    return n


def _seen(case):
    """Positions of each sequence that at least one of its rows sees."""
    n = []
    for length in _lengths(case):
        low = max(0, length - case["rows"] - case["window"] + 1) if case["window"] else 0
        n.append(length - max(0, low - case["sinks"]))
    return n


def work(case):
    if case["op"] == "sample":
        size = 4 if case["dtype"] == "f32" else 2
        return {"bytes": case["rows"] * (case["vocab"] * size + 5 * 4 + 8), "flops": 6 * case["rows"] * case["vocab"]}
    tokens, d = case["seqs"] * case["rows"], case["head_dim"]
    if case["op"] == "append":
        size = 4 if case["dtype"] == "f32" else 2
        heads = case["q_heads"] + 2 * case["kv_heads"]
        return {"bytes": tokens * (heads * d * (size + 2) + 4 * case["rot"]) + 8 * d + 8 * case["seqs"],
                "flops": tokens * (8 * (case["q_heads"] + case["kv_heads"]) * d)}
    seen = sum(_seen(case))
    return {"bytes": seen * case["kv_heads"] * d * 4 + tokens * case["q_heads"] * d * 4 + seen // case["page"] * 4,
            "flops": 4 * seen * case["rows"] * case["q_heads"] * d}


def _rope_table(positions, rot):
    """cos and sin of every position, in one row of rot floats: a user's program makes it once."""
    i = torch.arange(rot // 2, device="cuda", dtype=torch.float64)
    a = torch.arange(positions, device="cuda", dtype=torch.float64)[:, None] * 10000.0 ** (-2.0 * i / rot)
    return torch.cat((a.cos(), a.sin()), 1).float()


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    normal = lambda *shape, dtype=torch.float32: torch.randn(shape, generator=g, device="cuda", dtype=dtype)  # noqa: E731
    s = SimpleNamespace(case=case)
    if case["op"] == "sample":
        rows, vocab = case["rows"], case["vocab"]
        s.logits = normal(rows, vocab) * case["spread"]
        # a few likely tokens stand out of the rest, as they do behind a trained model
        at = torch.randint(vocab, (rows, 30), generator=g, device="cuda")
        s.logits.scatter_add_(1, at, 3.0 * case["spread"] + normal(rows, 30).abs() * case["spread"])
        s.logits = s.logits.to(torch.float32 if case["dtype"] == "f32" else torch.bfloat16)
        full = lambda v, t: torch.full((rows,), v, dtype=t, device="cuda")  # noqa: E731
        s.temperature, s.top_k = full(case["temperature"], torch.float32), full(case["top_k"], torch.int32)
        s.top_p, s.min_p = full(case["top_p"], torch.float32), full(case["min_p"], torch.float32)
        s.u = torch.rand(rows, generator=g, device="cuda")
        if own:
            s.tokens = torch.empty(rows, dtype=torch.int32, device="cuda")
            s.probs = torch.empty(rows, dtype=torch.float32, device="cuda")
        return s
    seqs, rows, d, page = case["seqs"], case["rows"], case["head_dim"], case["page"]
    tokens, hq, hkv = seqs * rows, case["q_heads"], case["kv_heads"]
    lengths = _lengths(case)
    used = [-(-n // page) for n in lengths]
    s.max_pages, pages = max(used), sum(used)
    order = torch.randperm(pages, generator=g, device="cuda").int()
    s.page_table = torch.full((seqs, s.max_pages), -1, dtype=torch.int32, device="cuda")
    at = 0
    for i, n in enumerate(used):
        s.page_table[i, :n] = order[at:at + n]
        at += n
    s.lengths = torch.tensor(lengths, dtype=torch.int32, device="cuda")
    s.k_cache = normal(pages, hkv, page, d, dtype=torch.bfloat16)
    s.v_cache = normal(pages, hkv, page, d, dtype=torch.bfloat16)
    if case["op"] == "append":
        dtype = torch.float32 if case["dtype"] == "f32" else torch.bfloat16
        if case["fused"]:  # one projection's output: queries, keys and values side by side in a row
            qkv = normal(tokens, (hq + 2 * hkv) * d).to(dtype)
            s.q, s.k, s.v = qkv[:, :hq * d], qkv[:, hq * d:(hq + hkv) * d], qkv[:, (hq + hkv) * d:]
        else:
            s.q, s.k, s.v = (normal(tokens, h * d).to(dtype) for h in (hq, hkv, hkv))
        s.q_weight, s.k_weight = 1 + 0.1 * normal(d), 1 + 0.1 * normal(d)
        s.rope = _rope_table(max(lengths), case["rot"])
    else:
        s.q = 1.5 * normal(tokens, hq, d)
        s.q = s.q.to(torch.bfloat16)
    if own:
        import bit_affine_quantized_group_gb300 as qmm
        s.qmm = qmm
        attn = case["op"] == "attn"
        s.plan = qmm.KVPlan(q_heads=hq, kv_heads=hkv, head_dim=d, page_size=page, max_seqs=seqs, max_rows=rows if attn else 1,
                            max_pages=s.max_pages, window=case["window"] if attn else 0, sinks=case["sinks"] if attn else 0,
                            rot_dim=d if attn else case["rot"], interleaved=False if attn else case["interleaved"], eps=EPS)
        s.cache = qmm.KVCache(s.k_cache, s.v_cache)
        s.out = torch.empty((tokens, hq, d), dtype=torch.bfloat16, device="cuda")
    return s


def run(state):
    op = state.case["op"]
    if own:
        if op == "sample":
            import bit_affine_quantized_group_gb300 as qmm
            qmm.sample(state.logits, state.temperature, state.top_k, state.top_p, state.min_p, state.u, state.tokens, state.probs)
            return {"tokens": state.tokens, "probs": state.probs}
        if op == "append":
            state.qmm.qk_norm_rope(state.plan, state.q, state.k, state.v, state.q_weight, state.k_weight, state.rope,
                                   state.lengths, state.page_table, state.cache, state.out)
            return {"q": state.out, "k_cache": state.k_cache, "v_cache": state.v_cache}
        state.qmm.attention(state.plan, state.q, state.cache, state.page_table, state.lengths, state.out)
        return {"out": state.out}
    return {"sample": _plain_sample, "append": _plain_append, "attn": _plain_attention}[op](state)


def _positions(s):
    rows = s.case["rows"]
    return s.lengths[:, None] - rows + torch.arange(rows, device="cuda")


def _plain_append(s):
    c, d = s.case, s.case["head_dim"]
    pos = _positions(s).long()
    cos, sin = s.rope[pos.reshape(-1)][:, None, :].chunk(2, 2)

    def norm_rotate(x, weight):
        x = x.float().view(x.shape[0], -1, d)
        x = x * torch.rsqrt((x * x).mean(2, keepdim=True) + EPS) * weight
        r, rest = x[..., :c["rot"]], x[..., c["rot"]:]
        if c["interleaved"]:
            a, b = r[..., 0::2], r[..., 1::2]
            r = torch.stack((a * cos - b * sin, b * cos + a * sin), 3).flatten(2)
        else:
            a, b = r.chunk(2, 2)
            r = torch.cat((a * cos - b * sin, b * cos + a * sin), 2)
        return torch.cat((r, rest), 2).to(torch.bfloat16)

    page = s.page_table.long().gather(1, pos // c["page"]).view(-1)
    slot = (pos % c["page"]).view(-1)
    s.k_cache[page, :, slot] = norm_rotate(s.k, s.k_weight)
    s.v_cache[page, :, slot] = s.v.reshape(len(page), -1, d).to(torch.bfloat16)
    return {"q": norm_rotate(s.q, s.q_weight), "k_cache": s.k_cache, "v_cache": s.v_cache}


def _visible(c, pos, j):
    """Which of the positions j a row at pos sees."""
    seen = j <= pos
    if c["window"]:
        seen = seen & ((pos - j < c["window"]) | (j < c["sinks"]))
    return seen


def _plain_attention(s):
    c, d, hkv = s.case, s.case["head_dim"], s.case["kv_heads"]
    seqs, rows = c["seqs"], c["rows"]
    group = c["q_heads"] // hkv
    table = s.page_table.clamp(min=0).long()
    k = s.k_cache[table].float().transpose(1, 2).reshape(seqs, hkv, -1, d)
    v = s.v_cache[table].float().transpose(1, 2).reshape(seqs, hkv, -1, d)
    q = s.q.float().view(seqs, rows, hkv, group, d).transpose(1, 2).reshape(seqs, hkv, rows * group, d)
    scores = (q @ k.transpose(2, 3) * d ** -0.5).view(seqs, hkv, rows, group, -1)
    seen = _visible(c, _positions(s)[:, None, :, None, None], torch.arange(k.shape[2], device="cuda"))
    scores = torch.where(seen, scores, float("-inf"))
    e = torch.exp(scores - scores.amax(4, keepdim=True).clamp(min=-3e38))
    e = e / e.sum(4, keepdim=True).clamp(min=1e-38)
    out = e.view(seqs, hkv, rows * group, -1) @ v
    out = out.view(seqs, hkv, rows, group, d).transpose(1, 2).reshape(seqs * rows, c["q_heads"], d)
    return {"out": out.to(torch.bfloat16)}


def _plain_sample(s):
    l = s.logits.float()
    l = torch.where(torch.isnan(l), float("-inf"), l)
    vocab = l.shape[1]
    l, index = l.sort(dim=1, descending=True, stable=True)
    rank = torch.arange(vocab, device="cuda")[None]
    greedy = ~(s.temperature > 0)[:, None]
    z = (l - l[:, :1]) / torch.where(greedy, 1.0, s.temperature[:, None])
    w = torch.where(l == l[:, :1], 1.0, torch.exp(z))
    w = torch.where(l == float("-inf"), 0.0, w)
    mass = (w * WEIGHT_ONE).long()
    k = s.top_k[:, None]
    mass = torch.where((k <= 0) | (rank < k), mass, 0)
    before = mass.cumsum(1) - mass
    p = s.top_p[:, None].double()
    keep = ~(p < 1) | (before.double() < p * mass.sum(1, keepdim=True).double())
    keep = (keep & ~(w < s.min_p[:, None]) & ~greedy) | (rank == 0)
    kept = torch.zeros_like(mass).scatter_(1, index, torch.where(keep, mass, 0))
    up_to = kept.cumsum(1)
    total = up_to[:, -1:]
    target = (s.u[:, None].double() * total.double()).long().minimum(total - 1).clamp(min=0)
    token = (up_to <= target).sum(1, keepdim=True)
    some = total > 0
    prob = kept.gather(1, token.clamp(max=vocab - 1)).float() / total.clamp(min=1).float()
    return {"tokens": torch.where(some, token, -1).int().view(-1), "probs": torch.where(some, prob, 0.0).view(-1)}


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "sample":
        return {"tokens": None, "probs": _exact_sample(s)}
    if case["op"] == "append":
        return _exact_append(s)
    c, d, hkv = case, case["head_dim"], case["kv_heads"]
    group, outs = c["q_heads"] // hkv, []
    for i, n in enumerate(_lengths(c)):
        j = torch.arange(n, device="cuda")
        first = n - c["rows"]
        if c["window"]:  # what no row sees is left out
            j = j[(j < c["sinks"]) | (j > first - c["window"])]
        page, slot = s.page_table[i].long()[j // c["page"]], j % c["page"]
        k, v = s.k_cache[page, :, slot].double(), s.v_cache[page, :, slot].double()
        q = s.q.view(c["seqs"], c["rows"], hkv, group, d)[i].double()
        a = torch.einsum("rhgd,jhd->rhgj", q, k) / math.sqrt(d)
        pos = first + torch.arange(c["rows"], device="cuda")
        seen = j[None] <= pos[:, None]
        if c["window"]:
            seen &= (j[None] > pos[:, None] - c["window"]) | (j[None] < c["sinks"])
        a = torch.softmax(a.masked_fill(~seen[:, None, None], float("-inf")), 3)
        outs.append(torch.einsum("rhgj,jhd->rhgd", a, v).reshape(c["rows"], c["q_heads"], d))
    return {"out": torch.cat(outs)}


def _exact_append(s):
    c, d = s.case, s.case["head_dim"]
    half = c["rot"] // 2
    pos = torch.cat([torch.arange(n - c["rows"], n, device="cuda") for n in _lengths(c)])
    turn = torch.complex(s.rope[pos, :half].double(), s.rope[pos, half:].double())[:, None]

    def one(x, weight):
        x = x.double().reshape(len(pos), -1, d)
        x = x / torch.sqrt(x.square().sum(2, keepdim=True) / d + EPS) * weight.double()
        if c["interleaved"]:
            y = torch.view_as_complex(x[..., :c["rot"]].reshape(*x.shape[:2], half, 2)) * turn
            x[..., :c["rot"]] = torch.view_as_real(y).flatten(2)
        else:
            y = torch.complex(x[..., :half], x[..., half:c["rot"]].clone()) * turn
            x[..., :half], x[..., half:c["rot"]] = y.real, y.imag
        return x

    seq = torch.arange(c["seqs"], device="cuda").repeat_interleave(c["rows"])
    page, slot = s.page_table[seq, pos // c["page"]].long(), pos % c["page"]
    k, v = s.k_cache.double(), s.v_cache.double()
    k[page, :, slot] = one(s.k, s.k_weight)
    v[page, :, slot] = s.v.double().reshape(len(pos), -1, d)
    return {"q": one(s.q, s.q_weight), "k_cache": k, "v_cache": v}


def _exact_sample(s):
    c, l = s.case, s.logits.double()
    if c["temperature"] <= 0:
        return torch.ones(c["rows"], dtype=torch.float64, device="cuda")
    p, index = torch.softmax(l / float(s.temperature[0]), 1).sort(dim=1, descending=True, stable=True)
    if c["top_k"] > 0:
        p[:, c["top_k"]:] = 0
        p = p / p.sum(1, keepdim=True)
    top = p[:, :1].clone()
    if c["top_p"] < 1:
        p[p.cumsum(1) - p >= float(s.top_p[0])] = 0
    p[p < float(s.min_p[0]) * top] = 0
    p = torch.zeros_like(p).scatter_(1, index, p)
    up_to = p.cumsum(1)
    token = torch.searchsorted(up_to, s.u[:, None].double() * up_to[:, -1:], right=True)
    return (p.gather(1, token) / up_to[:, -1:]).view(-1)

"""Cases of the operators that serve many requests around the quantized projections: `append` (norms, rotation and append to
a cache of 8- or 4-bit codes, then the read-back of the sequences), `read` (the read-back alone), `attn` (new tokens over
such a cache), `adapter` (low-rank adapters of many requests beside a projection) and `logprobs` (log probabilities of given
tokens, entropy and top alternatives).

`run` computes an operator in its plain form, or, with `own`, by the calls that a user makes. A cache holds each 64 elements
of a head as codes c with a binary16 scale s and bias b, and stands for s c + b. Row r of sequence s has the cache position
lengths[s] - rows + r; the lengths count the new tokens.
"""
import math
import random
from types import SimpleNamespace

import torch

own = False

EPS = 1e-6
GROUP = 64           # elements of a head that share a scale and a bias
LARGEST = 65280.0    # what a cache of codes holds at most: larger values are brought to it


def listed():
    return [
        # one decoded token of a short conversation: the smallest call
        dict(name="append_q8_1x1", op="append", seqs=1, rows=1, q_heads=32, kv_heads=8, head_dim=128, page=16, min_len=257,
             max_len=257, rot=128, fused=True, interleaved=False, dtype="bf16", bits=8),
        # prompts written to the cache, and read back as dense keys and values for the prompt's own attention
        dict(name="append_q8_4x2048", op="append", seqs=4, rows=2048, q_heads=32, kv_heads=8, head_dim=128, page=64,
             min_len=2048, max_len=2100, rot=128, fused=True, interleaved=False, dtype="bf16", bits=8),
        # the last part of two short sequences
        dict(name="read_q4_2x100", op="read", seqs=2, head_dim=256, kv_heads=2, page=16, min_len=700, max_len=913, start=813,
             bits=4, dtype="f32"),
        # a batch of ragged sequences that moves elsewhere
        dict(name="read_q8_16_ragged", op="read", seqs=16, head_dim=128, kv_heads=8, page=64, min_len=1, max_len=8191, start=0,
             bits=8, dtype="bf16"),
        # the first tokens of a conversation
        dict(name="attn_q8_1x1_257", op="attn", seqs=1, rows=1, q_heads=32, kv_heads=8, head_dim=128, page=16, min_len=257,
             max_len=257, window=0, sinks=0, bits=8),
        # one user with a long document, in the smallest codes
        dict(name="attn_q4_1x1_131072", op="attn", seqs=1, rows=1, q_heads=32, kv_heads=8, head_dim=128, page=16,
             min_len=131072, max_len=131072, window=0, sinks=0, bits=4),
        # a serving batch with ragged lengths
        dict(name="attn_q8_64x1_ragged", op="attn", seqs=64, rows=1, q_heads=40, kv_heads=8, head_dim=128, page=64, min_len=1,
             max_len=8191, window=0, sinks=0, bits=8),
        # a decode step of 16 requests, each with an adapter of its own
        dict(name="adapter_16x1", op="adapter", rows=16, run=1, adapters=16, rank=16, K=4096, N=6144, dtype="bf16"),
        # four rows to verify of each of 16 requests, wide adapters beside the up-projection
        dict(name="adapter_16x4_wide", op="adapter", rows=64, run=4, adapters=32, rank=64, K=5120, N=17408, dtype="f32"),
        # prompts of four requests
        dict(name="adapter_4x512", op="adapter", rows=2048, run=512, adapters=8, rank=32, K=5120, N=6144, dtype="bf16"),
        # one user's token over the repository's lm_head
        dict(name="logprobs_1", op="logprobs", rows=1, vocab=151936, top=5, spread=3.0, dtype="f32"),
        # a prompt that is scored, with an odd vocabulary
        dict(name="logprobs_512_odd", op="logprobs", rows=512, vocab=100277, top=20, spread=2.0, dtype="bf16"),
    ]


def _spread(rng, lo, hi):
    """A whole number between lo and hi, even over the logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("append", "read", "attn", "attn", "adapter", "logprobs"))
    if op == "logprobs":
        rows, vocab = _spread(rng, 1, 700), _spread(rng, 1000, 200000)
        while rows * vocab > 40_000_000:
            rows = max(1, rows // 2)
        return dict(op=op, rows=rows, vocab=vocab, top=rng.choice((0, 1, 5, 20, 32)), spread=round(rng.uniform(1.0, 3.5), 2),
                    dtype=rng.choice(("f32", "bf16")))
    if op == "adapter":
        rows, rank = _spread(rng, 1, 2048), rng.choice((8, 16, 16, 32, 64, 128))
        K, N = 64 * _spread(rng, 8, 128), _spread(rng, 256, 17408)
        while rows * (K + N) > 30_000_000:
            rows //= 2
        adapters = _spread(rng, 1, 64)
        while adapters * rank * (K + N) > 50_000_000 or rows * adapters * rank * (K + N) > 10_000_000_000:
            adapters = max(1, adapters // 2)
            rank = max(8, rank // 2) if adapters == 1 else rank
        return dict(op=op, rows=rows, run=min(rows, rng.choice((1, 1, 2, 5, 8, 100, 600))), adapters=adapters, rank=rank, K=K, N=N,
                    dtype=rng.choice(("f32", "bf16")))
    head_dim = rng.choice((64, 128, 128, 256))
    kv_heads = rng.choice((1, 2, 4, 8))
    case = dict(op=op, bits=rng.choice((8, 8, 4)), kv_heads=kv_heads, head_dim=head_dim, page=rng.choice((16, 32, 64, 128)))
    if op == "read":
        seqs, longest = _spread(rng, 1, 64), _spread(rng, 2, 32768)
        while seqs * longest * kv_heads * head_dim > 60_000_000:
            seqs, longest = (seqs // 2, longest) if seqs > 1 else (1, longest // 2)
        case.update(seqs=seqs, min_len=rng.randint(1, longest), max_len=longest, start=rng.choice((0, longest // 3)),
                    dtype=rng.choice(("f32", "bf16")))
        return case
    case["q_heads"] = kv_heads * rng.choice((1, 2, 4, 5, 7, 8, 16))
    if op == "append":
        seqs = _spread(rng, 1, 128)
        rows = _spread(rng, 1, 16) if rng.random() < 0.6 else _spread(rng, 17, 2048)
        while seqs * rows * (case["q_heads"] + 2 * kv_heads) * head_dim > 48_000_000 or \
                (case["bits"] == 4 and seqs * rows * kv_heads * head_dim > 1_000_000):
            seqs, rows = (seqs // 2, rows) if seqs > 1 else (1, rows // 2)
        longest = _spread(rng, rows, rows + 300)
        case.update(seqs=seqs, rows=rows, min_len=rng.randint(rows, longest), max_len=longest + 1, fused=False,
                    rot=rng.choice((head_dim, head_dim // 2, head_dim // 4)), interleaved=rng.random() < 0.4,
                    dtype=rng.choice(("bf16", "f32")))
        return case
    seqs, rows = _spread(rng, 1, 64), rng.choice((1, 1, 1, 2, 4, 5, 8, 16))
    longest = _spread(rng, 16, 131072)
    while seqs * longest * kv_heads * head_dim > 250_000_000 or seqs * longest * case["q_heads"] * rows > 150_000_000:
        seqs, longest = (seqs // 2, longest) if seqs > 1 else (1, longest * 3 // 4)
    case.update(seqs=seqs, rows=rows, min_len=rng.randint(rows, max(rows, longest)), max_len=max(rows, longest) + 1,
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


def _ids(case):
    """Adapters of the rows: one for each run of rows, now and then none."""
    rng = random.Random("%(rows)d %(run)d %(adapters)d" % case)
    runs = -(-case["rows"] // case["run"])
    of_run = [i % case["adapters"] for i in range(runs)]
    rng.shuffle(of_run)
    for i in range(7, runs, 16):
        of_run[i] = -1
    return [of_run[m // case["run"]] for m in range(case["rows"])]


def work(case):
    if case["op"] == "logprobs":
        size = 4 if case["dtype"] == "f32" else 2
        return {"bytes": case["rows"] * (case["vocab"] * size + 12 + 8 * case["top"]), "flops": 5 * case["rows"] * case["vocab"]}
    if case["op"] == "adapter":
        ids = _ids(case)
        size = 4 if case["dtype"] == "f32" else 2
        used, rows = len(set(ids) - {-1}), sum(i >= 0 for i in ids)
        return {"bytes": used * case["rank"] * (case["K"] + case["N"]) * 2 + rows * case["K"] * 2 + case["rows"] * (case["N"] * 2 * size + 4),
                "flops": 2 * rows * case["rank"] * (case["K"] + case["N"])}
    d, kv = case["head_dim"], case["kv_heads"]
    position = 2 * kv * (d * case["bits"] // 8 + 4 * d // GROUP)   # bytes of a position's keys and values
    if case["op"] == "read":
        n = sum(max(0, length - case["start"]) for length in _lengths(case))
        return {"bytes": n * (position + 2 * kv * d * (4 if case["dtype"] == "f32" else 2)), "flops": n * 4 * kv * d}
    tokens = case["seqs"] * case["rows"]
    if case["op"] == "append":
        size, n = 4 if case["dtype"] == "f32" else 2, sum(_lengths(case))
        heads = case["q_heads"] + 2 * kv
        return {"bytes": tokens * (heads * d * size + case["q_heads"] * d * 2 + position + 4 * case["rot"]) + n * (position + 4 * kv * d),
                "flops": tokens * (8 * (case["q_heads"] + kv) * d + 12 * kv * d) + n * 4 * kv * d}
    seen = sum(_seen(case))
    return {"bytes": seen * position + tokens * case["q_heads"] * d * 4 + seen // case["page"] * 4,
            "flops": 4 * seen * case["rows"] * case["q_heads"] * d}


def _rope_table(positions, rot):
    """cos and sin of every position, in one row of rot floats: a user's program makes it once."""
    i = torch.arange(rot // 2, device="cuda", dtype=torch.float64)
    a = torch.arange(positions, device="cuda", dtype=torch.float64)[:, None] * 10000.0 ** (-2.0 * i / rot)
    return torch.cat((a.cos(), a.sin()), 1).float()


def _quantise(x, bits):
    """Codes, and scales with biases, of values [..., head_dim] in 32 or 64 bits."""
    top = 2 ** bits - 1
    x = x.clamp(-LARGEST, LARGEST).unflatten(-1, (-1, GROUP))
    low, high = x.amin(-1, keepdim=True), x.amax(-1, keepdim=True)
    bias, scale = low.half(), ((high - low) / top).half()
    wide = scale.to(x.dtype)
    code = torch.round((x - bias.to(x.dtype)) * (1 / wide)).clamp(0, top)
    code = torch.where(wide > 0, code, 0).to(torch.uint8).flatten(-2)
    if bits == 4:
        code = code[..., 0::2] | code[..., 1::2] << 4
    return code, torch.cat((scale, bias), -1)


def _values(code, affine, bits, dtype=torch.float32):
    """What codes [..., head_dim * bits / 8] with scales and biases [..., head_dim / 64, 2] stand for."""
    if bits == 4:
        code = torch.stack((code & 15, code >> 4), -1).flatten(-2)
    a = affine.to(dtype)
    return (code.unflatten(-1, (-1, GROUP)).to(dtype) * a[..., :1] + a[..., 1:]).flatten(-2)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    normal = lambda *shape, dtype=torch.float32: torch.randn(shape, generator=g, device="cuda", dtype=dtype)  # noqa: E731
    s = SimpleNamespace(case=case)
    dtype = torch.float32 if case.get("dtype") == "f32" else torch.bfloat16
    if own:
        import bit_affine_quantized_group_gb300 as qmm
        s.qmm = qmm
    if case["op"] == "logprobs":
        rows, vocab, top = case["rows"], case["vocab"], case["top"]
        s.logits = normal(rows, vocab) * case["spread"]
        # a few likely tokens stand out of the rest, as they do behind a trained model, and are often the given ones
        at = torch.randint(vocab, (rows, 1), generator=g, device="cuda") + torch.arange(30, device="cuda") * (vocab // 31)
        at = at % vocab
        s.logits.scatter_add_(1, at, 3.0 * case["spread"] + normal(rows, 30).abs() * case["spread"])
        s.logits = s.logits.to(dtype)
        other = torch.randint(vocab, (rows,), generator=g, device="cuda")
        s.tokens = torch.where(torch.rand(rows, generator=g, device="cuda") < 0.7, at[:, 0], other).int()
        s.token_logprobs, s.entropy = torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")
        s.top_tokens = torch.empty((rows, top), dtype=torch.int32, device="cuda") if top else None
        s.top_logprobs = torch.empty((rows, top), device="cuda") if top else None
        return s
    if case["op"] == "adapter":
        rows, K, N, rank, n = case["rows"], case["K"], case["N"], case["rank"], case["adapters"]
        s.x = normal(rows, K).to(torch.bfloat16)
        s.y = normal(rows, N).to(dtype)   # the shared projection's result
        s.a = (normal(n, rank, K) * K ** -0.5).to(torch.bfloat16)
        s.b = (normal(n, N, rank) * rank ** -0.5).to(torch.bfloat16)
        s.scale = 0.5 + torch.rand(n, generator=g, device="cuda")
        s.ids = torch.tensor(_ids(case), dtype=torch.int32, device="cuda")
        s.out = torch.empty_like(s.y)
        if own:
            s.plan = s.qmm.AdapterPlan(K, N, rank, adapters=n, max_rows=rows, out_dtype=dtype)
        return s
    d, page, seqs, hkv, bits = case["head_dim"], case["page"], case["seqs"], case["kv_heads"], case["bits"]
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
    s.k, s.k_affine = _quantise(normal(pages, hkv, page, d), bits)
    s.v, s.v_affine = _quantise(normal(pages, hkv, page, d), bits)
    hq, rows = case.get("q_heads", hkv), case.get("rows", 1)
    tokens = seqs * rows
    if case["op"] == "append":
        if case["fused"]:  # one projection's output: queries, keys and values side by side in a row
            qkv = normal(tokens, (hq + 2 * hkv) * d).to(dtype)
            s.new_q, s.new_k, s.new_v = qkv[:, :hq * d], qkv[:, hq * d:(hq + hkv) * d], qkv[:, (hq + hkv) * d:]
        else:
            s.new_q, s.new_k, s.new_v = (normal(tokens, h * d).to(dtype) for h in (hq, hkv, hkv))
        s.q_weight, s.k_weight = 1 + 0.1 * normal(d), 1 + 0.1 * normal(d)
        s.rope = _rope_table(max(lengths), case["rot"])
    if case["op"] == "attn":
        s.q = (1.5 * normal(tokens, hq, d)).to(torch.bfloat16)
    else:   # dense keys and values; rows behind a sequence's end stay zero
        start = case.get("start", 0)
        s.starts = torch.full((seqs,), start, dtype=torch.int32, device="cuda")
        out = torch.bfloat16 if case["op"] == "append" else dtype
        s.k_out, s.v_out = (torch.zeros((seqs, max(lengths) - start, hkv, d), dtype=out, device="cuda") for _ in range(2))
    s.out = torch.empty((tokens, hq, d), dtype=torch.bfloat16, device="cuda")
    if own:
        attn = case["op"] == "attn"
        s.plan = s.qmm.KVPlan(q_heads=hq, kv_heads=hkv, head_dim=d, page_size=page, max_seqs=seqs, max_rows=rows if attn else 1,
                              max_pages=s.max_pages, window=case.get("window", 0), sinks=case.get("sinks", 0),
                              rot_dim=case.get("rot", d), interleaved=case.get("interleaved", False), eps=EPS)
        s.cache = s.qmm.QuantKVCache(s.k, s.v, s.k_affine, s.v_affine, bits)
    return s


def run(state):
    s, op = state, state.case["op"]
    if not own:
        return {"append": _plain_append, "read": _plain_read, "attn": _plain_attention, "adapter": _plain_adapter,
                "logprobs": _plain_logprobs}[op](s)
    if op == "logprobs":
        s.qmm.logprobs(s.logits, s.tokens, s.token_logprobs, s.entropy, s.top_tokens, s.top_logprobs)
        return _scores(s.token_logprobs, s.entropy, s.top_tokens, s.top_logprobs)
    if op == "adapter":
        s.qmm.add_adapters(s.plan, s.x, s.a, s.b, s.scale, s.ids, s.y, s.out)
        return {"out": s.out}
    if op == "attn":
        s.qmm.attention(s.plan, s.q, s.cache, s.page_table, s.lengths, s.out)
        return {"out": s.out}
    if op == "append":
        s.qmm.qk_norm_rope(s.plan, s.new_q, s.new_k, s.new_v, s.q_weight, s.k_weight, s.rope, s.lengths, s.page_table,
                           s.cache, s.out)
    s.qmm.kv_read(s.plan, s.cache, s.page_table, s.lengths, s.k_out, s.v_out, s.starts)
    return {"q": s.out, "k": s.k_out, "v": s.v_out} if op == "append" else {"k": s.k_out, "v": s.v_out}


def _scores(token_logprobs, entropy, top_tokens, top_logprobs):
    out = {"token_logprobs": token_logprobs, "entropy": entropy}
    if top_tokens is not None:
        out.update(top_tokens=top_tokens, top_logprobs=top_logprobs)
    return out


def _positions(s):
    rows = s.case["rows"]
    return s.lengths[:, None] - rows + torch.arange(rows, device="cuda")


def _norm_rotate(s, x, weight):
    c, d = s.case, s.case["head_dim"]
    cos, sin = s.rope[_positions(s).long().reshape(-1)][:, None, :].chunk(2, 2)
    x = x.float().view(x.shape[0], -1, d)
    x = x * torch.rsqrt((x * x).mean(2, keepdim=True) + EPS) * weight
    r, rest = x[..., :c["rot"]], x[..., c["rot"]:]
    if c["interleaved"]:
        a, b = r[..., 0::2], r[..., 1::2]
        r = torch.stack((a * cos - b * sin, b * cos + a * sin), 3).flatten(2)
    else:
        a, b = r.chunk(2, 2)
        r = torch.cat((a * cos - b * sin, b * cos + a * sin), 2)
    return torch.cat((r, rest), 2)


def _plain_append(s):
    c, d = s.case, s.case["head_dim"]
    pos = _positions(s).long()
    page = s.page_table.long().gather(1, pos // c["page"]).view(-1)
    slot = (pos % c["page"]).view(-1)
    s.k[page, :, slot], s.k_affine[page, :, slot] = _quantise(_norm_rotate(s, s.new_k, s.k_weight), c["bits"])
    s.v[page, :, slot], s.v_affine[page, :, slot] = _quantise(s.new_v.float().reshape(len(page), -1, d), c["bits"])
    return {"q": _norm_rotate(s, s.new_q, s.q_weight).to(torch.bfloat16), **_plain_read(s)}


def _plain_read(s):
    c = s.case
    pos = s.starts[:, None].long() + torch.arange(s.k_out.shape[1], device="cuda")
    some = pos < s.lengths[:, None]
    page = s.page_table.long().gather(1, torch.where(some, pos, 0) // c["page"]).clamp(min=0)
    slot = pos % c["page"]
    k = _values(s.k[page, :, slot], s.k_affine[page, :, slot], c["bits"])
    v = _values(s.v[page, :, slot], s.v_affine[page, :, slot], c["bits"])
    some = some[..., None, None]
    s.k_out.copy_(torch.where(some, k.to(s.k_out.dtype), s.k_out))
    s.v_out.copy_(torch.where(some, v.to(s.v_out.dtype), s.v_out))
    return {"k": s.k_out, "v": s.v_out}


def _plain_attention(s):
    c, d, hkv = s.case, s.case["head_dim"], s.case["kv_heads"]
    seqs, rows = c["seqs"], c["rows"]
    group = c["q_heads"] // hkv
    table = s.page_table.clamp(min=0).long()
    k = _values(s.k[table], s.k_affine[table], c["bits"]).transpose(1, 2).reshape(seqs, hkv, -1, d)
    v = _values(s.v[table], s.v_affine[table], c["bits"]).transpose(1, 2).reshape(seqs, hkv, -1, d)
    q = s.q.float().view(seqs, rows, hkv, group, d).transpose(1, 2).reshape(seqs, hkv, rows * group, d)
    scores = (q @ k.transpose(2, 3) * d ** -0.5).view(seqs, hkv, rows, group, -1)
    pos, j = _positions(s)[:, None, :, None, None], torch.arange(k.shape[2], device="cuda")
    seen = j <= pos
    if c["window"]:
        seen = seen & ((pos - j < c["window"]) | (j < c["sinks"]))
    scores = torch.where(seen, scores, float("-inf"))
    e = torch.exp(scores - scores.amax(4, keepdim=True).clamp(min=-3e38))
    e = e / e.sum(4, keepdim=True).clamp(min=1e-38)
    out = e.view(seqs, hkv, rows * group, -1) @ v
    out = out.view(seqs, hkv, rows, group, d).transpose(1, 2).reshape(seqs * rows, c["q_heads"], d)
    return {"out": out.to(torch.bfloat16)}


def _plain_adapter(s):
    n, rank, K = s.a.shape
    mine = s.ids[:, None] == torch.arange(n, device="cuda")
    low = (s.x.float() @ s.a.float().view(n * rank, K).T).view(-1, n, rank) * s.scale[:, None]
    low = torch.where(mine[:, :, None], low, 0).view(-1, n * rank)   # the row's own adapter alone
    up = s.b.float().transpose(1, 2).reshape(n * rank, -1)
    s.out.copy_(s.y.float() + low @ up)
    return {"out": s.out}


def _plain_logprobs(s):
    l = s.logits.float()
    l = torch.where(torch.isnan(l), float("-inf"), l)
    below = l - l.amax(1, keepdim=True)
    w = torch.exp(below)
    total = w.sum(1, keepdim=True)
    log_total = torch.log(total)
    entropy = log_total[:, 0] - torch.where(w > 0, w * below, 0).sum(1) / total[:, 0]
    given = below.gather(1, s.tokens[:, None].long()) - log_total
    if s.top_tokens is None:
        return _scores(given[:, 0], entropy, None, None)
    below, index = below.sort(dim=1, descending=True, stable=True)
    top = s.top_tokens.shape[1]
    return _scores(given[:, 0], entropy, index[:, :top].int(), below[:, :top] - log_total)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "logprobs":
        p = torch.log_softmax(s.logits.double(), 1)
        best, index = p.sort(dim=1, descending=True, stable=True)
        entropy = -(p.exp() * p).sum(1)
        some = case["top"] > 0
        return _scores(p[torch.arange(case["rows"], device="cuda"), s.tokens.long()], entropy,
                       index[:, :case["top"]].int() if some else None, best[:, :case["top"]] if some else None)
    if case["op"] == "adapter":
        out = s.y.double()
        for i in range(case["adapters"]):
            rows = (s.ids == i).nonzero()[:, 0]
            if len(rows):
                low = torch.einsum("mk,rk->mr", s.x[rows].double(), s.a[i].double()) * float(s.scale[i])
                out[rows] += torch.einsum("mr,nr->mn", low, s.b[i].double())
        return {"out": out}
    if case["op"] == "append":
        return _exact_append(s)
    if case["op"] == "read":
        return _exact_read(s)
    c, d, hkv = case, case["head_dim"], case["kv_heads"]
    group, outs = c["q_heads"] // hkv, []
    for i, n in enumerate(_lengths(c)):
        j = torch.arange(n, device="cuda")
        first = n - c["rows"]
        if c["window"]:  # what no row sees is left out
            j = j[(j < c["sinks"]) | (j > first - c["window"])]
        k, v = _exact_rows(s, i, j)
        q = s.q.view(c["seqs"], c["rows"], hkv, group, d)[i].double()
        a = torch.einsum("rhgd,jhd->rhgj", q, k) / math.sqrt(d)
        pos = first + torch.arange(c["rows"], device="cuda")
        seen = j[None] <= pos[:, None]
        if c["window"]:
            seen &= (j[None] > pos[:, None] - c["window"]) | (j[None] < c["sinks"])
        a = torch.softmax(a.masked_fill(~seen[:, None, None], float("-inf")), 3)
        outs.append(torch.einsum("rhgj,jhd->rhgd", a, v).reshape(c["rows"], c["q_heads"], d))
    return {"out": torch.cat(outs)}


def _exact_rows(s, seq, positions):
    """Keys and values of a sequence's positions in 64 bits: [positions, kv_heads, head_dim]."""
    page, slot = s.page_table[seq].long()[positions // s.case["page"]], positions % s.case["page"]

    def one(code, affine):
        code, affine = code[page, :, slot], affine[page, :, slot].double()
        if s.case["bits"] == 4:
            low, high = code % 16, code.div(16, rounding_mode="floor")
            code = torch.cat((low[..., None], high[..., None]), -1).reshape(*low.shape[:2], -1)
        scale, bias = (affine[..., i].repeat_interleave(GROUP, 2) for i in (0, 1))
        return torch.addcmul(bias, code.double(), scale)

    return one(s.k, s.k_affine), one(s.v, s.v_affine)


def _exact_read(s):
    c, k_out, v_out = s.case, s.k_out.double(), s.v_out.double()
    for i, n in enumerate(_lengths(c)):
        j = torch.arange(c.get("start", 0), n, device="cuda")
        k_out[i, :len(j)], v_out[i, :len(j)] = _exact_rows(s, i, j)
    return {"k": k_out, "v": v_out}


def _exact_append(s):
    c, d = s.case, s.case["head_dim"]
    half, top = c["rot"] // 2, 2 ** c["bits"] - 1
    pos = torch.cat([torch.arange(n - c["rows"], n, device="cuda") for n in _lengths(c)])
    turn = torch.complex(s.rope[pos, :half].double(), s.rope[pos, half:].double())[:, None]

    def turned(x, weight):
        x = x.double().reshape(len(pos), -1, d)
        x = x / torch.sqrt(x.square().sum(2, keepdim=True) / d + EPS) * weight.double()
        if c["interleaved"]:
            y = torch.view_as_complex(x[..., :c["rot"]].reshape(*x.shape[:2], half, 2)) * turn
            x[..., :c["rot"]] = torch.view_as_real(y).flatten(2)
        else:
            y = torch.complex(x[..., :half], x[..., half:c["rot"]].clone()) * turn
            x[..., :half], x[..., half:c["rot"]] = y.real, y.imag
        return x

    def stored(x):
        x = x.reshape(*x.shape[:2], -1, GROUP)
        bias = x.min(3, keepdim=True).values
        scale = ((x.max(3, keepdim=True).values - bias) / top).to(torch.float16).double()
        bias = bias.to(torch.float16).double()
        return (((x - bias) / scale).round().clamp(0, top) * scale + bias).flatten(2)

    k, v = stored(turned(s.new_k, s.k_weight)), stored(s.new_v.double().reshape(len(pos), -1, d))
    out = _exact_read(s)
    at = 0
    for i, n in enumerate(_lengths(c)):
        out["k"][i, n - c["rows"]:n], out["v"][i, n - c["rows"]:n] = k[at:at + c["rows"]], v[at:at + c["rows"]]
        at += c["rows"]
    return {"q": turned(s.new_q, s.q_weight), **out}

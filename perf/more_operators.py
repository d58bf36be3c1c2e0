"""Cases of the operators of a decode step whose sequences share a prompt: the append of keys and values with the
position rotation, attention of sequences that share a prefix's pages, and sampling of tokens from logits.

``run`` computes each operator in its plain form (elementary torch operations, 32-bit arithmetic, 64 bits for angles and
for the sums that a token is drawn from) or, with ``own`` set, through the library's entry points.  Layouts are the
library's: cache pages [pages, Hkv, 16, D], block tables [rows, max pages], token rows [T, heads, D] with prefix sums,
logits [rows, vocabulary].
"""

import math
import random

import torch

own = False

PAGE = 16
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


# ------------------------------------------------------------------ cases

def listed():
    return [
        # one decoded token of each sequence of the serving mix, one layer of a model step: latency
        dict(name="rope_decode", op="rope", batch=32, q_heads=32, kv_heads=8, dim=128, rotary=128, pairs="split",
             base=500000.0, dtype="bf16", new_lo=1, new_hi=1, ctx_lo=1000, ctx_hi=1600, lens=1),
        # a long prompt chunk in three ragged pieces, q, k and v slices of the fused projection
        dict(name="rope_prompt", op="rope", batch=3, q_heads=32, kv_heads=8, dim=128, rotary=128, pairs="split",
             base=500000.0, dtype="bf16", new_lo=2501, new_hi=2903, ctx_lo=0, ctx_hi=4099, lens=2),
        # chunks far behind the start of books, neighbouring pairs, half of each head rotated: the angles' exactness
        dict(name="rope_far", op="rope", batch=5, q_heads=64, kv_heads=8, dim=128, rotary=64, pairs="next",
             base=10000.0, dtype="fp16", new_lo=1, new_hi=701, ctx_lo=200000, ctx_hi=1000000, lens=3),
        # two samples of one short prompt on the tiny shape: latency
        dict(name="prefix_tiny", op="prefix", groups=1, each_lo=2, each_hi=2, q_heads=8, kv_heads=2, dim=64, dtype="bf16",
             prefix_lo=500, prefix_hi=510, tail_lo=1, tail_hi=40, new_lo=1, new_hi=1, lens=4),
        # four samples of each of 16 prompts of the serving mix, some way into their answers
        dict(name="prefix_serving", op="prefix", groups=16, each_lo=4, each_hi=4, q_heads=32, kv_heads=8, dim=128,
             dtype="bf16", prefix_lo=1000, prefix_hi=1600, tail_lo=1, tail_hi=600, new_lo=1, new_hi=1, lens=5),
        # 64 samples over one book (the benchmark's 60K point)
        dict(name="prefix_long", op="prefix", groups=1, each_lo=64, each_hi=64, q_heads=32, kv_heads=8, dim=128,
             dtype="fp16", prefix_lo=60000, prefix_hi=60000, tail_lo=100, tail_hi=700, new_lo=1, new_hi=1, lens=6),
        # questions of many users behind one system prompt, prefilled at once on the SpecBlock head layout: the largest
        dict(name="prefix_prompts", op="prefix", groups=1, each_lo=12, each_hi=12, q_heads=64, kv_heads=8, dim=128,
             dtype="bf16", prefix_lo=4099, prefix_hi=4099, tail_lo=0, tail_hi=15, new_lo=90, new_hi=301, lens=7),
        # one user's next token, every filter on, the tiny shape's vocabulary: latency
        dict(name="sample_one", op="sample", rows=1, vocab=32000, dtype="fp32", temperature=0.8, top_k=50, top_p=0.95,
             min_p=0.02, mixed=0, probs=0, lens=8),
        # the serving mix's tokens from the whole distribution, temperature alone
        dict(name="sample_plain", op="sample", rows=32, vocab=128256, dtype="bf16", temperature=1.0, top_k=0, top_p=1.0,
             min_p=0.0, mixed=0, probs=0, lens=9),
        # the usual nucleus, no limit on its number
        dict(name="sample_nucleus", op="sample", rows=64, vocab=128256, dtype="fp32", temperature=0.7, top_k=0, top_p=0.9,
             min_p=0.0, mixed=0, probs=0, lens=10),
        # a large batch whose users set their own values (greedy rows among them)
        dict(name="sample_mixed", op="sample", rows=256, vocab=151936, dtype="bf16", temperature=1.0, top_k=0, top_p=1.0,
             min_p=0.0, mixed=1, probs=0, lens=11),
        # the draft model's level of a tree: tokens and the distributions that stochastic acceptance wants beside them
        dict(name="sample_draft", op="sample", rows=60, vocab=128256, dtype="fp32", temperature=1.0, top_k=64, top_p=1.0,
             min_p=0.0, mixed=0, probs=1, lens=12),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope", "prefix", "prefix", "sample", "sample"])
    lens = rng.randrange(1 << 20)
    dtype = rng.choice(["bf16", "fp16"])
    q_heads, kv_heads, dim = rng.choice([(8, 2, 64), (32, 8, 128), (64, 8, 128), (20, 20, 64), (28, 4, 128), (12, 4, 64),
                                         (32, 1, 128)])
    if op == "rope":
        batch = _log(rng, 1, 64)
        new_hi = _log(rng, 1, max(1, 8192 // batch))
        ctx_hi = _log(rng, 1, 1000000)
        return dict(op=op, batch=batch, q_heads=q_heads, kv_heads=kv_heads, dim=dim,
                    rotary=rng.choice([dim, dim, dim // 2, 16 * rng.randrange(1, dim // 16 + 1)]),
                    pairs=rng.choice(["split", "split", "next"]), base=rng.choice([10000.0, 500000.0, 1000000.0]),
                    dtype=dtype, new_lo=rng.randrange(0, new_hi + 1), new_hi=new_hi,
                    ctx_lo=rng.randrange(0, ctx_hi + 1), ctx_hi=ctx_hi, lens=lens)
    if op == "prefix":
        groups = _log(rng, 1, 16)
        each_hi = _log(rng, 1, 64)
        new_hi = rng.choice([1, 1, 1, rng.randrange(2, 9), _log(rng, 9, 300)])
        prefix_hi = _log(rng, 16, 60000)
        tail_hi = _log(rng, 1, 1500)
        # no more than the largest listed calls: query rows times keys, and bytes of keys in the plain form
        while (groups * each_hi * new_hi * q_heads * (prefix_hi + tail_hi + new_hi) > 12 * 200 * 64 * 4400 or
               groups * each_hi * kv_heads * dim * (prefix_hi + tail_hi + new_hi) > 64 * 8 * 128 * 61000):
            if each_hi > 2 and rng.random() < 0.5:
                each_hi = each_hi * 2 // 3
            elif groups > 1 and rng.random() < 0.5:
                groups = groups // 2
            elif new_hi > 8:
                new_hi = new_hi * 2 // 3
            else:
                prefix_hi = prefix_hi * 2 // 3
        return dict(op=op, groups=groups, each_lo=rng.randrange(1, each_hi + 1), each_hi=each_hi, q_heads=q_heads,
                    kv_heads=kv_heads, dim=dim, dtype=dtype, prefix_lo=rng.randrange(0, prefix_hi + 1),
                    prefix_hi=prefix_hi, tail_lo=rng.randrange(0, tail_hi + 1), tail_hi=tail_hi,
                    new_lo=rng.randrange(1, new_hi + 1), new_hi=new_hi, lens=lens)
    vocab = rng.choice([32000, 128256, 151936, 50257, _log(rng, 2, 262144)])
    rows = min(_log(rng, 1, 256), 256 * 151936 // vocab)
    probs = int(rng.random() < 0.3)
    return dict(op=op, rows=max(1, rows // 4) if probs else rows, vocab=vocab, dtype=rng.choice(["fp32", "bf16", "fp16"]),
                temperature=round(rng.uniform(0.2, 1.5), 2), top_k=rng.choice([0, 0, _log(rng, 1, 2000)]),
                top_p=rng.choice([1.0, round(rng.uniform(0.1, 0.99), 2)]),
                min_p=rng.choice([0.0, 0.0, round(rng.uniform(0.001, 0.3), 3)]), mixed=int(rng.random() < 0.3), probs=probs,
                lens=lens)


def _lengths(case):
    """(new tokens, context length) of each sequence: part of the case, the same for every seed.  Of a prefix case also
    the sequences of each group and its shared tokens (whole pages: the ragged last page of a prompt is not shared)."""
    r = random.Random(case["lens"])
    if case["op"] == "rope":
        new = [r.randint(case["new_lo"], case["new_hi"]) for _ in range(case["batch"])]
        if sum(new) == 0:
            new[0] = case["new_hi"]
        return new, [r.randint(case["ctx_lo"], case["ctx_hi"]) for _ in new]
    each = [r.randint(case["each_lo"], case["each_hi"]) for _ in range(case["groups"])]
    prompts = [r.randint(case["prefix_lo"], case["prefix_hi"]) for _ in each]
    ctx = [p + r.randint(case["tail_lo"], case["tail_hi"]) for p, n in zip(prompts, each) for _ in range(n)]
    new = [r.randint(case["new_lo"], case["new_hi"]) for _ in ctx]
    return new, ctx, each, [p // PAGE * PAGE for p in prompts]


def _settings(case):
    """Temperature, top-k, top-p and min-p of each row: part of the case, the same for every seed."""
    n = case["rows"]
    if not case["mixed"]:
        return [[case[k]] * n for k in ("temperature", "top_k", "top_p", "min_p")]
    r = random.Random(case["lens"])
    return [[r.choice([0.0, 0.6, 0.7, 0.8, 1.0, 1.0, 1.2]) for _ in range(n)],
            [r.choice([0, 0, 0, 20, 40, 50, 100, 1000]) for _ in range(n)],
            [r.choice([1.0, 1.0, 0.8, 0.9, 0.95, 0.98]) for _ in range(n)],
            [r.choice([0.0, 0.0, 0.0, 0.02, 0.05, 0.1]) for _ in range(n)]]


# ------------------------------------------------------------------ inputs

def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _floats(v):
    return torch.tensor(v, dtype=torch.float32, device="cuda")


def _cu(new):
    out = [0]
    for n in new:
        out.append(out[-1] + n)
    return out


def _normal(gen, shape, dtype):
    return torch.randn(shape, generator=gen, device="cuda", dtype=dtype)


def _table(gen, first, held, num_pages, width):
    """Block table [rows, width]: logical pages first .. held - 1 of each row name different pages of the pool; -1
    elsewhere."""
    perm = torch.randperm(num_pages, generator=gen, device="cuda").to(torch.int32)
    a, h = _ints(first), _ints(held)
    at = torch.arange(width, device="cuda")
    before = torch.cumsum(h - a, 0) - (h - a)
    inside = (at >= a[:, None]) & (at < h[:, None])
    idx = (before[:, None] + at - a[:, None]).clamp(0, num_pages - 1)
    return torch.where(inside, perm[idx], -1).to(torch.int32).contiguous()


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed))
    dt = TYPES[case["dtype"]]
    s = dict(case=case)
    if case["op"] == "sample":
        return _prepare_sample(case, gen, dt, s)
    Hq, H, D = case["q_heads"], case["kv_heads"], case["dim"]
    if case["op"] == "rope":
        new, ctx = _lengths(case)
        first = [c // PAGE for c in ctx]  # (the pages before stand for a long past that this call does not touch)
    else:
        new, ctx, each, shared = _lengths(case)
        s["cu_groups"], s["prefix"] = _ints(_cu(each)), _ints(shared)
        lead = [int(i == 0) for n in each for i in range(n)]  # the first of a group holds the shared pages
        first = [0 if f else p // PAGE for f, p in zip(lead, [p for p, n in zip(shared, each) for _ in range(n)])]
    held = [(c + n + PAGE - 1) // PAGE for c, n in zip(ctx, new)]
    num_pages = sum(h - f for h, f in zip(held, first)) + 8
    s.update(table=_table(gen, first, held, num_pages, max(max(held), 1)), ctx=_ints(ctx), cu=_ints(_cu(new)),
             total=sum(new), most=max(new), kc=_normal(gen, (num_pages, H, PAGE, D), dt),
             vc=_normal(gen, (num_pages, H, PAGE, D), dt))
    if case["op"] == "rope":
        # rows of the fused projection: query heads, then key heads, then value heads
        rows = _normal(gen, (s["total"], Hq + 2 * H, D), dt)
        s["q"], s["k"], s["v"] = rows[:, :Hq], rows[:, Hq:Hq + H], rows[:, Hq + H:]
        s["q_out"] = torch.empty((s["total"], Hq, D), dtype=dt, device="cuda")
        s["new_ctx"] = torch.empty_like(s["ctx"])
        j = torch.arange(case["rotary"] // 2, dtype=torch.float64, device="cuda")
        s["inv_freq"] = (case["base"] ** (-2.0 * j / case["rotary"])).float()
        return s
    leads = [i for i, f in enumerate(lead) if f]
    lp = torch.arange(s["table"].shape[1], device="cuda")
    group = _ints([g for g, n in enumerate(each) for _ in range(n)]).long()
    s["table"] = torch.where(lp < (s["prefix"][group] // PAGE)[:, None], s["table"][_ints(leads).long()][group],
                             s["table"]).contiguous()
    s["q"] = _normal(gen, (s["total"], Hq, D), dt)
    s["out"] = torch.empty_like(s["q"])
    s["lse"] = torch.empty((s["total"], Hq), dtype=torch.float32, device="cuda")
    s["most_of_group"] = max(sum(new[a:b]) for a, b in zip(_cu(each), _cu(each)[1:]))
    if own:
        _plan(s)
    return s


def _prepare_sample(case, gen, dt, s):
    """Logits as a language model's: a broad bulk and a few likely tokens above it."""
    R, V = case["rows"], case["vocab"]
    x = 2.0 * torch.randn((R, V), generator=gen, device="cuda")
    likely = torch.randint(0, V, (R, 60), generator=gen, device="cuda")
    rise = 14.0 * torch.rand((R, 60), generator=gen, device="cuda")
    s["logits"] = x.scatter_add_(1, likely, rise).to(dt)
    s["u"] = torch.rand(R, generator=gen, device="cuda")
    t, k, p, m = _settings(case)
    s.update(temperature=_floats(t), top_k=_ints(k), top_p=_floats(p), min_p=_floats(m),
             tokens=torch.empty(R, dtype=torch.int32, device="cuda"), logprobs=torch.empty(R, device="cuda"))
    s["probs"] = torch.empty((R, V), device="cuda") if case["probs"] else None
    return s


# ------------------------------------------------------------------ one pass

def run(s):
    op = s["case"]["op"]
    if own:
        return {"rope": _own_rope, "prefix": _own_prefix, "sample": _own_sample}[op](s)
    return {"rope": _plain_rope, "prefix": _plain_prefix, "sample": _plain_sample}[op](s)


def _token_rows(s):
    """Sequence and position within it of every token row."""
    at = torch.arange(s["total"], device="cuda", dtype=torch.int32)
    b = torch.searchsorted(s["cu"][1:].contiguous(), at, right=True)
    return b, at - s["cu"][b]


def _rotate(x, cos, sin, case):
    """The first `rotary` elements of each head rotated, in 32 bits."""
    r = case["rotary"]
    y = x[..., :r].float()
    if case["pairs"] == "split":
        a, b = y[..., :r // 2], y[..., r // 2:]
        y = torch.cat([a * cos - b * sin, a * sin + b * cos], -1)
    else:
        a, b = y[..., 0::2], y[..., 1::2]
        y = torch.stack([a * cos - b * sin, a * sin + b * cos], -1).flatten(-2)
    return torch.cat([y.to(x.dtype), x[..., r:]], -1)


def _plain_rope(s):
    b, i = _token_rows(s)
    slot = (s["ctx"][b] + i).long()
    angle = slot[:, None].double() * s["inv_freq"].double()
    cos, sin = angle.cos().float()[:, None], angle.sin().float()[:, None]
    page = s["table"][b, slot // PAGE].long()
    s["kc"][page, :, slot % PAGE] = _rotate(s["k"], cos, sin, s["case"])
    s["vc"][page, :, slot % PAGE] = s["v"]
    return _rotate(s["q"], cos, sin, s["case"]), s["kc"], s["vc"], s["ctx"] + (s["cu"][1:] - s["cu"][:-1])


def _plain_prefix(s):
    """Attention of every sequence over all of its pages: what a prefix is shared for does not show in the result."""
    c = s["case"]
    B, Hq, H, D, S = s["ctx"].shape[0], c["q_heads"], c["kv_heads"], c["dim"], s["table"].shape[1] * PAGE
    n = s["cu"][1:] - s["cu"][:-1]
    i = torch.arange(s["most"], device="cuda")
    rows = (s["cu"][:-1, None] + i).clamp(max=s["total"] - 1)
    q = s["q"][rows].float().view(B, s["most"], H, Hq // H, D).permute(0, 2, 3, 1, 4).reshape(B, H, -1, D)
    pages = s["table"].clamp(min=0).long()
    k = s["kc"][pages].permute(0, 2, 1, 3, 4).reshape(B, H, S, D).float()
    scores = torch.matmul(q, k.transpose(-1, -2)).mul_(1.0 / math.sqrt(D)).view(B, H, Hq // H, s["most"], S)
    del k
    j = torch.arange(S, device="cuda")
    last = (s["ctx"][:, None] + i)[:, :, None]
    seen = (j <= last) & (j < (s["ctx"] + n)[:, None, None])
    scores.masked_fill_(~seen[:, None, None], -math.inf)
    top = scores.amax(-1, keepdim=True)
    p = scores.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    v = s["vc"][pages].permute(0, 2, 1, 3, 4).reshape(B, H, S, D).float()
    o = torch.matmul(p.view(B, H, -1, S), v).view(B, H, Hq // H, s["most"], D) / total
    b, at = _token_rows(s)
    o = o.permute(0, 3, 1, 2, 4).reshape(B, s["most"], Hq, D)[b, at]
    lse = (top + total.log())[..., 0].permute(0, 3, 1, 2).reshape(B, s["most"], Hq)[b, at]
    return o.to(s["q"].dtype), lse


def _plain_sample(s):
    """In 64 bits: a token is a comparison of sums over the whole vocabulary."""
    x = s["logits"].double()
    R, V = x.shape
    greedy = (s["temperature"] == 0)[:, None]
    t = torch.where(greedy[:, 0], 1.0, s["temperature"]).double()[:, None]
    order = torch.sort(x, descending=True, stable=True)
    w = ((order.values - order.values[:, :1]) / t).exp()
    at = torch.arange(V, device="cuda")
    k = torch.where(s["top_k"] <= 0, V, s["top_k"])[:, None]
    in_k = at < k
    within = (w * in_k).cumsum(1)
    # the least prefix whose sum reaches top_p of the k kept ones'
    p = s["top_p"].double()[:, None]
    in_p = (within - w < p * within[:, -1:]) | (p >= 1) | (at == 0)
    kept = in_k & in_p & (w >= s["min_p"].double()[:, None]) & (~greedy | (at == 0)) | (at == 0)
    weight = torch.zeros_like(x).scatter_(1, order.indices, w * kept)
    running = weight.cumsum(1)
    total = running[:, -1:]
    token = torch.argmax((running > s["u"].double()[:, None] * total).to(torch.uint8), 1)
    logprob = (weight.gather(1, token[:, None]) / total).log()[:, 0].float()
    probs = (weight / total).float() if s["probs"] is not None else None
    return token.to(torch.int32), logprob, probs


# ------------------------------------------------------------------ the library's calls

def _sv():
    from speculative_decoding_tree_sv_gb300 import binding
    return binding


def _plan(s):
    """The parameters and the workspace that a caller keeps."""
    sv = _sv()
    s["params"] = sv.make_prefix_params(q=s["q"], k_cache=s["kc"], v_cache=s["vc"], block_table=s["table"],
                                        ctx_lens=s["ctx"], cu_tokens=s["cu"], cu_groups=s["cu_groups"],
                                        prefix_lens=s["prefix"], out=s["out"], lse=s["lse"], max_tokens=s["most"],
                                        max_group_tokens=s["most_of_group"])
    s["work"] = torch.zeros(sv.sv_prefix_attention_workspace_size(s["params"]), dtype=torch.uint8, device="cuda")
    s["params"].workspace, s["params"].workspace_bytes = s["work"].data_ptr(), s["work"].numel()


def _own_rope(s):
    _sv().sv_rope_append(s["q"], s["k"], s["v"], s["q_out"], s["kc"], s["vc"], s["table"], s["ctx"], s["cu"],
                         s["inv_freq"], interleaved=s["case"]["pairs"] == "next", new_ctx_lens=s["new_ctx"])
    return s["q_out"], s["kc"], s["vc"], s["new_ctx"]


def _own_prefix(s):
    _sv().sv_prefix_attention(s["params"])
    return s["out"], s["lse"]


def _own_sample(s):
    _sv().sv_sample_tokens(s["logits"], s["u"], s["tokens"], temperature=s["temperature"], top_k=s["top_k"],
                           top_p=s["top_p"], min_p=s["min_p"], logprobs=s["logprobs"], probs=s["probs"])
    return s["tokens"], s["logprobs"], s["probs"]


# ------------------------------------------------------------------ what a pass cannot do without

def work(case):
    if case["op"] == "sample":
        size = 4 if case["dtype"] == "fp32" else 2
        return {"bytes": case["rows"] * (case["vocab"] * (size + 4 * case["probs"]) + 28), "flops": 0}
    row = 2 * case["dim"]  # bytes of a head's row
    if case["op"] == "rope":
        new, _ = _lengths(case)
        return {"bytes": 2 * sum(new) * (case["q_heads"] + 2 * case["kv_heads"]) * row,
                "flops": 3 * sum(new) * (case["q_heads"] + case["kv_heads"]) * case["rotary"]}
    new, ctx, each, shared = _lengths(case)
    group = [g for g, n in enumerate(each) for _ in range(n)]
    own_keys = sum(c + n - shared[g] for c, n, g in zip(ctx, new, group))
    seen = sum(n * c + n * (n + 1) // 2 for c, n in zip(ctx, new))
    return {"bytes": 2 * (sum(shared) + own_keys) * case["kv_heads"] * row + sum(new) * case["q_heads"] * (2 * row + 4),
            "flops": 4 * seen * case["q_heads"] * case["dim"]}


# ------------------------------------------------------------------ by definition, in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    return {"rope": _exact_rope, "prefix": _exact_prefix, "sample": _exact_sample}[case["op"]](s)


def _exact_rope(s):
    """Each pair as a complex number times e^(i position frequency), one sequence at a time."""
    case = s["case"]
    new, ctx = _lengths(case)
    r, table = case["rotary"], s["table"].long()

    def turned(x, turn):
        y = x.double()
        first, second = ((slice(0, r // 2), slice(r // 2, r)) if case["pairs"] == "split" else
                         (slice(0, r, 2), slice(1, r, 2)))
        z = torch.complex(y[..., first], y[..., second]) * turn[:, None]
        y[..., first], y[..., second] = z.real, z.imag
        return y

    kc, vc = s["kc"].double(), s["vc"].double()
    q_out = torch.empty(s["q"].shape, dtype=torch.float64, device="cuda")
    at = 0
    for b, (n, c) in enumerate(zip(new, ctx)):
        pos = torch.arange(c, c + n, device="cuda")
        angle = pos.double()[:, None] * s["inv_freq"].double()
        turn = torch.polar(torch.ones_like(angle), angle)
        rows = slice(at, at + n)
        q_out[rows] = turned(s["q"][rows], turn)
        kc[table[b, pos // PAGE], :, pos % PAGE] = turned(s["k"][rows], turn)
        vc[table[b, pos // PAGE], :, pos % PAGE] = s["v"][rows].double()
        at += n
    return q_out, kc, vc, s["ctx"] + _ints(new)


def _exact_prefix(s):
    """One sequence and key head at a time."""
    case = s["case"]
    new, ctx, _, _ = _lengths(case)
    Hq, H, D = case["q_heads"], case["kv_heads"], case["dim"]
    G = Hq // H
    out = torch.empty((s["total"], Hq, D), dtype=torch.float64, device="cuda")
    lse = torch.empty((s["total"], Hq), dtype=torch.float64, device="cuda")
    at = 0
    for b, (n, c) in enumerate(zip(new, ctx)):
        pages = s["table"][b, :(c + n + PAGE - 1) // PAGE].long()
        hidden = torch.arange(c + n, device="cuda") > torch.arange(c, c + n, device="cuda")[:, None]
        for h in range(H):
            k = s["kc"][pages, h].reshape(-1, D)[:c + n].double()
            v = s["vc"][pages, h].reshape(-1, D)[:c + n].double()
            x = s["q"][at:at + n, h * G:(h + 1) * G].double().transpose(0, 1) @ k.T / math.sqrt(D)
            x[:, hidden] = -math.inf
            lse[at:at + n, h * G:(h + 1) * G] = torch.logsumexp(x, 2).T
            out[at:at + n, h * G:(h + 1) * G] = (torch.softmax(x, 2) @ v).transpose(0, 1)
        at += n
    return out, lse


def _exact_sample(s):
    """Row by row over the sorted candidates alone."""
    case = s["case"]
    tokens, logprobs = [], []
    probs = torch.zeros(s["logits"].shape, dtype=torch.float64, device="cuda") if s["probs"] is not None else None
    for r, (t, k, p, m) in enumerate(zip(*_settings(case))):
        t, p, m = (float(torch.tensor(v, dtype=torch.float32)) for v in (t, p, m))  # the inputs have 32 bits
        x = s["logits"][r].double()
        if t == 0:
            best = int(torch.nonzero(x == x.max())[0])
            tokens.append(best)
            logprobs.append(0.0)
            if probs is not None:
                probs[r, best] = 1.0
            continue
        rank = torch.argsort(-x, stable=True)[:k if k > 0 else x.numel()]
        prob = torch.softmax(x[rank] / t, 0)
        stay = 1 + int((torch.cumsum(prob, 0)[:-1] < p).sum()) if p < 1 else prob.numel()
        stay = max(1, min(stay, int((prob >= m * prob[0]).sum())))
        place, by_place = torch.sort(rank[:stay])
        prob = (prob[:stay] / prob[:stay].sum())[by_place]
        i = int((torch.cumsum(prob, 0) <= float(s["u"][r])).sum())
        i = min(i, stay - 1)
        tokens.append(int(place[i]))
        logprobs.append(float(prob[i].log()))
        if probs is not None:
            probs[r, place] = prob
    return _ints(tokens), torch.tensor(logprobs, dtype=torch.float64, device="cuda"), probs

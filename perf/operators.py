"""Cases of the prompt and cache operators: chunk attention over the paged cache, the append of a
chunk's keys and values, and the page bookkeeping (fork, reserve, release, compact, copy).

``run`` computes each operator in its plain form (elementary torch operations, 32-bit arithmetic) or,
with ``own`` set, through the library's entry points.  Layouts are the library's: cache pages
[pages, Hkv, 16, D], block tables [rows, max pages], token rows [T, heads, D] with prefix sums.
"""

import math
import random

import torch

own = False

PAGE = 16
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}


# ------------------------------------------------------------------ cases

def listed():
    return [
        # one user, the first tokens of an answer: the smallest call, where only latency counts
        dict(name="decode_tiny", op="chunk", batch=1, q_heads=8, kv_heads=2, dim=64, dtype="bf16", new_lo=1, new_hi=1,
             long_rows=0, ctx_lo=511, ctx_hi=511, window=0, sink=0, lens=1),
        # the serving mix of the benchmark (32 sequences of 1000 to 1600 tokens) between speculative steps
        dict(name="decode_serving", op="chunk", batch=32, q_heads=32, kv_heads=8, dim=128, dtype="bf16", new_lo=1,
             new_hi=1, long_rows=0, ctx_lo=1000, ctx_hi=1600, window=0, sink=0, lens=2),
        # a few users with books in their context (the benchmark's 60K point), one token each
        dict(name="decode_long", op="chunk", batch=4, q_heads=32, kv_heads=8, dim=128, dtype="fp16", new_lo=1, new_hi=1,
             long_rows=0, ctx_lo=40000, ctx_hi=61440, window=0, sink=0, lens=3),
        # one engine step that mixes decoding sequences with chunks of four prompts, all ragged
        dict(name="mixed_step", op="chunk", batch=24, q_heads=32, kv_heads=8, dim=128, dtype="bf16", new_lo=1, new_hi=509,
             long_rows=4, ctx_lo=700, ctx_hi=2611, window=0, sink=0, lens=4),
        # the last chunk of a 32K prompt: the largest call, bound by the tensor cores
        dict(name="prompt_chunk", op="chunk", batch=1, q_heads=32, kv_heads=8, dim=128, dtype="bf16", new_lo=4096,
             new_hi=4096, long_rows=1, ctx_lo=28672, ctx_hi=28672, window=0, sink=0, lens=5),
        # sliding window with sink tokens on the SpecBlock head layout, two prompts of odd lengths
        dict(name="window_chunk", op="chunk", batch=2, q_heads=64, kv_heads=8, dim=128, dtype="fp16", new_lo=901,
             new_hi=1103, long_rows=2, ctx_lo=15001, ctx_hi=16384, window=4096, sink=64, lens=6),
        # the keys and values of one decoded token for every layer of the 32-layer shape
        dict(name="append_decode", op="append", batch=32, layers=32, kv_heads=8, dim=128, dtype="bf16", new_lo=1, new_hi=1,
             ctx_lo=1000, ctx_hi=1600, fused=0, lens=7),
        # one layer of a long prompt chunk in ragged pieces, keys and values slices of the fused projection
        dict(name="append_prompt", op="append", batch=3, layers=1, kv_heads=8, dim=128, dtype="fp16", new_lo=2501,
             new_hi=2903, ctx_lo=0, ctx_hi=4099, fused=32, lens=8),
        # two samples of one short prompt on the tiny shape: bookkeeping latency
        dict(name="fork_tiny", op="fork", parents=1, each=2, layers=1, kv_heads=2, dim=64, dtype="bf16", new_hi=4,
             ctx_lo=500, ctx_hi=510, spare=32, lens=9),
        # four samples of each of 16 prompts, 32 layers: pages shared, the ragged tail pages copied
        dict(name="fork_serving", op="fork", parents=16, each=4, layers=32, kv_heads=8, dim=128, dtype="bf16", new_hi=9,
             ctx_lo=1000, ctx_hi=1600, spare=128, lens=10),
        # a small pool with holes: latency of one compaction
        dict(name="compact_tiny", op="compact", rows=4, layers=1, kv_heads=2, dim=64, dtype="bf16", ctx_lo=100, ctx_hi=700,
             pages=256, lens=11),
        # a fragmented pool after half of its sequences have left
        dict(name="compact_serving", op="compact", rows=48, layers=8, kv_heads=8, dim=128, dtype="bf16", ctx_lo=1000,
             ctx_hi=2200, pages=8192, lens=12),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["chunk", "chunk", "chunk", "append", "fork", "compact"])
    lens = rng.randrange(1 << 20)
    dtype = rng.choice(["bf16", "fp16"])
    q_heads, kv_heads, dim = rng.choice([(8, 2, 64), (32, 8, 128), (64, 8, 128), (20, 20, 64), (28, 4, 128), (12, 4, 64),
                                         (32, 1, 128)])
    if op == "chunk":
        batch = _log(rng, 1, 48)
        new_hi = rng.choice([1, 1, rng.randrange(2, 9), _log(rng, 9, 4096)])
        ctx_hi = _log(rng, 1, 61440)
        while batch * q_heads * new_hi * (ctx_hi + new_hi) > 32 * 4096 * 30000 or batch * ctx_hi > 262144:
            if batch > 1:
                batch = batch // 2
            elif new_hi > 64:
                new_hi = new_hi * 2 // 3
            else:
                ctx_hi = ctx_hi * 2 // 3
        window, sink = rng.choice([(0, 0), (0, 0), (0, 0), (_log(rng, 16, 4096), rng.randrange(0, 130))])
        return dict(op=op, batch=batch, q_heads=q_heads, kv_heads=kv_heads, dim=dim, dtype=dtype,
                    new_lo=rng.randrange(1, new_hi + 1), new_hi=new_hi, long_rows=rng.randrange(0, batch + 1),
                    ctx_lo=rng.randrange(0, ctx_hi + 1), ctx_hi=ctx_hi, window=window, sink=sink, lens=lens)
    if op == "append":
        layers = rng.choice([1, 1, 4, 32])
        batch = _log(rng, 1, 48)
        new_hi = _log(rng, 1, max(1, 8192 // (batch * layers)))
        ctx_hi = _log(rng, 1, 4096)
        return dict(op=op, batch=batch, layers=layers, kv_heads=kv_heads, dim=dim, dtype=dtype,
                    new_lo=rng.randrange(0, new_hi + 1), new_hi=new_hi, ctx_lo=rng.randrange(0, ctx_hi + 1),
                    ctx_hi=ctx_hi, fused=q_heads if layers == 1 and rng.random() < 0.5 else 0, lens=lens)
    layers = rng.choice([1, 4, 16])
    if op == "fork":
        ctx_hi = _log(rng, 1, 2048)
        return dict(op=op, parents=rng.randrange(1, 17), each=rng.randrange(1, 5), layers=layers, kv_heads=kv_heads,
                    dim=dim, dtype=dtype, new_hi=rng.randrange(1, 40), ctx_lo=rng.randrange(0, ctx_hi + 1),
                    ctx_hi=ctx_hi, spare=rng.randrange(256, 512), lens=lens)
    rows = _log(rng, 1, 48)
    ctx_hi = _log(rng, 16, 2200)
    pages = rows * (ctx_hi // PAGE + 1) + rng.randrange(1, 4000)
    return dict(op=op, rows=rows, layers=min(layers, 8), kv_heads=kv_heads, dim=dim, dtype=dtype,
                ctx_lo=rng.randrange(0, ctx_hi + 1), ctx_hi=ctx_hi, pages=pages, lens=lens)


def _lengths(case):
    """(new tokens, context length) of each sequence: part of the case, the same for every seed."""
    r = random.Random(case["lens"])
    if case["op"] == "fork":
        return [], [r.randint(case["ctx_lo"], case["ctx_hi"]) for _ in range(case["parents"])]
    if case["op"] == "compact":
        return [], [r.randint(case["ctx_lo"], case["ctx_hi"]) for _ in range(case["rows"])]
    n = case["batch"]
    if case["op"] == "append":
        new = [r.randint(case["new_lo"], case["new_hi"]) for _ in range(n)]
        if sum(new) == 0:
            new[0] = case["new_hi"]
    else:  # `long_rows` sequences bring a chunk, the others one token
        new = [r.randint(case["new_lo"], case["new_hi"]) if i < case["long_rows"] else 1 for i in range(n)]
        r.shuffle(new)
    return new, [r.randint(case["ctx_lo"], case["ctx_hi"]) for _ in range(n)]


# ------------------------------------------------------------------ inputs

def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _cu(new):
    out = [0]
    for n in new:
        out.append(out[-1] + n)
    return out


def _normal(gen, shape, dtype):
    return torch.randn(shape, generator=gen, device="cuda", dtype=dtype)


def _table(gen, held, num_pages, width):
    """Block table [rows, width]: `held` pages per row, all different, spread over the pool; -1 behind them."""
    perm = torch.randperm(num_pages, generator=gen, device="cuda").to(torch.int32)
    h = _ints(held)
    at = torch.arange(width, device="cuda")
    first = torch.cumsum(h, 0) - h
    idx = (first[:, None] + at).clamp(max=num_pages - 1)
    return torch.where(at < h[:, None], perm[idx], -1).to(torch.int32).contiguous()


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed))
    dt, H, D = TYPES[case["dtype"]], case["kv_heads"], case["dim"]
    new, ctx = _lengths(case)
    s = dict(case=case)
    if case["op"] in ("chunk", "append"):
        held = [(c + n + PAGE - 1) // PAGE for c, n in zip(ctx, new)]
        num_pages = sum(held) + 8
        layers = case.get("layers", 1)
        s.update(table=_table(gen, held, num_pages, max(max(held), 1)), ctx=_ints(ctx), cu=_ints(_cu(new)), total=sum(new),
                 most=max(new), kc=_normal(gen, (layers, num_pages, H, PAGE, D), dt),
                 vc=_normal(gen, (layers, num_pages, H, PAGE, D), dt))
    if case["op"] == "chunk":
        s["q"] = _normal(gen, (s["total"], case["q_heads"], D), dt)
        s["kc"], s["vc"] = s["kc"][0], s["vc"][0]
        s["out"] = torch.empty_like(s["q"])
        s["lse"] = torch.empty((s["total"], case["q_heads"]), dtype=torch.float32, device="cuda")
    elif case["op"] == "append":
        if case["fused"]:  # rows of the fused projection: query heads, then key heads, then value heads
            rows = _normal(gen, (s["total"], case["fused"] + 2 * H, D), dt)
            s["k"], s["v"] = rows[None, :, case["fused"]:case["fused"] + H], rows[None, :, case["fused"] + H:]
        else:
            s["k"], s["v"] = (_normal(gen, (layers, s["total"], H, D), dt) for _ in range(2))
        s["new_ctx"] = torch.empty_like(s["ctx"])
    elif case["op"] == "fork":
        n, k = case["parents"], case["each"]
        rows = n * (1 + k)
        held = [(c + PAGE - 1) // PAGE for c in ctx]
        width = max(held) + (case["new_hi"] + PAGE - 1) // PAGE + 1
        num_pages = sum(held) + rows * (2 + (case["new_hi"] + PAGE - 1) // PAGE) + case["spare"]
        s["table"] = torch.cat([_table(gen, held, num_pages, width),
                                torch.full((n * k, width), -1, dtype=torch.int32, device="cuda")])
        s["held"] = _ints(held + [0] * (n * k))
        s["ctx"] = _ints(ctx + [0] * (n * k))
        s["keep"] = _ints(ctx + [0] * (n * k))
        s["parents"] = _ints([i for i in range(n) for _ in range(k)])
        s["children"] = _ints([n + i for i in range(n * k)])
        r = random.Random(case["lens"] + 1)
        grow = [r.randint(1, case["new_hi"]) for _ in range(rows)]
        s["new"] = _ints([c + g for c, g in zip(ctx + [ctx[i] for i in range(n) for _ in range(k)], grow)])
    elif case["op"] == "compact":
        held = [(c + PAGE - 1) // PAGE for c in ctx]
        num_pages = case["pages"]
        s["table"] = _table(gen, held, num_pages, max(max(held), 1))
        s["held"] = _ints(held)
        s["table_out"], s["live"] = torch.full_like(s["table"], -1), torch.zeros(1, dtype=torch.int32, device="cuda")
        rows = num_pages // 2
    if case["op"] in ("fork", "compact"):
        used = s["table"].flatten()
        s["refs"] = torch.zeros(num_pages + 1, dtype=torch.int32, device="cuda").scatter_add_(
            0, torch.where(used < 0, num_pages, used).long(), torch.ones_like(used))[:num_pages].contiguous()
        s["refs_out"] = torch.zeros_like(s["refs"])
        s["src"], s["dst"] = (torch.full((max(rows, 1),), -1, dtype=torch.int32, device="cuda") for _ in range(2))
        s["count"] = torch.zeros(1, dtype=torch.int32, device="cuda")
        s["kc"], s["vc"] = (_normal(gen, (case["layers"], num_pages, H, PAGE, D), dt) for _ in range(2))
    if own:
        _plan(s)
    return s


# ------------------------------------------------------------------ one pass

def run(s):
    op = s["case"]["op"]
    if own:
        return {"chunk": _own_chunk, "append": _own_append, "fork": _own_fork, "compact": _own_compact}[op](s)
    return {"chunk": _plain_chunk, "append": _plain_append, "fork": _plain_fork, "compact": _plain_compact}[op](s)


def _token_rows(s):
    """Sequence and position within it of every token row."""
    at = torch.arange(s["total"], device="cuda", dtype=torch.int32)
    b = torch.searchsorted(s["cu"][1:].contiguous(), at, right=True)
    return b, at - s["cu"][b]


def _plain_chunk(s):
    c = s["case"]
    B, Hq, H, D, S = c["batch"], c["q_heads"], c["kv_heads"], c["dim"], s["table"].shape[1] * PAGE
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
    if c["window"]:
        seen &= (j > last - c["window"]) | (j < c["sink"])
    scores.masked_fill_(~seen[:, None, None], -math.inf)
    top = scores.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, 0.0, top)
    p = scores.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    v = s["vc"][pages].permute(0, 2, 1, 3, 4).reshape(B, H, S, D).float()
    o = torch.matmul(p.view(B, H, -1, S), v).view(B, H, Hq // H, s["most"], D) / total
    b, at = _token_rows(s)
    o = o.permute(0, 3, 1, 2, 4).reshape(B, s["most"], Hq, D)[b, at]
    lse = (top + total.log())[..., 0].permute(0, 3, 1, 2).reshape(B, s["most"], Hq)[b, at]
    return o.to(s["q"].dtype), lse


def _plain_append(s):
    b, i = _token_rows(s)
    slot = (s["ctx"][b] + i).long()
    page = s["table"][b, slot // PAGE].long()
    s["kc"][:, page, :, slot % PAGE] = s["k"].transpose(0, 1)
    s["vc"][:, page, :, slot % PAGE] = s["v"].transpose(0, 1)
    return s["kc"], s["vc"], s["ctx"] + (s["cu"][1:] - s["cu"][:-1])


def _add(refs, pages, mask, sign):
    """refs[page] += sign for every masked entry of a table."""
    refs.scatter_add_(0, torch.where(mask, pages, 0).flatten().long(), sign * mask.flatten().int())


def _plain_fork(s):
    table, held, ctx, refs = s["table"], s["held"], s["ctx"], s["refs"]
    rows, width = table.shape
    lp = torch.arange(width, device="cuda")
    # release what lies behind the lengths to keep (the children of the step before)
    keep = torch.minimum((s["keep"] + PAGE - 1) // PAGE, held)
    drop = (lp >= keep[:, None]) & (lp < held[:, None])
    _add(refs, table, drop, -1)
    table.masked_fill_(drop, -1)
    held.copy_(keep)
    # fork: the children name their parent's pages
    pages = (ctx[s["parents"]] + PAGE - 1) // PAGE
    take = lp < pages[:, None]
    taken = table[s["parents"]]
    table[s["children"]] = torch.where(take, taken, table[s["children"]])
    _add(refs, taken, take, 1)
    held[s["children"]] = pages
    ctx[s["children"]] = ctx[s["parents"]]
    # reserve: every slot from the context's end to the new length is writable and not shared
    need = (s["new"] + PAGE - 1) // PAGE
    grows = (s["new"] > ctx)[:, None]
    first = (ctx // PAGE)[:, None]
    named = table.clamp(min=0).long()
    shared = grows & (lp >= first) & (lp < torch.minimum(held, need)[:, None]) & (refs[named] > 1)
    here = torch.zeros_like(refs)
    _add(here, table, shared, 1)
    row = torch.arange(rows, device="cuda", dtype=torch.int32)[:, None].expand(rows, width)
    lowest = torch.full((refs.numel() + 1,), rows, dtype=torch.int32, device="cuda").scatter_reduce_(
        0, torch.where(shared, named, refs.numel()).flatten(), row.flatten(), "amin")
    moved = shared & ~((here[named] == refs[named]) & (lowest[named] == row))
    fresh = moved | (grows & (lp >= held[:, None]) & (lp < need[:, None]))
    fresh = fresh & (fresh.sum() <= (refs == 0).sum())
    moved = moved & fresh
    free = torch.argsort((refs != 0).int(), stable=True).int()
    rank = (torch.cumsum(fresh.flatten().int(), 0) - 1).clamp(min=0, max=refs.numel() - 1).view(rows, width)
    page = free[rank]
    copied = moved & (lp == first) & ((ctx % PAGE) != 0)[:, None]
    at = torch.where(copied, torch.cumsum(copied.flatten().int(), 0).view(rows, width) - 1, rows).flatten()
    for_src = torch.cat([s["src"], s["src"][:1]]).scatter_(0, at, table.flatten())[:rows]
    for_dst = torch.cat([s["dst"], s["dst"][:1]]).scatter_(0, at, page.flatten())[:rows]
    s["count"].copy_(copied.sum())
    s["src"].copy_(for_src)
    s["dst"].copy_(for_dst)
    _add(refs, table, moved, -1)
    _add(refs, page, fresh, 1)
    table.copy_(torch.where(fresh, page, table))
    held.copy_(torch.where(fresh.any(1), torch.maximum(held, need), held))
    # copy the ragged tail pages; entries behind the list repeat its first pair
    valid = torch.arange(rows, device="cuda") < s["count"]
    none = s["count"] == 0
    a = torch.where(none, 0, torch.where(valid, s["src"], s["src"][0])).long()
    z = torch.where(none, 0, torch.where(valid, s["dst"], s["dst"][0])).long()
    s["kc"][:, z] = s["kc"][:, a]
    s["vc"][:, z] = s["vc"][:, a]
    return table, held, ctx, refs, s["count"], s["src"], s["dst"], s["kc"], s["vc"]


def _plain_compact(s):
    refs, table = s["refs"], s["table"]
    page = torch.arange(refs.numel(), device="cuda", dtype=torch.int32)
    used = refs > 0
    live = used.sum()
    src, dst = page[used & (page >= live)], page[~used & (page < live)]
    to = page.clone()
    to[src.long()] = dst
    at = torch.arange(table.shape[1], device="cuda")
    s["table_out"].copy_(torch.where(at < s["held"][:, None], to[table.clamp(min=0).long()], table))
    s["refs_out"].copy_(refs)
    s["refs_out"][dst.long()] = refs[src.long()]
    s["refs_out"][src.long()] = 0
    s["src"][:src.numel()] = src
    s["dst"][:dst.numel()] = dst
    s["count"].fill_(src.numel())
    s["live"].copy_(live)
    s["kc"][:, dst.long()] = s["kc"][:, src.long()]
    s["vc"][:, dst.long()] = s["vc"][:, src.long()]
    return s["table_out"], s["refs_out"], s["live"], s["count"], s["src"], s["dst"], s["kc"], s["vc"]


# ------------------------------------------------------------------ the library's calls

def _binding():
    from speculative_decoding_tree_sv_gb300 import binding
    return binding


def _plan(s):
    """What a program keeps between calls: its workspace and, for the attention, the filled parameters."""
    sv, c = _binding(), s["case"]
    if c["op"] == "chunk":
        s["params"] = sv.make_chunk_params(q=s["q"], k_cache=s["kc"], v_cache=s["vc"], block_table=s["table"],
                                           ctx_lens=s["ctx"], cu_tokens=s["cu"], out=s["out"], lse=s["lse"],
                                           max_tokens=s["most"], window_tokens=c["window"], sink_tokens=c["sink"])
        size = sv.sv_chunk_attention_workspace_size(s["params"])
    elif c["op"] == "append":
        size = 256
    else:
        size = sv.sv_pages_workspace_size(s["table"].shape[0], s["refs"].numel())
    s["ws"] = torch.zeros(size, dtype=torch.uint8, device="cuda")
    if c["op"] == "chunk":
        s["params"].workspace, s["params"].workspace_bytes = s["ws"].data_ptr(), size


def _own_chunk(s):
    _binding().sv_chunk_attention(s["params"])
    return s["out"], s["lse"]


def _own_append(s):
    _binding().sv_kv_append(s["k"], s["v"], s["kc"], s["vc"], s["table"], s["ctx"], s["cu"],
                            new_ctx_lens=s["new_ctx"], workspace=s["ws"])
    return s["kc"], s["vc"], s["new_ctx"]


def _own_fork(s):
    sv = _binding()
    sv.sv_pages_release(s["keep"], s["table"], s["held"], s["refs"], workspace=s["ws"])
    sv.sv_pages_fork(s["parents"], s["children"], s["table"], s["ctx"], s["held"], s["refs"], workspace=s["ws"])
    sv.sv_pages_reserve(s["ctx"], s["new"], s["table"], s["held"], s["refs"], s["src"], s["dst"], s["count"],
                        workspace=s["ws"])
    sv.sv_pages_copy(s["kc"], s["vc"], s["src"], s["dst"], s["count"], workspace=s["ws"])
    return s["table"], s["held"], s["ctx"], s["refs"], s["count"], s["src"], s["dst"], s["kc"], s["vc"]


def _own_compact(s):
    sv = _binding()
    sv.sv_pages_compact(s["table"], s["held"], s["refs"], s["table_out"], s["refs_out"], s["src"], s["dst"], s["count"],
                        s["live"], workspace=s["ws"])
    sv.sv_pages_copy(s["kc"], s["vc"], s["src"], s["dst"], s["count"], workspace=s["ws"])
    return s["table_out"], s["refs_out"], s["live"], s["count"], s["src"], s["dst"], s["kc"], s["vc"]


# ------------------------------------------------------------------ work and exact values

def _seen(case, first, n):
    """Keys that the rows first .. first+n-1 attend, summed."""
    if not case["window"]:
        return n * (first + 1) + n * (n - 1) // 2
    total = 0
    for p in range(first, first + n):
        lo = max(0, p - case["window"] + 1)
        total += p + 1 - lo + min(lo, case["sink"])
    return total


def work(case):
    new, ctx = _lengths(case)
    row = case["kv_heads"] * case["dim"] * 2
    if case["op"] == "chunk":
        bytes_ = flops = 0
        for n, c in zip(new, ctx):
            keys = c + n
            if case["window"]:
                lo = max(0, c - case["window"] + 1)
                keys = keys - lo + min(lo, case["sink"])
            bytes_ += keys * 2 * row + n * case["q_heads"] * (case["dim"] * 4 + 4)
            flops += 4 * case["q_heads"] * case["dim"] * _seen(case, c, n)
        return {"bytes": bytes_, "flops": flops}
    if case["op"] == "append":
        return {"bytes": 4 * sum(new) * case["layers"] * row, "flops": 0}
    page = 2 * PAGE * row * case["layers"]  # keys and values of one page, every layer
    if case["op"] == "fork":
        # each child (and not its parent, the lowest row, which keeps the page) copies a ragged tail
        moved = sum(case["each"] for c in ctx if c % PAGE)
        names = sum((c + PAGE - 1) // PAGE for c in ctx) * (1 + case["each"])
        return {"bytes": 2 * moved * page + 8 * names, "flops": 0}
    # an even spread: the pages that live above the live count, on average
    live = sum((c + PAGE - 1) // PAGE for c in ctx)
    moved = live * (case["pages"] - live) / case["pages"]
    return {"bytes": 2 * moved * page + 8 * case["pages"] + 8 * live, "flops": 0}


def exact(case, seed):
    """Attention by its definition in 64 bits, one sequence and key head at a time; the other operators move bits."""
    if case["op"] != "chunk":
        return None
    s = prepare(case, seed)
    new, ctx = _lengths(case)
    Hq, H, D = case["q_heads"], case["kv_heads"], case["dim"]
    G = Hq // H
    out = torch.empty((s["total"], Hq, D), dtype=torch.float64, device="cuda")
    lse = torch.empty((s["total"], Hq), dtype=torch.float64, device="cuda")
    at = 0
    for b, (n, c) in enumerate(zip(new, ctx)):
        pages = s["table"][b, :(c + n + PAGE - 1) // PAGE].long()
        key = torch.arange(c + n, device="cuda")
        me = torch.arange(c, c + n, device="cuda")[:, None]
        hidden = key > me
        if case["window"]:
            hidden = hidden | ((me - key >= case["window"]) & (key >= case["sink"]))
        for h in range(H):
            k = s["kc"][pages, h].reshape(-1, D)[:c + n].double()
            v = s["vc"][pages, h].reshape(-1, D)[:c + n].double()
            for g in range(h * G, (h + 1) * G):
                x = s["q"][at:at + n, g].double() @ k.T / math.sqrt(D)
                x[hidden] = -math.inf
                lse[at:at + n, g] = torch.logsumexp(x, 1)
                out[at:at + n, g] = torch.softmax(x, 1) @ v
        at += n
    return out, lse

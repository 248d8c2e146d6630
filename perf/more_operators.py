"""More operators of a decode step, as a user's program calls them, with their plain forms.

Four of them: the append of new tokens to a paged cache in 8 bits (e4m3 codes,
a power-of-two scale for each block of slots and head), attention over that
cache, attention with a sliding window and first tokens that stay visible
(over either cache), and the choice of tokens from logits by temperature,
top-k, top-p and min-p with given uniform numbers.
"""
import math

import torch

own = False

F16, BF16, F32 = "float16", "bfloat16", "float32"
LEAST, MOST = -96, 120      # exponents of the scales that an append chooses


# ---------------------------------------------------------------- the cases

def _append(name, seqs, new, ctx, heads, kv, dim, rot, interleaved, page, block, dtype):
    """new: the most new tokens of a sequence; ctx: the longest sequence; block: slots that share a scale."""
    return {"name": name, "op": "append", "seqs": seqs, "new": new, "ctx": ctx, "heads": heads, "kv": kv, "dim": dim,
            "rot": rot, "interleaved": interleaved, "page": page, "block": block, "dtype": dtype}


def _attend(name, seqs, new, ctx, heads, kv, dim, page, block, dtype, window=0, sinks=0, tree=False, head_major=False):
    """block: slots that share a scale, 0 for a cache of the queries' type; window: 0 for all that is before a token."""
    return {"name": name, "op": "attend", "seqs": seqs, "new": new, "ctx": ctx, "heads": heads, "kv": kv, "dim": dim,
            "page": page, "block": block, "dtype": dtype, "window": window, "sinks": sinks, "tree": tree,
            "head_major": head_major}


def _sample(name, rows, vocab, top_k, top_p, min_p, dtype, masked):
    """top_k 0, top_p 1, min_p 0: not used; masked: the share of tokens that a grammar has ruled out."""
    return {"name": name, "op": "sample", "rows": rows, "vocab": vocab, "top_k": top_k, "top_p": top_p, "min_p": min_p,
            "dtype": dtype, "masked": masked}


def listed():
    return [
        # a beam batch's single tokens into an 8-bit cache, heads shared: latency
        _append("append8_beams", 16, 1, 3000, 32, 8, 128, 128, False, 32, 32, BF16),
        # a batch of prompts into an 8-bit cache
        _append("append8_prompts", 5, 4001, 4001, 32, 32, 128, 128, False, 64, 16, F16),
        # one token over a short context: the smallest call
        _attend("attend8_one", 1, 1, 700, 32, 32, 128, 16, 16, F16),
        # a beam batch of the 32-head decoder over ragged contexts
        _attend("attend8_beams", 16, 1, 2500, 32, 32, 128, 16, 16, F16),
        # one token over a very long context with shared heads: the split over the context
        _attend("attend8_long", 1, 1, 131071, 32, 8, 128, 64, 64, BF16, head_major=True),
        # a whole prompt of the 32-head decoder over what it has just stored in 8 bits: the largest
        _attend("attend8_prompt", 1, 8192, 8192, 32, 32, 128, 64, 32, F16),
        # single tokens of long streams that keep a window and their first tokens
        _attend("window_beams", 16, 1, 60000, 32, 8, 128, 32, 0, BF16, window=4096, sinks=4),
        # trie candidates over an 8-bit cache through a window
        _attend("window8_tree", 4, 27, 6000, 32, 8, 128, 32, 32, F16, window=1000, sinks=16, tree=True),
        # a long prompt through a window: the diagonal band
        _attend("window_prompt", 2, 6001, 7001, 16, 4, 64, 64, 0, F16, window=1024, sinks=4),
        # one row of the vocabulary product: latency
        _sample("sample_one", 1, 32000, 50, 0.9, 0.0, F32, 0.0),
        # a beam batch under grammar masks, without a bound on the number of candidates
        _sample("sample_beams", 16, 32000, 0, 0.95, 0.02, F16, 0.5),
        # a full serving batch over a large vocabulary, nucleus only
        _sample("sample_batch", 256, 128003, 0, 0.9, 0.0, F32, 0.0),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "attend", "attend", "sample"])
    if op == "sample":
        rows = _log(rng, 1, 256)
        vocab = _log(rng, 1000, min(200000, 256 * 128003 // rows))
        c = _sample("", rows, vocab, rng.choice([0, 0, _log(rng, 1, 2000)]), rng.choice([1.0, 0.5, 0.8, 0.9, 0.95, 0.99]),
                    rng.choice([0.0, 0.0, 0.02, 0.1]), rng.choice([F16, BF16, F32]), rng.choice([0.0, 0.0, 0.5, 0.99]))
        del c["name"]
        return c
    kv = rng.choice([1, 2, 4, 8, 16, 32])
    heads = kv * rng.choice([g for g in (1, 2, 3, 4, 5, 8) if g * kv <= 40])
    dim = rng.choice([64, 80, 96, 128, 128, 256] if heads <= 16 else [64, 80, 96, 128, 128])
    page = rng.choice([8, 16, 32, 64, 128, 256])
    block = rng.choice([b for b in (8, 16, 32, 64, 128) if b <= page])
    dtype = rng.choice([F16, BF16])
    if op == "append":
        seqs = _log(rng, 1, 64)
        new = _log(rng, 1, max(1, 5 * 4001 * 96 * 128 // (seqs * (heads + 2 * kv) * dim)))
        new = min(new, 4001)
        ctx = min(_log(rng, new, 100000), max(new, 400000 // seqs))
        c = _append("", seqs, new, ctx, heads, kv, dim, 2 * (dim // rng.choice([2, 4, 8])), rng.random() < 0.5, page, block, dtype)
    else:
        # within what the plain form's scores and gathered cache may take, and the largest listed case's products
        kind = rng.choice(["one", "tree", "chunk"])
        seqs = _log(rng, 1, 64 if kind == "one" else 8)
        ctx = _log(rng, 1, max(2, min(131071, (1 << 29) // (seqs * kv * dim))))
        new = 1 if kind == "one" else _log(rng, 2, 64) if kind == "tree" else _log(rng, 1, 4096)
        new = max(1, min(new, ctx, (1 << 30) // (seqs * heads * ctx), 130000000000 // (seqs * heads * ctx * dim)))
        how = rng.choice(["8", "8 window", "window"])
        window = _log(rng, 1, 8192) if "window" in how else 0
        c = _attend("", seqs, new, ctx, heads, kv, dim, page, block if "8" in how else 0, dtype, window,
                    rng.choice([0, 1, 4, _log(rng, 1, 200)]) if window else 0, kind == "tree", rng.random() < 0.5)
    del c["name"]
    return c


def _spread(n, low):
    """n shares in (low, 1], the first one 1: the same ones for every seed."""
    return [low + (1.0 - low) * (1.0 - (i * 0.6180339887498949) % 1.0) for i in range(n)]


def _lengths(case):
    """(new tokens, tokens in all) of each sequence."""
    # prompts and chunks are ragged; of single tokens and candidates each sequence has its all
    new = [case["new"]] * case["seqs"] if case["new"] <= 64 else [max(1, int(case["new"] * f)) for f in _spread(case["seqs"], 0.3)]
    return new, [max(n, int(case["ctx"] * f)) for n, f in zip(new, _spread(case["seqs"], 0.2))]


def _ancestors(n):
    """Row i: the candidates that candidate i follows, and itself (each one has two children)."""
    up = []
    for i in range(n):
        up.append(([] if i == 0 else up[(i - 1) // 2]) + [i])
    return up


def _seen(case, n, c):
    """How many slots each new token of a sequence sees, and how many any of them does."""
    window, sinks, old = case["window"] or c + 1, case["sinks"], c - n
    if case["tree"]:
        paths = [len(u) for u in _ancestors(n)]
        low = [max(0, min(old, old + m - window)) for m in paths]
        return [m + old - b + min(b, sinks) for m, b in zip(paths, low)], c - min(low) + min(min(low), sinks)
    low = [max(0, old + i + 1 - window) for i in range(n)]
    return [old + i + 1 - b + min(b, sinks) for i, b in enumerate(low)], c - low[0] + min(low[0], sinks)


def work(case):
    size = {F16: 2, BF16: 2, F32: 4}
    b = size[case["dtype"]]
    if case["op"] == "sample":
        n = case["rows"] * case["vocab"]
        return {"bytes": n * b + 28 * case["rows"], "flops": 4 * n}
    new, ctx = _lengths(case)
    if case["op"] == "append":
        rows, h, kv, d = sum(new), case["heads"], case["kv"], case["dim"]
        turned = rows * (h + kv) * case["rot"]
        scales = sum(n / case["block"] + 1 for n in new) * kv * 2
        return {"bytes": rows * d * (2 * b * h + 2 * kv * (b + 1)) + scales, "flops": 3 * turned + 4 * rows * kv * d}
    seen, read = 0, 0
    for n, c in zip(new, ctx):
        each, some = _seen(case, n, c)
        seen, read = seen + sum(each), read + some
    io = 2 * sum(new) * case["heads"] * case["dim"] * b
    slot = case["dim"] + 1.0 / case["block"] if case["block"] else b * case["dim"]
    return {"bytes": io + 2 * read * case["kv"] * slot, "flops": 4 * case["dim"] * case["heads"] * seen}


# ---------------------------------------------------------------- inputs

def _turns(case):
    """Turns per position of each rotated pair (64 bits)."""
    return 10000.0 ** (-torch.arange(0, case["rot"], 2, dtype=torch.float64) / case["rot"]) / (2 * math.pi)


def _words(n):
    w = torch.zeros(n, -(-n // 32), dtype=torch.int64)
    for i, up in enumerate(_ancestors(n)):
        for j in up:
            w[i, j // 32] |= 1 << (j % 32)
    return w.where(w < 1 << 31, w - (1 << 32)).to(torch.int32)


def _in_8_bits(x, block):
    """x [pages, page, heads, dim] as codes of its shape and scales [pages, page / block, heads]."""
    pages, page, heads, dim = x.shape
    y = x.reshape(pages, page // block, block, heads, dim)
    part, e = torch.frexp(y.abs().amax((2, 4)))
    e = (e - 9 + (part > 0.875)).clamp(LEAST, MOST)
    codes = (y * torch.exp2(-e.float())[:, :, None, :, None]).to(torch.float8_e4m3fn)
    return codes.reshape(x.shape), (e + 127).to(torch.uint8).view(torch.float8_e8m0fnu)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    dev = torch.device("cuda", torch.cuda.current_device())
    dtype = getattr(torch, case["dtype"])
    s = {"case": case}
    if case["op"] == "sample":
        rows, vocab = case["rows"], case["vocab"]
        # a bulk of unlikely tokens and, now and then, a few that the context asks for
        x = 2.0 * torch.randn(rows, vocab, device=dev, generator=g)
        x += 6.0 * (torch.rand(rows, vocab, device=dev, generator=g) < 30.0 / vocab)
        if case["masked"]:
            x.masked_fill_(torch.rand(rows, vocab, device=dev, generator=g) < case["masked"], -math.inf)
        s["x"] = x.to(dtype)
        s["uniform"] = torch.rand(rows, device=dev, generator=g)
        s["temperature"] = 0.5 + torch.rand(rows, device=dev, generator=g)
        s["temperature"][7::8] = 0.0       # requests that want the likeliest token
        s["ids"] = torch.empty(rows, dtype=torch.int32, device=dev)
        s["logprob"] = torch.empty(rows, dtype=torch.float32, device=dev)
        if case["top_k"]:
            s["top_k"] = torch.full((rows,), case["top_k"], dtype=torch.int32, device=dev)
        if case["top_p"] < 1.0:
            s["top_p"] = torch.full((rows,), case["top_p"], device=dev)
        if case["min_p"]:
            s["min_p"] = torch.full((rows,), case["min_p"], device=dev)
        return s
    new, ctx = _lengths(case)
    heads, kv, dim, page, block = case["heads"], case["kv"], case["dim"], case["page"], case["block"]
    tokens, per_seq = sum(new), [-(-c // page) for c in ctx]
    n_pages = sum(per_seq) + 3
    # pages in no order, as a cache in use hands them out
    order = torch.randperm(n_pages, device=dev, generator=g).int()
    s["pages"] = torch.zeros(len(new), max(per_seq), dtype=torch.int32, device=dev)
    at = 0
    for i, n in enumerate(per_seq):
        s["pages"][i, :n] = order[at: at + n]
        at += n
    s["new_start"] = torch.tensor([sum(new[:i]) for i in range(len(new) + 1)], dtype=torch.int32, device=dev)
    s["ctx_len"] = torch.tensor(ctx, dtype=torch.int32, device=dev)
    s["most_new"], s["most_ctx"] = max(new), max(ctx)
    # what the q, k, v product writes: one row a token
    qkv = torch.randn(tokens, heads + 2 * kv, dim, device=dev, generator=g).to(dtype)
    shape = (n_pages, page, kv, dim)
    k, v = (torch.randn(shape, device=dev, generator=g).to(dtype) for _ in range(2))
    if block:
        k, ks = _in_8_bits(k.float(), block)
        v, vs = _in_8_bits(v.float(), block)
        s["scales"] = torch.stack([ks.view(torch.uint8), vs.view(torch.uint8)], -1).contiguous().view(torch.float8_e8m0fnu)
    if case["op"] == "append":
        s["q"], s["k"], s["v"] = qkv[:, :heads], qkv[:, heads: heads + kv], qkv[:, heads + kv:]
        s["q_out"] = torch.empty(tokens, heads, dim, dtype=dtype, device=dev)
        s["turns"] = _turns(case).to(dev)
    else:
        # scores of trained heads reach over a few units
        s["q"] = 2.0 * qkv[:, :heads].contiguous()
        if case["head_major"]:
            k, v = (x.transpose(1, 2).contiguous().transpose(1, 2) for x in (k, v))
        s["out"] = torch.empty(tokens, heads, dim, dtype=dtype, device=dev)
        s["tree"] = _words(case["new"]).repeat(len(new), 1).to(dev) if case["tree"] else None
    s["k_cache"], s["v_cache"] = k, v
    if own:
        import sparse_weight_only_amd as sg
        s["cache"] = sg.PagedCache8.from_tensors(k, v, s["scales"]) if block else sg.PagedCache.from_tensors(k, v)
        s["seqs"] = sg.Sequences(s["new_start"], s["ctx_len"], s["pages"])
        if case["op"] == "append":
            s["rope"] = sg.Rope(case["rot"], base=10000.0, interleaved=case["interleaved"], device=dev)
    return s


# ---------------------------------------------------------------- one pass

def run(s):
    op = s["case"]["op"]
    if op == "append":
        if own:
            s["cache"].append(s["seqs"], s["k"], s["v"], rope=s["rope"], q=s["q"], q_out=s["q_out"])
            return {"q": s["q_out"], "k": s["k_cache"], "v": s["v_cache"], "scales": s["scales"]}
        return _plain_append(s)
    if op == "attend":
        if own:
            return s["cache"].attend(s["seqs"], s["q"], tree=s["tree"], out=s["out"], max_ctx=s["most_ctx"],
                                     window=s["case"]["window"], sinks=s["case"]["sinks"])
        return _plain_attend(s)
    if own:
        import sparse_weight_only_amd as sg
        sg.sample(s["x"], s["uniform"], temperature=s["temperature"], top_k=s.get("top_k"), top_p=s.get("top_p"),
                  min_p=s.get("min_p"), out=s["ids"], logprob=s["logprob"])
        return {"ids": s["ids"], "logprob": s["logprob"]}
    return _plain_sample(s)


def _rows_of(start, n):
    """The ragged list that each of n entries is in."""
    return torch.searchsorted(start[1:], torch.arange(n, device=start.device, dtype=start.dtype), right=True)


def _plain_append(s):
    case = s["case"]
    tokens, rot, page, block, kv, dim = s["q"].shape[0], case["rot"], case["page"], case["block"], case["kv"], case["dim"]
    seq = _rows_of(s["new_start"], tokens)
    slot = s["ctx_len"][seq] - s["new_start"][seq + 1] + torch.arange(tokens, device=seq.device, dtype=torch.int32)
    angle = (slot.double()[:, None] * s["turns"] % 1.0) * (2 * math.pi)
    cos, sin = (f(angle).float()[:, None] for f in (torch.cos, torch.sin))

    def turn(x):
        y = x.float()
        out = y.clone()
        one, two = (slice(0, rot, 2), slice(1, rot, 2)) if case["interleaved"] else (slice(0, rot // 2), slice(rot // 2, rot))
        a, b = y[..., one], y[..., two]
        out[..., one], out[..., two] = a * cos - b * sin, a * sin + b * cos
        return out

    def at_of(q, t):
        """The block, counted through the cache, and the row in it of slots t of sequences q."""
        return s["pages"][q, t // page].long() * (page // block) + (t % page).long() // block, (t % block).long()

    blk, row = at_of(seq, slot)
    seqs = s["ctx_len"].shape[0]
    first = s["ctx_len"] - (s["new_start"][1:] - s["new_start"][:-1])
    head, kept = at_of(torch.arange(seqs, device=seq.device), first)     # each sequence's first block, its older rows
    older = torch.arange(block, device=seq.device) < kept[:, None]
    scales = s["scales"].view(torch.uint8)
    for i, (cache, x) in enumerate(((s["k_cache"], turn(s["k"])), (s["v_cache"], s["v"].float()))):
        codes = cache.view(torch.uint8).view(-1, block, kv, dim)
        e = scales.view(-1, kv, 2)[..., i].int() - 127
        part, need = torch.frexp(x.abs().amax(-1))
        need = (need - 9 + (part > 0.875)).clamp(LEAST, MOST)
        top = torch.full_like(e, LEAST).scatter_reduce_(0, blk[:, None].expand(-1, kv), need, "amax")
        had = torch.full_like(e, LEAST)
        had[head] = e[head].where(kept[:, None] > 0, had[head])
        top = torch.maximum(top, had)
        by = torch.exp2((e[head] - top[head]).float())[:, None, :, None].where(older[:, :, None, None], torch.ones((), device=seq.device))
        codes[head] = (codes[head].view(torch.float8_e4m3fn).float() * by).to(torch.float8_e4m3fn).view(torch.uint8)
        codes[blk, row] = (x * torch.exp2(-top[blk].float())[..., None]).to(torch.float8_e4m3fn).view(torch.uint8)
        scales.view(-1, kv, 2)[blk, :, i] = (top[blk] + 127).to(torch.uint8)
    s["q_out"].copy_(turn(s["q"]))
    return {"q": s["q_out"], "k": s["k_cache"], "v": s["v_cache"], "scales": s["scales"]}


def _plain_attend(s):
    case = s["case"]
    heads, kv, dim, page, block = case["heads"], case["kv"], case["dim"], case["page"], case["block"]
    start, ctx, most_new, most_ctx = s["new_start"], s["ctx_len"], s["most_new"], s["most_ctx"]
    seqs, tokens, dev = ctx.shape[0], s["q"].shape[0], ctx.device
    n_new = start[1:] - start[:-1]
    i = torch.arange(most_new, device=dev)
    rows = (start[:-1, None] + i).clamp(max=tokens - 1)                                   # [S, n]
    q = s["q"][rows].float().reshape(seqs, most_new, kv, heads // kv, dim)
    q = q.permute(0, 2, 3, 1, 4).reshape(seqs, kv, heads // kv * most_new, dim)
    old, window = (ctx - n_new)[:, None], case["window"] or most_ctx + 1
    if case["window"] + case["sinks"] + most_new < most_ctx and case["window"]:
        # each sequence's first slots, and those that a window may reach
        low = (old - window).clamp(min=case["sinks"])
        t = torch.cat([torch.arange(case["sinks"], device=dev).expand(seqs, -1),
                       low + torch.arange(window + most_new, device=dev)], 1)
    else:
        t = torch.arange(most_ctx, device=dev).expand(seqs, -1)
    page_of = s["pages"].long().gather(1, (t // page).clamp(max=s["pages"].shape[1] - 1))  # [S, L]

    def values(c, i):
        x = c.view(torch.uint8)[page_of, t % page].view(c.dtype).float() if block else c[page_of, t % page].float()
        if block:
            x = x * torch.exp2(s["scales"].view(torch.uint8)[page_of, t % page // block][..., i].float() - 127.0)[..., None]
        return x                                                                          # [S, L, kv, dim]

    k, v = values(s["k_cache"], 0), values(s["v_cache"], 1)
    t, old = t[:, None], old[:, None]
    keys = t.shape[-1]
    if s["tree"] is None:
        at = old + i[:, None]
        seen = (t <= at) & ((t > at - window) | (t < case["sinks"]))                      # [S, n, L]
    else:
        j = (t - old).clamp(0, most_new - 1)
        word = s["tree"][rows].gather(2, (j // 32).expand(seqs, most_new, keys))
        path = ((word >> (j % 32)) & 1).bool() & (t >= old) & (t < ctx[:, None, None])
        m = path.sum(-1, keepdim=True)
        seen = path | ((t < old) & ((t >= old + m - window) | (t < case["sinks"])))
    seen = seen[:, None, None].expand(seqs, 1, heads // kv, most_new, keys).reshape(seqs, 1, -1, keys)
    score = torch.matmul(q, k.permute(0, 2, 3, 1).contiguous()).mul_(1.0 / math.sqrt(dim))
    score.masked_fill_(~seen, -math.inf)
    top = score.amax(-1, keepdim=True)
    top = top.where(top > -math.inf, torch.zeros_like(top))
    score.sub_(top).exp_()
    total = score.sum(-1, keepdim=True)
    out = torch.matmul(score, v.permute(0, 2, 1, 3).contiguous()) / total.where(total > 0, torch.ones_like(total))
    out = out.reshape(seqs, kv, heads // kv, most_new, dim).permute(0, 3, 1, 2, 4).reshape(seqs, most_new, heads, dim)
    seq = _rows_of(start, tokens)
    return out[seq, torch.arange(tokens, device=dev) - start[seq]].to(s["q"].dtype)


def _plain_sample(s):
    x, dev = s["x"].double(), s["x"].device
    rows, vocab = x.shape
    t = s["temperature"].double()[:, None]
    greedy = t <= 0
    top = x.amax(-1, keepdim=True)
    p = torch.exp((x - top) / t.where(~greedy, torch.ones_like(t)))
    p = p.where(~greedy, (x == top).double())
    ranked, order = torch.sort(p, dim=-1, descending=True, stable=True)
    place = torch.arange(vocab, device=dev)
    kept = (ranked > 0) & (~greedy | (place < 1))
    if "min_p" in s:
        kept &= ranked >= s["min_p"].double()[:, None]
    if "top_k" in s:
        kept &= place < s["top_k"][:, None]
    ranked = ranked.where(kept, torch.zeros_like(ranked))
    if "top_p" in s:
        run_up = ranked.cumsum(-1)
        kept &= run_up - ranked < s["top_p"].double()[:, None] * run_up[:, -1:]
        ranked = ranked.where(kept, torch.zeros_like(ranked))
    p = torch.zeros_like(p).scatter_(1, order, ranked)
    run_up = p.cumsum(-1)
    total = run_up[:, -1:]
    ids = torch.searchsorted(run_up, s["uniform"].double()[:, None] * total, right=True)
    logprob = torch.log(p.gather(1, ids.clamp(max=vocab - 1)) / total)
    return {"ids": ids[:, 0].int(), "logprob": logprob[:, 0].float()}


# ---------------------------------------------------------------- 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "append":
        return _exact_append(case, s)
    if case["op"] == "attend":
        return _exact_attend(case, s)
    return _exact_sample(case, s)


def _exact_append(case, s):
    """Codes before their rounding, in units of their scales."""
    new, ctx = _lengths(case)
    rot, half, page, block = case["rot"], case["rot"] // 2, case["page"], case["block"]
    freq = [10000.0 ** (-2.0 * j / rot) for j in range(half)]
    dev = s["q"].device
    slots = torch.cat([torch.arange(c - n, c) for n, c in zip(new, ctx)]).to(dev)
    angle = slots.double()[:, None, None] * torch.tensor(freq, dtype=torch.float64, device=dev)
    turner = torch.polar(torch.ones_like(angle), angle)

    def turn(x):
        x = x.double()
        pairs = x[..., :rot].reshape(*x.shape[:-1], half, 2) if case["interleaved"] else \
            x[..., :rot].reshape(*x.shape[:-1], 2, half).transpose(-1, -2)
        z = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * turner)
        z = z if case["interleaved"] else z.transpose(-1, -2)
        return torch.cat([z.reshape(*x.shape[:-1], rot), x[..., rot:]], -1)

    scales = torch.exp2(s["scales"].view(torch.uint8).double() - 127)
    out = {"q": turn(s["q"]), "scales": scales}
    for i, (name, cache, x) in enumerate((("k", s["k_cache"], turn(s["k"])), ("v", s["v_cache"], s["v"].double()))):
        codes = cache.double()
        at = 0
        for q, (n, c) in enumerate(zip(new, ctx)):
            t = c - n
            while t < c:
                end = min(c, (t // block + 1) * block)
                pg, r0, b = int(s["pages"][q, t // page]), t % page, t % page // block
                y = x[at: at + end - t]
                a = y.abs().amax((0, 2)).clamp(min=2.0 ** -200)
                need = torch.ceil(torch.log2(a / 448.0) - 1e-12).clamp(LEAST, MOST)
                if t % block:
                    had = torch.log2(scales[pg, b, :, i])
                    need = torch.maximum(had, need)
                    codes[pg, b * block: r0] *= torch.exp2(had - need)[:, None]
                codes[pg, r0: r0 + end - t] = y * torch.exp2(-need)[:, None]
                scales[pg, b, :, i] = torch.exp2(need)
                at, t = at + end - t, end
        out[name] = codes
    return out


def _exact_attend(case, s):
    new, ctx = _lengths(case)
    group, page, dim, block = case["heads"] // case["kv"], case["page"], case["dim"], case["block"]
    dev = s["q"].device
    out, at = torch.zeros(s["q"].shape, dtype=torch.float64, device=dev), 0
    for i, (n, c) in enumerate(zip(new, ctx)):
        slots = torch.arange(c, device=dev)
        where = s["pages"][i].long()[slots // page]
        old, window = c - n, case["window"] or c + 1
        hidden = torch.zeros(n, c, dtype=torch.bool, device=dev)
        if case["tree"]:
            for j, up in enumerate(_ancestors(n)):
                hidden[j, old:] = True
                hidden[j, [old + a for a in up]] = False
                hidden[j, min(case["sinks"], old): max(0, min(old, old + len(up) - window))] = True
        else:
            ahead = slots - torch.arange(old, c, device=dev)[:, None]
            hidden = (ahead > 0) | ((ahead <= -window) & (slots >= case["sinks"]))
        for h in range(case["kv"]):
            k, v = (b[where, slots % page, h].double() for b in (s["k_cache"], s["v_cache"]))
            if block:
                by = torch.exp2(s["scales"].view(torch.uint8)[where, slots % page // block, h].double() - 127)
                k, v = k * by[:, :1], v * by[:, 1:]
            for hq in range(h * group, (h + 1) * group):
                a = s["q"][at: at + n, hq].double() @ k.t().contiguous() / math.sqrt(dim)
                a.masked_fill_(hidden, -math.inf)
                out[at: at + n, hq] = torch.softmax(a, -1) @ v
        at += n
    return out


def _exact_sample(case, s):
    ids, logprob = [], []
    for r in range(case["rows"]):
        x, t = s["x"][r].double(), float(s["temperature"][r])
        if t <= 0:
            ids.append(int(torch.nonzero(x == x.max())[0]))
            logprob.append(0.0)
            continue
        z = (x - x.max()) / t
        # by descending value and, for equal ones, ascending id
        order = torch.argsort(z, descending=True, stable=True)
        order = order[z[order] > -math.inf]
        if case["min_p"]:
            order = order[z[order] >= math.log(float(s["min_p"][r]))]
        if case["top_k"]:
            order = order[: case["top_k"]]
        p = torch.exp(z[order])
        if case["top_p"] < 1.0:
            need = float(s["top_p"][r]) * float(p.sum())
            order = order[: int((p.cumsum(0) < need).sum()) + 1]
        order = order.sort().values
        p = torch.exp(z[order])
        run_up = p.cumsum(0)
        i = min(int((run_up <= float(s["uniform"][r]) * float(run_up[-1])).sum()), len(order) - 1)
        ids.append(int(order[i]))
        logprob.append(math.log(float(p[i]) / float(run_up[-1])))
    dev = s["x"].device
    return {"ids": torch.tensor(ids, dtype=torch.int32, device=dev), "logprob": torch.tensor(logprob, dtype=torch.float64, device=dev)}

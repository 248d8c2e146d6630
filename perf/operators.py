"""The decode-step operators around the GEMVs, as a user's program calls them, with their plain forms.

Three operators: the append of new tokens to a paged cache with their rotary
positions, the attention of those tokens over the cache, and penalties,
biases and grammar masks on logits.
"""
import math

import torch

own = False

F16, BF16, F32 = "float16", "bfloat16", "float32"


# ---------------------------------------------------------------- the cases

def _append(name, seqs, new, ctx, heads, kv, dim, rot, interleaved, page, dtype, factor=1.0, context=0):
    """new: the most new tokens of a sequence; ctx: the longest sequence, new tokens included."""
    return {"name": name, "op": "append", "seqs": seqs, "new": new, "ctx": ctx, "heads": heads, "kv": kv, "dim": dim,
            "rot": rot, "interleaved": interleaved, "page": page, "dtype": dtype, "factor": factor, "context": context}


def _attend(name, seqs, new, ctx, heads, kv, dim, page, dtype, tree=False, head_major=False):
    return {"name": name, "op": "attend", "seqs": seqs, "new": new, "ctx": ctx, "heads": heads, "kv": kv, "dim": dim,
            "page": page, "dtype": dtype, "tree": tree, "head_major": head_major}


def _logits(name, rows, vocab, hist, bias, masks, dtype, out):
    return {"name": name, "op": "logits", "rows": rows, "vocab": vocab, "hist": hist, "bias": bias, "masks": masks,
            "dtype": dtype, "out": out}


def listed():
    return [
        # one token of one sequence between the q, k, v product and the attention: latency
        _append("append_one", 1, 1, 700, 32, 32, 128, 128, False, 16, F16),
        # a beam batch, shared heads, half of each head rotated, a stretched context
        _append("append_beams", 16, 1, 60000, 32, 8, 128, 64, True, 32, BF16, 8.0, 8192),
        # a batch of prompts
        _append("append_prompts", 5, 4001, 4001, 32, 32, 128, 128, False, 64, F16),
        # one token over a short context: the smallest call
        _attend("attend_one", 1, 1, 700, 32, 32, 128, 16, F16),
        # a beam batch of the 32-head decoder over ragged contexts
        _attend("attend_beams", 16, 1, 2500, 32, 32, 128, 16, F16),
        # one token over a very long context with shared heads: the split over the context
        _attend("attend_long", 1, 1, 131071, 32, 8, 128, 64, BF16, head_major=True),
        # trie candidates verified in one step
        _attend("attend_tree", 4, 27, 6000, 32, 8, 128, 32, F16, tree=True),
        # a chunk of a prompt over what is cached, 64-column heads
        _attend("attend_chunk", 2, 777, 9001, 16, 4, 64, 128, BF16),
        # a whole prompt of the 32-head decoder: the largest
        _attend("attend_prompt", 1, 8192, 8192, 32, 32, 128, 64, F16),
        # one row of the vocabulary product: latency
        _logits("logits_one", 1, 32000, 300, 8, 1, F16, F32),
        # a beam batch, each beam with its own trie node's children
        _logits("logits_beams", 16, 32000, 900, 0, 16, F16, F16),
        # a full serving batch over a large vocabulary with long histories
        _logits("logits_batch", 256, 128003, 4000, 300, 40, F32, F32),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "attend", "logits"])
    if op == "logits":
        rows = _log(rng, 1, 256)
        vocab = _log(rng, 1000, min(200000, 256 * 128003 // rows))
        c = _logits("", rows, vocab, _log(rng, 1, 4000), rng.choice([0, _log(rng, 1, 300)]),
                    rng.choice([0, _log(rng, 1, 40)]), rng.choice([F16, BF16, F32]), rng.choice([F32, "same"]))
        c["out"] = c["dtype"] if c["out"] == "same" else c["out"]
    else:
        kv = rng.choice([1, 2, 4, 8, 16, 32])
        heads = kv * rng.choice([g for g in (1, 2, 3, 4, 5, 8) if g * kv <= 40])
        dim = rng.choice([64, 80, 96, 128, 128, 256] if heads <= 16 else [64, 80, 96, 128, 128])
        page = rng.choice([8, 16, 32, 64, 128, 256])
        dtype = rng.choice([F16, BF16])
        if op == "append":
            seqs = _log(rng, 1, 64)
            new = _log(rng, 1, max(1, 5 * 4001 * 96 * 128 // (seqs * (heads + 2 * kv) * dim)))
            new = min(new, 4001)
            ctx = min(_log(rng, new, 100000), max(new, 400000 // seqs))
            c = _append("", seqs, new, ctx, heads, kv, dim, 2 * (dim // rng.choice([2, 4, 8])), rng.random() < 0.5, page, dtype,
                        rng.choice([1.0, 4.0, 32.0]), rng.choice([0, 4096, 8192]))
        else:
            # within what the plain form's scores and gathered cache may take, and the largest listed case's products
            kind = rng.choice(["one", "tree", "chunk"])
            seqs = _log(rng, 1, 64 if kind == "one" else 8)
            ctx = _log(rng, 1, max(2, min(131071, (1 << 29) // (seqs * kv * dim))))
            new = 1 if kind == "one" else _log(rng, 2, 64) if kind == "tree" else _log(rng, 1, 4096)
            new = max(1, min(new, ctx, (1 << 30) // (seqs * heads * ctx), 130000000000 // (seqs * heads * ctx * dim)))
            c = _attend("", seqs, new, ctx, heads, kv, dim, page, dtype, kind == "tree", rng.random() < 0.5)
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


def work(case):
    size = {F16: 2, BF16: 2, F32: 4}
    b = size[case["dtype"]]
    if case["op"] == "logits":
        n = case["rows"] * case["vocab"]
        return {"bytes": n * (b + size[case["out"]]) + case["rows"] * (4 * case["hist"] + 8 * case["bias"])
                + case["masks"] * 4 * -(-case["vocab"] // 32), "flops": 6 * n}
    new, ctx = _lengths(case)
    if case["op"] == "append":
        cols = sum(new) * (case["heads"] + 2 * case["kv"]) * case["dim"]
        turned = sum(new) * (case["heads"] + case["kv"]) * case["rot"]
        return {"bytes": 2 * b * cols + 4 * case["rot"], "flops": 3 * turned}
    if case["tree"]:
        seen = sum(n * (c - n) + sum(len(u) for u in _ancestors(n)) for n, c in zip(new, ctx))
    else:
        seen = sum(n * (c - n) + n * (n + 1) // 2 for n, c in zip(new, ctx))
    io = 2 * sum(new) * case["heads"] * case["dim"] * b
    return {"bytes": io + 2 * sum(ctx) * case["kv"] * case["dim"] * b, "flops": 4 * case["dim"] * case["heads"] * seen}


# ---------------------------------------------------------------- inputs

def _turns(case):
    """Turns per position of each rotated pair (64 bits), stretched for long contexts."""
    f = 10000.0 ** (-torch.arange(0, case["rot"], 2, dtype=torch.float64) / case["rot"]) / (2 * math.pi)
    if case["factor"] == 1.0:
        return f
    if not case["context"]:
        return f / case["factor"]
    g = ((case["context"] * f - 1.0) / (32.0 - 1.0)).clamp(0.0, 1.0)
    return f * (g + (1.0 - g) / case["factor"])


def _magnitude(case):
    return 1.0 + 0.1 * math.log(case["factor"]) if case["context"] else 1.0


def _words(n):
    w = torch.zeros(n, -(-n // 32), dtype=torch.int64)
    for i, up in enumerate(_ancestors(n)):
        for j in up:
            w[i, j // 32] |= 1 << (j % 32)
    return w.where(w < 1 << 31, w - (1 << 32)).to(torch.int32)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    dev = torch.device("cuda", torch.cuda.current_device())
    dtype = getattr(torch, case["dtype"])
    s = {"case": case}
    if case["op"] == "logits":
        rows, vocab = case["rows"], case["vocab"]
        s["x"] = (3.0 * torch.randn(rows, vocab, device=dev, generator=g)).to(dtype)
        s["out"] = torch.empty(rows, vocab, dtype=getattr(torch, case["out"]), device=dev)
        # text repeats itself: ids of low rank far more often than others
        ids = (vocab * torch.rand(rows * case["hist"], device=dev, generator=g) ** 3).long().clamp(max=vocab - 1)
        s["history"] = ids.int()
        s["history_start"] = torch.arange(rows + 1, device=dev, dtype=torch.int32) * case["hist"]
        s["prompt"] = (case["hist"] * torch.rand(rows, device=dev, generator=g)).int()
        s["repetition"] = 1.0 + 0.3 * torch.rand(rows, device=dev, generator=g)
        s["frequency"] = 0.5 * torch.rand(rows, device=dev, generator=g)
        s["presence"] = 0.5 * torch.rand(rows, device=dev, generator=g)
        if case["bias"]:
            n = case["bias"]
            # distinct ids in each row
            at = torch.rand(rows, n, device=dev, generator=g)
            s["bias_ids"] = ((torch.arange(n, device=dev) + at) * (vocab / n)).int().clamp(max=vocab - 1).reshape(-1)
            s["bias_values"] = 2.0 * torch.randn(rows * n, device=dev, generator=g)
            s["bias_start"] = torch.arange(rows + 1, device=dev, dtype=torch.int32) * n
        if case["masks"]:
            s["masks"] = torch.randint(-(1 << 31), 1 << 31, (case["masks"], -(-vocab // 32)), device=dev, generator=g).int()
            s["mask_of"] = (torch.arange(rows, device=dev) % (case["masks"] + 1) - int(case["masks"] > 1)).int()
            s["mask_of"] = s["mask_of"].clamp(max=case["masks"] - 1)
        return s
    new, ctx = _lengths(case)
    heads, kv, dim, page = case["heads"], case["kv"], case["dim"], case["page"]
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
    if case["op"] == "append":
        s["q"], s["k"], s["v"] = qkv[:, :heads], qkv[:, heads: heads + kv], qkv[:, heads + kv:]
        s["q_out"] = torch.empty(tokens, heads, dim, dtype=dtype, device=dev)
        s["k_cache"] = torch.zeros(n_pages, page, kv, dim, dtype=dtype, device=dev)
        s["v_cache"] = torch.zeros(n_pages, page, kv, dim, dtype=dtype, device=dev)
        s["turns"], s["magnitude"] = _turns(case).to(dev), _magnitude(case)
    else:
        # scores of trained heads reach over a few units
        s["q"] = 2.0 * qkv[:, :heads].contiguous()
        shape = (n_pages, kv, page, dim) if case["head_major"] else (n_pages, page, kv, dim)
        s["k_cache"], s["v_cache"] = (torch.randn(shape, device=dev, generator=g, dtype=torch.float32).to(dtype) for _ in range(2))
        if case["head_major"]:
            s["k_cache"], s["v_cache"] = s["k_cache"].transpose(1, 2), s["v_cache"].transpose(1, 2)
        s["out"] = torch.empty(tokens, heads, dim, dtype=dtype, device=dev)
        s["tree"] = _words(case["new"]).repeat(len(new), 1).to(dev) if case["tree"] else None
    if own:
        import sparse_weight_only_amd as sg
        s["cache"] = sg.PagedCache.from_tensors(s["k_cache"], s["v_cache"])
        s["seqs"] = sg.Sequences(s["new_start"], s["ctx_len"], s["pages"])
        if case["op"] == "append":
            s["rope"] = sg.Rope(case["rot"], base=10000.0, interleaved=case["interleaved"], factor=case["factor"],
                                context=case["context"], low=1.0, high=32.0, magnitude=s["magnitude"], device=dev)
    return s


# ---------------------------------------------------------------- one pass

def run(s):
    op = s["case"]["op"]
    if op == "append":
        if own:
            s["cache"].append(s["seqs"], s["k"], s["v"], rope=s["rope"], q=s["q"], q_out=s["q_out"])
            return {"q": s["q_out"], "k": s["k_cache"], "v": s["v_cache"]}
        return _plain_append(s)
    if op == "attend":
        if own:
            return s["cache"].attend(s["seqs"], s["q"], tree=s["tree"], out=s["out"], max_ctx=s["most_ctx"])
        return _plain_attend(s)
    if own:
        import sparse_weight_only_amd as sg
        return sg.adjust_logits(
            s["x"], out=s["out"], history=s["history"], history_start=s["history_start"], prompt_len=s["prompt"],
            repetition=s["repetition"], frequency=s["frequency"], presence=s["presence"], bias_ids=s.get("bias_ids"),
            bias_values=s.get("bias_values"), bias_start=s.get("bias_start"), masks=s.get("masks"), mask_row=s.get("mask_of"))
    return _plain_logits(s)


def _rows_of(start, n):
    """The ragged list that each of n entries is in."""
    return torch.searchsorted(start[1:], torch.arange(n, device=start.device, dtype=start.dtype), right=True)


def _plain_append(s):
    case = s["case"]
    tokens, rot = s["q"].shape[0], case["rot"]
    seq = _rows_of(s["new_start"], tokens)
    slot = s["ctx_len"][seq] - s["new_start"][seq + 1] + torch.arange(tokens, device=seq.device, dtype=torch.int32)
    angle = (slot.double()[:, None] * s["turns"] % 1.0) * (2 * math.pi)
    cos, sin = (s["magnitude"] * f(angle).float()[:, None] for f in (torch.cos, torch.sin))

    def turn(x):
        y = x.float()
        out = y.clone()
        one, two = (slice(0, rot, 2), slice(1, rot, 2)) if case["interleaved"] else (slice(0, rot // 2), slice(rot // 2, rot))
        a, b = y[..., one], y[..., two]
        out[..., one], out[..., two] = a * cos - b * sin, a * sin + b * cos
        return out.to(x.dtype)

    page, row = s["pages"][seq, slot // case["page"]].long(), (slot % case["page"]).long()
    s["k_cache"][page, row] = turn(s["k"])
    s["v_cache"][page, row] = s["v"]
    s["q_out"].copy_(turn(s["q"]))
    return {"q": s["q_out"], "k": s["k_cache"], "v": s["v_cache"]}


def _plain_attend(s):
    case = s["case"]
    heads, kv, dim, page = case["heads"], case["kv"], case["dim"], case["page"]
    start, ctx, most_new, most_ctx = s["new_start"], s["ctx_len"], s["most_new"], s["most_ctx"]
    seqs, tokens, dev = ctx.shape[0], s["q"].shape[0], ctx.device
    n_new = start[1:] - start[:-1]
    i = torch.arange(most_new, device=dev)
    rows = (start[:-1, None] + i).clamp(max=tokens - 1)                                   # [S, n]
    q = s["q"][rows].float().reshape(seqs, most_new, kv, heads // kv, dim)
    q = q.permute(0, 2, 3, 1, 4).reshape(seqs, kv, heads // kv * most_new, dim)
    k, v = (c[s["pages"][:, : -(-most_ctx // page)].long()].reshape(seqs, -1, kv, dim)[:, :most_ctx].float()
            for c in (s["k_cache"], s["v_cache"]))
    t = torch.arange(most_ctx, device=dev)
    old = (ctx - n_new)[:, None, None]
    if s["tree"] is None:
        seen = t <= old + i[:, None]                                                      # [S, n, L]
    else:
        j = (t - old).clamp(0, most_new - 1)
        word = s["tree"][rows].gather(2, (j // 32).expand(seqs, most_new, most_ctx))
        seen = (t < old) | ((t < ctx[:, None, None]) & ((word >> (j % 32)) & 1).bool())
    seen = seen[:, None, None].expand(seqs, 1, heads // kv, most_new, most_ctx).reshape(seqs, 1, -1, most_ctx)
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


def _plain_logits(s):
    case = s["case"]
    rows, vocab = case["rows"], case["vocab"]
    x, dev = s["x"].float(), s["x"].device
    ids = s["history"].long()
    row = _rows_of(s["history_start"], ids.shape[0])
    behind = torch.arange(ids.shape[0], device=dev) - s["history_start"][row] >= s["prompt"][row]
    seen = torch.zeros(rows * vocab, dtype=torch.int32, device=dev)
    count = torch.zeros(rows * vocab, dtype=torch.int32, device=dev)
    seen.index_add_(0, row * vocab + ids, torch.ones_like(s["history"]))
    count.index_add_(0, row * vocab + ids, behind.int())
    seen, count = seen.view(rows, vocab) > 0, count.view(rows, vocab)
    r = s["repetition"][:, None]
    x = torch.where(seen, torch.where(x > 0, x / r, x * r), x)
    x = x - s["frequency"][:, None] * count - s["presence"][:, None] * (count > 0)
    if case["bias"]:
        at = _rows_of(s["bias_start"], s["bias_ids"].shape[0]) * vocab + s["bias_ids"].long()
        x.view(-1)[at] += s["bias_values"]
    if case["masks"]:
        of = s["mask_of"].long()
        bits = (s["masks"][of.clamp(min=0)][:, :, None] >> torch.arange(32, device=dev, dtype=torch.int32)) & 1
        allowed = bits.view(rows, -1)[:, :vocab].bool() | (of < 0)[:, None]
        x = x.masked_fill(~allowed, -math.inf)
    return x.to(s["out"].dtype)


# ---------------------------------------------------------------- 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "append":
        return _exact_append(case, s)
    if case["op"] == "attend":
        return _exact_attend(case, s)
    return _exact_logits(case, s)


def _exact_append(case, s):
    new, ctx = _lengths(case)
    rot, half, page = case["rot"], case["rot"] // 2, case["page"]
    freq = []
    for j in range(half):
        f = 10000.0 ** (-2.0 * j / rot)
        if case["factor"] != 1.0 and case["context"]:
            g = min(1.0, max(0.0, (case["context"] * f / (2 * math.pi) - 1.0) / 31.0))
            f *= g + (1.0 - g) / case["factor"]
        else:
            f /= case["factor"]
        freq.append(f)
    slots = torch.cat([torch.arange(c - n, c) for n, c in zip(new, ctx)]).to(s["q"].device)
    where = torch.cat([s["pages"][i].long().repeat_interleave(page)[c - n: c] for i, (n, c) in enumerate(zip(new, ctx))])
    angle = slots.double()[:, None, None] * torch.tensor(freq, dtype=torch.float64, device=slots.device)
    turner = s["magnitude"] * torch.polar(torch.ones_like(angle), angle)

    def turn(x):
        x = x.double()
        pairs = x[..., :rot].reshape(*x.shape[:-1], half, 2) if case["interleaved"] else \
            x[..., :rot].reshape(*x.shape[:-1], 2, half).transpose(-1, -2)
        z = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * turner)
        z = z if case["interleaved"] else z.transpose(-1, -2)
        return torch.cat([z.reshape(*x.shape[:-1], rot), x[..., rot:]], -1)

    k, v = s["k_cache"].double(), s["v_cache"].double()
    k[where, slots % page], v[where, slots % page] = turn(s["k"]), s["v"].double()
    return {"q": turn(s["q"]), "k": k, "v": v}


def _exact_attend(case, s):
    new, ctx = _lengths(case)
    group, page, dim = case["heads"] // case["kv"], case["page"], case["dim"]
    out, at = torch.zeros(s["q"].shape, dtype=torch.float64, device=s["q"].device), 0
    for i, (n, c) in enumerate(zip(new, ctx)):
        slots = torch.arange(c, device=out.device)
        where = s["pages"][i].long()[slots // page]
        late = torch.zeros(n, c, dtype=torch.bool, device=out.device)
        if case["tree"]:
            own_keys = torch.ones(n, n, dtype=torch.bool)
            for j, up in enumerate(_ancestors(n)):
                own_keys[j, up] = False
            late[:, c - n:] = own_keys.to(out.device)
        else:
            late[:, c - n:] = torch.ones(n, n, dtype=torch.bool, device=out.device).triu(1)
        for h in range(case["kv"]):
            k, v = (b[where, slots % page, h].double() for b in (s["k_cache"], s["v_cache"]))
            for hq in range(h * group, (h + 1) * group):
                a = s["q"][at: at + n, hq].double() @ k.t().contiguous() / math.sqrt(dim)
                a.masked_fill_(late, -math.inf)
                out[at: at + n, hq] = torch.softmax(a, -1) @ v
        at += n
    return out


def _exact_logits(case, s):
    rows, vocab = case["rows"], case["vocab"]
    x = s["x"].double()
    ids = s["history"].long().view(rows, -1)
    turn = torch.arange(case["hist"], device=x.device).expand(rows, -1) >= s["prompt"][:, None]
    count = torch.zeros(rows, vocab, dtype=torch.float64, device=x.device).scatter_add_(1, ids, turn.double())
    seen = torch.zeros(rows, vocab, dtype=torch.bool, device=x.device).scatter_(1, ids, True)
    r, f, p = (s[n].double()[:, None] for n in ("repetition", "frequency", "presence"))
    x = torch.where(seen & (x > 0), x / r, torch.where(seen, x * r, x)) - f * count - p * (count > 0)
    if case["bias"]:
        x.scatter_add_(1, s["bias_ids"].long().view(rows, -1), s["bias_values"].double().view(rows, -1))
    if case["masks"]:
        tokens = torch.arange(vocab, device=x.device)
        for i, m in enumerate(s["mask_of"].tolist()):
            if m >= 0:
                x[i, (s["masks"][m][tokens // 32] >> (tokens % 32).int()) & 1 == 0] = -math.inf
    return x

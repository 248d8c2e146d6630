"""FP64 definitions of the operators between the GEMVs of a decode step.

Each is written per token or per row, in the order of its definition, with
plain loops: rotary positions, the append to a paged cache (of the values'
own type, or in 8 bits), attention over it, penalties, biases and masks on
logits, and the choice of tokens. ``attend`` also returns the mean absolute
value that its error bound is relative to.
"""
from __future__ import annotations

import math

import numpy as np


def rope_turns(rot, base=10000.0, factor=1.0, context=0.0, low=1.0, high=32.0):
    out = []
    for j in range(rot // 2):
        f = base ** (-2.0 * j / rot)
        keep = 0.0
        if context > 0:
            keep = min(1.0, max(0.0, (context * f / (2 * math.pi) - low) / (high - low)))
        out.append(f * (keep + (1.0 - keep) / factor) / (2 * math.pi))
    return np.array(out)


def rope(x, positions, turns, interleaved=False, magnitude=1.0):
    """x [T, H, D] (any float type) -> FP64 [T, H, D]."""
    y = np.asarray(x, np.float64).copy()
    half = len(turns)
    for t, pos in enumerate(positions):
        for j in range(half):
            # whole turns are taken off exactly before the angle is formed
            a = 2 * math.pi * math.remainder(int(pos) * float(turns[j]), 1.0)
            i0, i1 = (2 * j, 2 * j + 1) if interleaved else (j, j + half)
            u, w = y[t, :, i0].copy(), y[t, :, i1].copy()
            y[t, :, i0] = magnitude * (u * math.cos(a) - w * math.sin(a))
            y[t, :, i1] = magnitude * (u * math.sin(a) + w * math.cos(a))
    return y


def slots(new_start, ctx_len):
    """[(sequence, new token of it, slot)] for each row in [new_start[0], new_start[-1]), by row."""
    out = {}
    for s in range(len(ctx_len)):
        n = int(new_start[s + 1]) - int(new_start[s])
        for i in range(n):
            out[int(new_start[s]) + i] = (s, i, int(ctx_len[s]) - n + i)
    return out


def append(k_cache, v_cache, k, v, new_start, ctx_len, pages):
    """Copies rows of k and v (values as stored) into copies of the caches [pages, page, H, D]."""
    kc, vc = k_cache.copy(), v_cache.copy()
    n_pages, page = kc.shape[:2]
    for row, (s, _, slot) in slots(new_start, ctx_len).items():
        if slot < 0 or slot >= page * pages.shape[1]:
            continue
        at = int(pages[s, slot // page])
        if 0 <= at < n_pages:
            kc[at, slot % page], vc[at, slot % page] = k[row], v[row]
    return kc, vc


# The values of e4m3's codes 0..126 (127 is NaN): sign apart, 4 exponent and 3
# mantissa bits, subnormals in steps of 2^-9.
E4M3 = np.array([(m / 8 * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7)) for e in range(16) for m in range(8)][:127])


def to_e4m3(x):
    """Codes of FP64 values up to 448 in magnitude, to the nearest, ties to the even code; what is not finite: 0x7f."""
    x = np.asarray(x, np.float64)
    a = np.where(np.isfinite(x), np.abs(x), 0.0)
    assert a.max(initial=0.0) <= 448.0
    lo = np.clip(np.searchsorted(E4M3, a, side="right") - 1, 0, 125)
    mid = (E4M3[lo] + E4M3[lo + 1]) / 2
    code = np.where(a > mid, lo + 1, np.where(a < mid, lo, lo + lo % 2))
    return np.where(np.isfinite(x), code | np.where(np.signbit(x), 128, 0), 0x7F).astype(np.uint8)


def of_e4m3(codes):
    codes = np.asarray(codes)
    v = np.append(E4M3, np.nan)[codes & 127]
    return np.where(codes & 128, -v, v)


def values8(codes, scales, which):
    """FP64 values of codes [pages, page, H, D] with scale bytes [pages, blocks, H, 2]; which: 0 for K, 1 for V."""
    each = codes.shape[1] // scales.shape[1]
    return of_e4m3(codes) * 2.0 ** (np.repeat(scales[..., which].astype(int), each, 1) - 127)[..., None]


def exponent8(a):
    """The least e from -96 to 120 with a <= 448 2^e."""
    e = -96
    while a > 448.0 * 2.0 ** e and e < 120:
        e += 1
    return e


def append8(codes, scales, x, which, new_start, ctx_len, pages):
    """Rows x [T, H, D] (FP64, k turned) into copies of codes [pages, page, H, D] and scale bytes [pages, blocks, H, 2]."""
    codes, scales = codes.copy(), scales.copy()
    n_pages, page, H, _ = codes.shape
    each = page // scales.shape[1]
    rows = {}                                                   # block -> its new rows
    for row, (s, i, slot) in slots(new_start, ctx_len).items():
        if 0 <= slot < page * pages.shape[1] and 0 <= int(pages[s, slot // page]) < n_pages:
            rows.setdefault((int(pages[s, slot // page]), slot % page // each), []).append((slot % page % each, row))
    for (at, blk), new in rows.items():
        first = min(new)[0]
        for h in range(H):
            y = np.stack([x[row, h] for _, row in new])
            e = exponent8(np.abs(y[np.isfinite(y)]).max(initial=0.0))
            if first > 0:
                was = int(scales[at, blk, h, which]) - 127
                e = max(e, was)
                old = slice(blk * each, blk * each + first)
                codes[at, old, h] = to_e4m3_keeping_nan(codes[at, old, h], was - e)
            scales[at, blk, h, which] = e + 127
            for r, row in new:
                codes[at, blk * each + r, h] = to_e4m3(x[row, h] * 2.0 ** -e)
    return codes, scales


def to_e4m3_keeping_nan(codes, by):
    """Codes times 2^by (by <= 0), rounded; a NaN stays as it is."""
    return codes if by == 0 else np.where(codes & 127 == 127, codes, to_e4m3(np.nan_to_num(of_e4m3(codes)) * 2.0 ** by))


def attend(q, k_cache, v_cache, new_start, ctx_len, pages, scale, tree=None, window=0, sinks=0):
    """(out, mean, worst, keys): FP64 attention [T, Hq, D] (zeros where no key is
    visible, NaN for rows of no sequence), sum p |v| / sum p, the largest
    sum_d |q_d k_d| scale of each (row, head), and its number of visible keys."""
    T, Hq, D = q.shape
    n_pages, page, H, _ = k_cache.shape
    out = np.full((T, Hq, D), np.nan)
    mean, worst, keys = np.zeros((T, Hq, D)), np.zeros((T, Hq)), np.zeros((T, Hq), int)
    for row, (s, i, slot) in slots(new_start, ctx_len).items():
        ctx = min(int(ctx_len[s]), pages.shape[1] * page)
        old = ctx - (int(new_start[s + 1]) - int(new_start[s]))
        see = []
        low = old + i + 1 - window                  # the first slot that a window leaves, the sinks apart
        if tree is not None:
            low = min(old, old - window + sum(int(tree[row, j // 32]) >> (j % 32) & 1 for j in range(min(ctx - old, 32 * tree.shape[1]))))
        for t in range(ctx):
            if window and sinks <= t < low:
                continue
            if not 0 <= int(pages[s, t // page]) < n_pages:
                continue
            if tree is None:
                ok = t <= old + i
            else:
                j = t - old                  # a token below slot 0 sees nothing, whatever its bits
                ok = old + i >= 0 and (j < 0 or (j < 32 * tree.shape[1] and bool(int(tree[row, j // 32]) >> (j % 32) & 1)))
            if ok:
                see.append((int(pages[s, t // page]), t % page))
        out[row] = 0.0
        if not see:
            continue
        at = tuple(np.array(see).T)
        for h in range(Hq):
            kk = k_cache[at[0], at[1], h // (Hq // H)].astype(np.float64)
            vv = v_cache[at[0], at[1], h // (Hq // H)].astype(np.float64)
            qq = q[row, h].astype(np.float64)
            a = scale * (kk @ qq)
            p = np.exp(a - a.max())
            out[row, h] = p @ vv / p.sum()
            mean[row, h] = p @ np.abs(vv) / p.sum()
            worst[row, h] = scale * (np.abs(kk) @ np.abs(qq)).max()
            keys[row, h] = len(see)
    return out, mean, worst, keys


def adjust_logits(x, history=None, prompt_len=None, repetition=None, frequency=None, presence=None, bias=None, masks=None):
    """x [R, V]; history, bias: a list of ids, or of (id, value), for each row;
    masks: a list of allowed-token truth values (or None) for each row. FP64."""
    y = np.asarray(x, np.float64).copy()
    rows, vocab = y.shape
    for b in range(rows):
        ids = list(history[b]) if history is not None else []
        cut = 0 if prompt_len is None else int(prompt_len[b])
        for v in sorted({int(i) for i in ids if 0 <= i < vocab}):
            n = sum(1 for i in ids[max(cut, 0):] if i == v)
            r = 1.0 if repetition is None else float(repetition[b])
            y[b, v] = y[b, v] / r if y[b, v] > 0 else y[b, v] * r
            if n:
                y[b, v] -= (0.0 if frequency is None else float(frequency[b])) * n
                y[b, v] -= 0.0 if presence is None else float(presence[b])
        if bias is not None:
            done = set()                     # an id given twice: the first one holds
            for v, a in bias[b]:
                if 0 <= v < vocab and int(v) not in done:
                    done.add(int(v))
                    y[b, int(v)] += float(a)
        if masks is not None and masks[b] is not None:
            y[b, ~np.asarray(masks[b], bool)] = -np.inf
    return y


def sample(x, uniform, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0):
    """(token, ln of its share, the least distance of a border from where it would decide otherwise) of one row of logits, FP64."""
    x = np.asarray(x, np.float64)
    x = np.where(np.isnan(x), -np.inf, x)
    if x.max(initial=-np.inf) == -np.inf:
        return -1, -math.inf, math.inf
    if not temperature > 0:
        return int(x.argmax()), 0.0, math.inf
    order = sorted((i for i in range(len(x)) if x[i] > -np.inf), key=lambda i: (-x[i], i))
    with np.errstate(invalid="ignore"):
        p = np.where(x == x.max(), 1.0, np.exp((x - x.max()) / temperature))
    far = math.inf
    if min_p > 0:
        far = min([far] + [abs(p[i] - min(min_p, 1.0)) for i in order if p[i] != 1.0])
        order = [i for i in order if p[i] >= min(min_p, 1.0)]
    if top_k > 0:
        order = order[:top_k]
    if top_p < 1:
        total, run = math.fsum(p[i] for i in order), 0.0
        for n, i in enumerate(order):
            run += p[i]
            far = min(far, abs(run / total - top_p))
            if run >= max(top_p, 0.0) * total:
                break
        order = order[: n + 1]
    order.sort()
    total = math.fsum(p[i] for i in order)
    run = np.cumsum([p[i] for i in order]) / total
    u = min(max(uniform, 0.0), 1.0 - 2.0 ** -53) if uniform == uniform else 0.0
    at = min(int((run <= u).sum()), len(order) - 1)
    far = min([far] + [abs(r - u) for r in run[:-1]])
    return order[at], math.log(p[order[at]] / total), far

"""FP64 definitions of the operators between the GEMVs of a decode step.

Each is written per token or per row, in the order of its definition, with
plain loops: rotary positions, the append to a paged cache, attention over
it, and penalties, biases and masks on logits. ``attend`` also returns the
mean absolute value that its error bound is relative to.
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


def attend(q, k_cache, v_cache, new_start, ctx_len, pages, scale, tree=None):
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
        for t in range(ctx):
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

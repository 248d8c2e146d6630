"""Decode-step operators where they can go wrong between the cases of the parity
tests. Tolerances as those count them (u the type's half step, e = 2^-24),
except where a test counts its own.
"""
import numpy as np
import pytest

import sparse_weight_only_amd as sg
from gpu_util import say
from oracle import decode as odec
from test_gpu_decode import A, BF16, E, F16, F32, U, Setup, host, ints

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _device():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    sg.lib()


# ---------------------------------------------------------- empty tensors

@pytest.mark.parametrize("n,ctx", [([4], [4]), ([3, 0, 5], [40, 7, 5]), ([90], [100]), ([40], [1100])])
def test_tree_without_words(n, ctx):
    """No word: no new token sees a new token, as bits past the words count as 0."""
    say("case tree without words", n, ctx)
    s = Setup(n, ctx, 16, 4, 2, 64, F16, 31)
    want = s.want(tree=np.zeros((s.tokens, 0), np.uint32))
    out = s.cache.attend(s.seqs, s.q, tree=torch.zeros(s.tokens, 0, dtype=torch.int32, device="cuda"))
    s.check(out, want, "no words")
    for q in range(len(n)):
        if n[q] == ctx[q]:
            assert (host(out)[s.new_start[q]: s.new_start[q + 1]] == 0).all()


def test_no_tokens():
    """Nothing is done, whatever else is given."""
    say("case no tokens")
    cache = sg.PagedCache(4, 16, 2, 64)
    seqs = sg.Sequences(ints([0, 0]), ints([5]), ints([[0]]))
    none = torch.zeros(0, 2, 64, dtype=F16, device="cuda")
    for words in (0, 2):
        assert cache.attend(seqs, none, tree=torch.zeros(0, words, dtype=torch.int32, device="cuda")).shape == (0, 2, 64)
    rope, at = sg.Rope(64), ints([])
    assert cache.append(seqs, none, none, rope=rope, q=none, positions=at).shape == (0, 2, 64)
    assert rope.apply(none, at).shape == (0, 2, 64)


def test_no_rows():
    """Nothing is done, whatever else is given."""
    say("case no rows")
    x, masks = torch.zeros(0, 50, device="cuda"), ints([[-1, -1], [3, 0]])
    empty = torch.zeros(0, device="cuda")
    for kw in (dict(masks=masks, mask_row=ints([])), dict(masks=masks[:0]), dict(masks=masks[:0], mask_row=ints([])),
               dict(history=ints([]), history_start=ints([0]), prompt_len=ints([]), repetition=empty, frequency=empty, presence=empty),
               dict(bias_ids=ints([]), bias_values=empty, bias_start=ints([0]))):
        assert sg.adjust_logits(x, **kw).shape == (0, 50)


def test_mask_tables_that_are_empty_or_short_are_refused():
    """A row without its mask would be left unmasked."""
    say("case short mask tables")
    x, masks = torch.zeros(3, 50, device="cuda"), torch.zeros(5, 2, dtype=torch.int32, device="cuda")
    for m in (masks[:0], masks[:2], masks[:4]):
        with pytest.raises(ValueError if len(m) == 0 else sg.SgemvError):
            sg.adjust_logits(x, masks=m)
    with pytest.raises(ValueError, match="no mask"):
        sg.adjust_logits(x, masks=masks[:0], mask_row=ints([0, 0, 0]))
    assert np.isneginf(host(sg.adjust_logits(x, masks=masks[:3]))).all()


# ------------------------------------------- candidates below slot 0

@pytest.mark.parametrize("n,ctx", [([4], [2]), ([4, 2, 3], [2, 30, 0]), ([70, 3], [60, 90]), ([300], [17]), ([40, 30], [1090, 9])])
def test_candidates_below_slot_zero_see_nothing(n, ctx):
    """Lengths shorter than the new tokens: those without a slot get zeros, the others what their bits say."""
    say("case tree below slot 0", n, ctx)
    per = -(-max(ctx + [1]) // 16)
    s = Setup(n, ctx, 16, 4, 2, 64, F16, 32, per_seq=per)
    words = (max(n) + 31) // 32
    tree = np.random.default_rng(33).integers(0, 2 ** 32, (s.tokens, words), dtype=np.uint32)
    out = s.cache.attend(s.seqs, s.q, tree=torch.from_numpy(tree.view(np.int32)).cuda())
    s.check(out, s.want(tree=tree), "below slot 0")
    for q in range(len(n)):
        a = int(s.new_start[q])
        assert (host(out)[a: a + max(0, n[q] - ctx[q])] == 0).all(), "a token without a slot saw a key"


# ------------------------------------------------- infinite keys

@pytest.mark.parametrize("n,ctx", [([1], [200]), ([3], [90]), ([90], [1200]), ([300], [400])])
def test_keys_of_minus_infinity(n, ctx):
    """A score of -inf is a weight of 0 like any other: it leaves the others as
    they are, and times an infinite value it is no number, in every kernel."""
    say("case infinite keys", n)
    s = Setup(n, ctx, 16, 2, 1, 64, F16, 38)
    s.q[..., 7] = s.q[..., 7].abs() + 0.5
    slot = ctx[0] - n[0] // 2 - 1
    at = int(s.pages[0, slot // 16]), slot % 16
    s.kc[at[0], at[1], 0, 7] = float("-inf")
    with np.errstate(invalid="ignore"):
        want = s.want()
    worst = want[2]
    worst[~np.isfinite(worst)] = 64 * 5.0 * 5.0 * 64 ** -0.5   # of the finite scores: at most this
    got = s.cache.attend(s.seqs, s.q)
    s.check(got, want, "-inf")
    s.vc[at[0], at[1], 0, 5] = float("inf")
    got = host(s.cache.attend(s.seqs, s.q))
    sees = np.arange(ctx[0] - n[0], ctx[0]) >= slot
    assert np.isnan(got[sees][:, :, 5]).all() and np.isfinite(got[~sees]).all() and np.isfinite(np.delete(got, 5, 2)).all()
    s.kc[..., 7] = float("-inf")
    s.vc[at[0], at[1], 0, 5] = 0.0
    assert (host(s.cache.attend(s.seqs, s.q)) == 0).all(), "all scores are -inf"


# ------------------------------------- weights far below the largest

# what, dim, new tokens, slots, expected max, the plan's (tile rows, parts), strong keys: one in each wave's walk
# (few rows: waves take 32-key blocks in turn; halves: each half of the first block of a part)
FAR = [
    ("few", 64, 1, 1 << 20, 1, (16, 1), [32 * w for w in range(8)]),
    ("few", 256, 1, 1 << 19, 1, (16, 1), [32 * w for w in range(4)]),
    ("halves", 64, 100, 1 << 20, 1025, (128, 4), [(p << 18) + 32 * h for p in range(4) for h in range(2)]),
    ("many", 128, 200, 1 << 17, 1, (256, 1), [0]),
    ("many", 256, 200, 1 << 17, 1, (256, 1), [0]),
]


@pytest.mark.parametrize("case", FAR, ids=lambda c: f"{c[0]}_d{c[1]}")
@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("below", [14.0, 23.3, 24.9, 25.1, 31.0])
def test_many_small_weights_beside_a_large_one(case, dtype, below):
    """Keys `below` powers of two under the few strong ones add up over a long
    context. V is 0 at the strong keys and 1 at the others, so that the result
    is the others' share, A. Off by 3 u A, the scores' 2 D e S A, sums over n
    keys 2 n e A; in FP16 each weight by half a subnormal of 2^-24 relative to
    a largest weight of 2^7 at least, n 2^-32 of the strong ones' share; the
    result's own half subnormal."""
    what, dim, new, slots, max_ctx, plan, strong = case
    say("case small weights", case, dtype, below)
    page = 4096
    k = torch.zeros(slots // page, page, 1, dim, dtype=dtype, device="cuda")
    v = torch.ones_like(k)
    k[..., 0] = -1.0
    for t in strong:
        k[t // page, t % page], v[t // page, t % page] = 0.0, 0.0
    cache = sg.PagedCache.from_tensors(k, v)
    seqs = sg.Sequences(ints([0, new]), ints([slots]), torch.arange(slots // page, dtype=torch.int32, device="cuda").reshape(1, -1))
    q = torch.zeros(new, 1, dim, dtype=dtype, device="cuda")
    q[..., 0] = 1.0
    scale = float(np.float32(below * np.log(2.0)))
    pl = cache.plan(seqs, new, 1, max_ctx)
    assert (pl.tile_rows, pl.splits) == plan, "the case has left its path"
    got = host(cache.attend(seqs, q, scale=scale, max_ctx=max_ctx))
    n = slots - new + 1 + np.arange(new, dtype=np.float64)[:, None, None]
    rest = (n - len(strong)) * np.exp(-scale)
    ref = rest / (rest + len(strong))
    tol = ref * (3 * U[dtype] + 2 * dim * E * scale + 2 * n * E)
    if dtype == F16:
        tol = tol + n * 2.0 ** -32 + A[F16]
    assert (np.abs(got - ref) <= tol).all(), f"off by {np.abs(got - ref).max():.3e} of {ref.max():.3e}, allowed {tol.max():.3e}"


# --------------------------------------------- every slot by itself

# n, ctx, heads, kv, dim, max_ctx, tile rows, more than one part
NEEDLE = [
    ([1], [3001], 4, 4, 128, 0, 16, True),
    ([1], [3001], 4, 2, 256, 0, 16, True),
    ([3], [801], 4, 4, 64, 1, 16, False),
    ([30], [2777], 4, 2, 128, 0, 128, True),
    ([30], [2777], 8, 4, 64, 0, 128, True),
    ([130], [2310], 4, 4, 128, 0, 256, True),
    ([130], [2310], 4, 2, 256, 0, 256, True),
    ([150], [777], 4, 4, 80, 1, 256, False),
]


@pytest.mark.parametrize("case", NEEDLE, ids=lambda c: f"n{c[0][0]}_c{c[1][0]}_d{c[4]}_t{c[6]}")
@pytest.mark.parametrize("dtype", [F16, BF16])
def test_every_kind_of_slot_counts_once(case, dtype):
    """q = 0, so that a row's n visible keys weigh the same, and V is 0 except
    in one slot a cache head: what comes out is its value / n (the powers of
    two and their sums are exact; a reciprocal and a product in FP32, one
    rounding), for first and last slots of blocks, parts, pages and the
    context. A slot that is lost, counted twice or seen too early shows whole."""
    n, ctx, heads, kv, dim, max_ctx, tile, split = case
    say("case needle", case, dtype)
    s = Setup(n, ctx, 8, heads, kv, dim, dtype, 34)
    s.q.zero_()
    new, all_ = n[0], ctx[0]
    pl = s.cache.plan(s.seqs, new, heads, max_ctx)
    assert pl.tile_rows == tile and (pl.splits > 1) == split, "the case has left its path"
    blocks = -(-all_ // pl.block_keys)
    per = -(-blocks // pl.splits) * pl.block_keys
    marks = {0, 1, 3, 4, 7, 8, 15, 16, 31, 32, 33, 47, 48, 63, 64, 65, 95, 96, 127, 128, 255, 256, all_ // 2,
             all_ - new - 1, all_ - new, all_ - new // 2 - 1, all_ - 2, all_ - 1, all_ // pl.block_keys * pl.block_keys}
    marks |= {p * per + d for p in range(1, pl.splits) for d in (-1, 0, 32)}
    marks |= {m - 1 for m in (all_ // 8 * 8, all_ // 32 * 32, all_ // 64 * 64)}
    marks = sorted(m for m in marks if 0 <= m < all_)
    marks += marks[: -len(marks) % kv]
    value = 1000.0 + 8.0 * np.arange(dim)               # below 2^12, multiples of 8: exact in FP16
    if dtype == BF16:
        value = 1024.0 + 16.0 * (np.arange(dim) % 64)   # eight bits
    seen = all_ - new + 1 + np.arange(new, dtype=np.float64)
    flat = torch.from_numpy(s.pages[0].astype(np.int64)).cuda()
    hv = torch.tensor(value, device="cuda").to(dtype)
    assert np.array_equal(host(hv), value)
    for i in range(0, len(marks), kv):
        s.vc.zero_()
        at = marks[i: i + kv]
        for h, t in enumerate(at):
            s.vc[flat[t // 8], t % 8, h] = hv
        got = host(s.cache.attend(s.seqs, s.q, max_ctx=max_ctx))
        there = np.array([at[h // (heads // kv)] for h in range(heads)])[None, :] < seen[:, None]
        ref = there[:, :, None] * value / seen[:, None, None]
        assert (np.abs(got - ref) <= ref * (U[dtype] + 3 * E)).all(), f"slots {at}"


# ------------------------------------------------ the joins' later turns

JOIN = [
    # n, ctx, heads, kv, dim, dtype, parts
    ([128, 20], [4096, 700], 8, 1, 128, F16, 16),
    ([128, 20], [4096, 700], 8, 1, 128, BF16, 16),
    ([64, 64], [3000, 2304], 8, 1, 64, F16, 11),
    ([64, 64], [3000, 2304], 8, 1, 64, BF16, 11),
    ([100, 30], [2600, 300], 8, 1, 256, F16, 10),
    ([100, 30], [2600, 300], 8, 1, 256, BF16, 10),
    ([130], [2800], 8, 2, 184, F16, 10),
]


@pytest.mark.parametrize("case", JOIN, ids=lambda c: f"n{c[0][0]}_c{c[1][0]}_d{c[4]}_{str(c[5])[6:]}")
def test_join_of_many_rows_and_many_parts(case):
    """More than 1024 rows in more than eight parts, the largest scores behind
    the eighth, and a sequence with fewer parts beside it."""
    n, ctx, heads, kv, dim, dtype, parts = case
    say("case join", case)
    s = Setup(n, ctx, 16, heads, kv, dim, dtype, 35)
    pl = s.cache.plan(s.seqs, s.tokens, heads)
    assert s.tokens * heads >= 1024 and pl.splits == parts > 8, "the case has left its path"
    blocks = -(-ctx[0] // pl.block_keys)
    late = 8 * -(-blocks // parts) * pl.block_keys
    assert late < ctx[0] - 2 * 16
    for p in s.pages[0, late // 16 + 1:]:
        s.kc[int(p)] *= 2.0
    out = s.cache.attend(s.seqs, s.q)
    s.check(out, s.want(), "join")
    assert torch.equal(out, s.cache.attend(s.seqs, s.q)), "not the same bits twice"


# ------------------------------------------------------ many sequences

MANY_SEQS = [
    # n, ctx, heads, kv, dim, dtype, tile rows, parts
    ([1] * 70, [1 + 7 * i % 300 for i in range(70)], 4, 2, 64, F16, 16, 1),
    ([1, 0, 2] * 43 + [1], [5 + 11 * i % 200 for i in range(130)], 2, 1, 128, BF16, 16, 1),
    ([1] * 69 + [3], [2 + i for i in range(69)] + [2000], 2, 1, 128, F16, 16, 3),
    ([3, 0] * 40, [3 + i for i in range(79)] + [1600], 16, 1, 64, BF16, 128, 6),
    ([100, 0] * 40 + [9], [101 + i % 50 for i in range(80)] + [1300], 2, 1, 72, F16, 128, 3),
    ([300, 0] * 33, [300 + i % 20 for i in range(66)], 1, 1, 128, F16, 256, 1),
]


@pytest.mark.parametrize("case", MANY_SEQS, ids=lambda c: f"s{len(c[0])}_t{c[6]}_p{c[7]}")
def test_more_than_64_sequences(case):
    n, ctx, heads, kv, dim, dtype, tile, parts = case
    say("case many sequences", len(n), case[2:])
    s = Setup(n, ctx, 16, heads, kv, dim, dtype, 36, 1, 2)
    pl = s.cache.plan(s.seqs, s.tokens, heads)
    assert len(n) > 64 and (pl.tile_rows, pl.splits) == (tile, parts), "the case has left its path"
    out = torch.full_like(s.q, 55.0)
    s.cache.attend(s.seqs, s.q, out=out)
    want = s.want()
    s.check(out, want, "many sequences")
    assert (host(out)[np.isnan(want[0][:, 0, 0])] == 55.0).all(), "a row of no sequence was written"


# --------------------------------------------------------- head widths

@pytest.mark.parametrize("dim", [104, 120, 136, 160, 192, 216, 248])
@pytest.mark.parametrize("n,ctx,tile", [([1, 2], [900, 33], 16), ([150], [260], 256), ([20], [1200], 0)])
def test_head_widths_between(dim, n, ctx, tile):
    say("case width", dim, n, ctx)
    dtype = BF16 if dim % 16 else F16
    s = Setup(n, ctx, 8, 3, 1, dim, dtype, 37, head_major=dim > 200)
    tile = tile or (128 if dim <= 128 else 256)
    assert s.cache.plan(s.seqs, s.tokens, 3).tile_rows == tile, "the case has left its path"
    s.check(s.cache.attend(s.seqs, s.q), s.want(), f"{dim} columns")


# --------------------------------------------------------- bias lists

@pytest.mark.parametrize("n", [255, 300, 511, 512, 513])
@pytest.mark.parametrize("spread", [200, 4096, 9001])
@pytest.mark.parametrize("history", [False, True])
def test_bias_lists_around_the_limits(n, spread, history):
    """Lists that the lanes hold and that they do not, more entries in one part
    than the lanes go through and fewer, copies among them; every step is exact."""
    say("case bias limits", n, spread, history)
    rng = np.random.default_rng(n + spread)
    ids, vals = rng.integers(0, spread, (2, n)), rng.integers(-50, 50, (2, n)) * 0.25
    x = torch.randint(-9, 9, (2, 9001), device="cuda").float()
    args = dict(bias_ids=ints(ids.ravel()), bias_start=ints([0, n, 2 * n]), bias_values=torch.tensor(vals.ravel(), dtype=F32, device="cuda"))
    want = dict(bias=[list(zip(i, v)) for i, v in zip(ids, vals)])
    if history:
        h, two = [[3, 3, 5], list(range(50))], torch.full((2,), 2.0, device="cuda")
        args.update(history=ints(h[0] + h[1]), history_start=ints([0, 3, 53]), repetition=two, presence=two)
        want.update(history=h, repetition=[2.0] * 2, presence=[2.0] * 2)
    ref = odec.adjust_logits(host(x), **want)
    assert np.array_equal(host(sg.adjust_logits(x, **args)), ref)
    assert np.array_equal(host(sg.adjust_logits(x, out=x, **args)), ref)

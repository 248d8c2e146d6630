"""GPU parity of the decode-step operators against their FP64 oracle.

Tolerances are sums of roundings, counted before the first run. u is the
type's half step (2^-11 FP16, 2^-8 BF16), e = 2^-24 FP32's, a = 2^-25 half the
smallest FP16 subnormal (0 for BF16, whose range is FP32's):

* append / rope: m (x cos - y sin): the angle's fraction of a turn to 2^-25 of
  a turn, 2 ulp of sine and cosine, four roundings: below 2^-20 m (|x| + |y|);
  then one rounding of the result: u |ref| + a.
* attention: relative to A = sum p |v| / sum p: each p rounded once, in both
  sums: with weights w_t summing to 1 and p_t (1 + d_t), |d_t| <= u, the result
  moves by sum w d (v - o) / (1 + sum w d), at most u (A + |o|) <= 2 u A to
  first order; the result rounded once (u A at most), so 3 u A; scores off by
  D e times sum |q k| scale on the first side of the exponential and as much
  again for scale and maximum, so 2 D e S; the sums over n keys, in any order,
  2 n e; half subnormals of p, n a max |v| (the largest p is at least 1 and
  enters the sum), and of the result, a.
* logits: at most 6 FP32 operations on terms no larger than M = the sum of
  the magnitudes: 6 e M, then u |ref| + a (e |ref| for FP32).
"""
import numpy as np
import pytest

import synth
import sparse_weight_only_amd as sg
from gpu_util import say
from oracle import decode as odec

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

F16, BF16, F32 = torch.float16, torch.bfloat16, torch.float32
U = {F16: 2.0 ** -11, BF16: 2.0 ** -8, F32: 2.0 ** -24}
A = {F16: 2.0 ** -25, BF16: 0.0, F32: 0.0}
E = 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def _device():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    sg.lib()


def host(x):
    return x.detach().double().cpu().numpy()


def ints(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


class Setup:
    """Ragged sequences over a shuffled page table, and what they hold."""

    def __init__(self, n, ctx, page, heads, kv, dim, dtype, seed=0, lead=0, trail=0, head_major=False, spare=2, per_seq=None):
        g = torch.Generator(device="cuda").manual_seed(seed)
        rng = np.random.default_rng(seed)
        self.n, self.ctx, self.page, self.dtype = n, ctx, page, dtype
        self.heads, self.kv, self.dim = heads, kv, dim
        per_seq = per_seq or max(-(-c // page) for c in ctx)
        need = [min(per_seq, -(-c // page)) for c in ctx]
        self.n_pages = sum(need) + spare
        order = rng.permutation(self.n_pages)
        self.pages = np.zeros((len(n), per_seq), np.int32)
        at = 0
        for s, m in enumerate(need):
            self.pages[s, :m] = order[at: at + m]
            at += m
        self.unused = order[at:]
        self.new_start = np.concatenate([[lead], lead + np.cumsum(n)]).astype(np.int32)
        self.tokens = int(self.new_start[-1]) + trail
        shape = (self.n_pages, kv, page, dim) if head_major else (self.n_pages, page, kv, dim)
        def make(*s):
            return torch.randn(s, device="cuda", generator=g).to(dtype)
        self.kc, self.vc = make(*shape), make(*shape)
        if head_major:
            self.kc, self.vc = self.kc.transpose(1, 2), self.vc.transpose(1, 2)
        self.q = make(self.tokens, heads, dim)
        self.k, self.v = make(self.tokens, kv, dim), make(self.tokens, kv, dim)
        self.cache = sg.PagedCache.from_tensors(self.kc, self.vc)
        self.seqs = sg.Sequences(ints(self.new_start), ints(ctx), ints(self.pages))

    def want(self, scale=None, tree=None):
        return odec.attend(host(self.q), host(self.kc), host(self.vc), self.new_start, self.ctx, self.pages,
                           scale or self.dim ** -0.5, tree)

    def tolerance(self, want):
        out, mean, worst, keys = want
        u, a = U[self.dtype], A[self.dtype]
        big = np.abs(host(self.vc)[np.isfinite(host(self.vc))]).max()
        w = worst[:, :, None]
        n = keys[:, :, None]
        return mean * (3 * u + 2 * self.dim * E * w + 2 * n * E) + n * a * big + a

    def check(self, out, want, what=""):
        ref = want[0]
        mine = ~np.isnan(ref[:, 0, 0])
        got, tol = host(out), self.tolerance(want)
        far = np.abs(got[mine] - ref[mine]) - tol[mine]
        assert not np.isnan(got[mine]).any(), f"{what}: NaN"
        assert (far <= 0).all(), f"{what}: {far.max():.3e} past the tolerance"


# ---------------------------------------------------------------- append

APPEND = [
    # n, ctx, page, heads, kv, dim, rot, interleaved, dtype, lead, trail
    ([1], [1], 8, 1, 1, 8, 8, False, F16, 0, 0),
    ([1], [700], 16, 32, 32, 128, 128, False, F16, 0, 0),
    ([3, 0, 5, 1], [3, 7, 60, 33], 16, 4, 2, 64, 64, True, BF16, 0, 0),
    ([2, 9], [30, 9], 8, 5, 5, 80, 20, False, F16, 1, 2),
    ([4, 4], [100, 4], 32, 6, 3, 96, 24, True, BF16, 2, 1),
    ([1] * 70, list(range(1, 71)), 64, 8, 1, 128, 96, False, F16, 0, 0),
    ([17], [17], 8, 3, 3, 256, 2, False, BF16, 0, 3),
    ([40], [1000], 256, 2, 1, 256, 256, True, F16, 0, 0),
    ([2600], [2600], 16, 2, 2, 64, 64, False, F16, 0, 0),       # workgroups of a whole token
]


@pytest.mark.parametrize("case", APPEND, ids=lambda c: f"n{len(c[0])}x{max(c[0])}_d{c[5]}_r{c[6]}_{'i' if c[7] else 'h'}")
@pytest.mark.parametrize("in_place", [False, True])
def test_append(case, in_place):
    n, ctx, page, heads, kv, dim, rot, inter, dtype, lead, trail = case
    say("case append", case, in_place)
    s = Setup(n, ctx, page, heads, kv, dim, dtype, 1, lead, trail)
    rope = sg.Rope(rot, interleaved=inter, factor=4.0, context=64.0, low=1.0, high=4.0, magnitude=1.25)
    turns = odec.rope_turns(rot, factor=4.0, context=64.0, low=1.0, high=4.0)
    kc0, vc0, q0 = host(s.kc), host(s.vc), host(s.q)
    out = s.q if in_place else torch.full_like(s.q, 77.0)
    s.cache.append(s.seqs, s.k, s.v, rope=rope, q=s.q, q_out=out)
    torch.cuda.synchronize()
    of = odec.slots(s.new_start, ctx)
    pos = [of[r][2] if r in of else 0 for r in range(s.tokens)]
    mine = np.array([r in of for r in range(s.tokens)])

    def close(got, x, rows):
        ref = odec.rope(x, pos, turns, inter, 1.25)
        half = rot // 2
        mag = np.abs(x).copy()
        i0, i1 = (slice(0, rot, 2), slice(1, rot, 2)) if inter else (slice(0, half), slice(half, rot))
        mag[..., i0], mag[..., i1] = 1.25 * (np.abs(x[..., i0]) + np.abs(x[..., i1])), 1.25 * (np.abs(x[..., i0]) + np.abs(x[..., i1]))
        tol = 2.0 ** -20 * mag + U[dtype] * np.abs(ref) + A[dtype]
        assert (np.abs(got - ref) <= tol)[rows].all()
        assert np.array_equal(got[rows][..., rot:], x[rows][..., rot:])

    got_q = host(out)
    close(got_q, q0, mine)
    assert np.array_equal(got_q[~mine], q0[~mine] if in_place else np.full_like(q0[~mine], 77.0))
    # the cache: v bit for bit, everything else untouched
    kc, vc = host(s.kc), host(s.vc)
    at = {r: (s.pages[sq, slot // page], slot % page) for r, (sq, _, slot) in of.items()}
    got_k = np.zeros((s.tokens, kv, dim))
    for r, (pg, sl) in at.items():
        got_k[r] = kc[pg, sl]
        assert np.array_equal(vc[pg, sl], host(s.v)[r])
        kc[pg, sl], vc[pg, sl] = kc0[pg, sl], vc0[pg, sl]
    close(got_k, host(s.k), mine)
    assert np.array_equal(kc, kc0) and np.array_equal(vc, vc0)


@pytest.mark.parametrize("dtype", [F16, BF16])
def test_rope_far_positions(dtype):
    """Positions where an FP32 angle would be off by whole radians."""
    say("case far positions", dtype)
    pos = [0, 1, -1, 1 << 20, (1 << 20) + 1, 12345678, -12345678, 2 ** 31 - 1, -2 ** 31]
    x = torch.randn(len(pos), 3, 64, device="cuda", generator=torch.Generator(device="cuda").manual_seed(2)).to(dtype)
    for inter in (False, True):
        rope = sg.Rope(48, interleaved=inter)
        y = host(rope.apply(x, ints(pos)))
        ref = odec.rope(host(x), pos, rope.turns.cpu().numpy(), inter)
        mag = np.abs(host(x)).max()
        # 2^31 turns-per-position products: the fraction to 2^-22 of a turn at most
        assert (np.abs(y - ref) <= (2.0 ** -20 + 2.0 ** -19) * 2 * mag + U[dtype] * np.abs(ref) + A[dtype]).all()
        assert np.array_equal(y[0], host(x)[0])
        z = rope.apply(x, ints(pos), out=torch.empty(3, len(pos), 64, dtype=dtype, device="cuda").transpose(0, 1))
        assert np.array_equal(host(z), y)


def test_append_strided_and_positions():
    """q, k, v as slices of one product's rows, a head-major cache, candidates' own positions, no q."""
    say("case append strided")
    n, ctx, page, heads, kv, dim = [5, 3], [20, 40], 8, 6, 2, 64
    s = Setup(n, ctx, page, heads, kv, dim, F16, 3, head_major=True)
    qkv = torch.randn(8, heads + 2 * kv, dim, device="cuda").half()
    q, k, v = qkv[:, :heads], qkv[:, heads: heads + kv], qkv[:, heads + kv:]
    rope = sg.Rope(64)
    pos = [15, 16, 16, 17, 17, 37, 38, 38]
    q_out = s.cache.append(s.seqs, k, v, rope=rope, q=q, positions=ints(pos))
    want_q = rope.apply(q, ints(pos))
    want_k = rope.apply(k, ints(pos))
    assert torch.equal(q_out, want_q) and q_out.shape == q.shape
    kc, vc = odec.append(host(s.kc), host(s.vc), host(want_k), host(v), s.new_start, ctx, s.pages)
    assert np.array_equal(host(s.kc), kc) and np.array_equal(host(s.vc), vc)
    # without a rope: k as it is
    s2 = Setup(n, ctx, page, heads, kv, dim, F16, 3)
    want = odec.append(host(s2.kc), host(s2.vc), host(k), host(v), s2.new_start, ctx, s2.pages)
    assert s2.cache.append(s2.seqs, k, v) is None
    assert np.array_equal(host(s2.kc), want[0]) and np.array_equal(host(s2.vc), want[1])


def test_append_to_pages_that_are_not_there():
    say("case append bad pages")
    s = Setup([2, 4, 3, 2], [10, 20, 2, 50], 8, 2, 2, 64, F16, 4, per_seq=6)
    s.pages[0, 1], s.pages[1, 2] = -1, s.n_pages          # new tokens of 0 in slots 8, 9; of 1 in 16..19
    seqs = sg.Sequences(ints(s.new_start), ints(s.ctx), ints(s.pages))   # 2: slots -1, 0, 1; 3: past its 48 slots
    ctx = [10, 20, 2, 48]
    want = odec.append(host(s.kc), host(s.vc), host(s.k), host(s.v), s.new_start, ctx, s.pages)
    s.cache.append(seqs, s.k, s.v)
    torch.cuda.synchronize()
    assert np.array_equal(host(s.kc), want[0]) and np.array_equal(host(s.vc), want[1])


# ---------------------------------------------------------------- attention

ATTEND = [
    # n, ctx, page, heads, kv, dim, dtype, lead, trail, head_major, max_ctx
    ([1], [1], 8, 1, 1, 8, F16, 0, 0, False, 0),
    ([1], [31], 16, 4, 4, 128, F16, 0, 0, False, 0),
    ([1], [32], 16, 4, 4, 128, BF16, 0, 0, False, 0),
    ([1, 1, 1], [33, 128, 129], 16, 8, 2, 64, F16, 0, 0, True, 0),
    ([1] * 9, [1, 2, 7, 63, 64, 65, 127, 300, 1], 8, 6, 2, 80, BF16, 0, 0, False, 0),
    ([1], [3001], 64, 8, 2, 128, F16, 0, 0, False, 0),               # split
    ([1], [3001], 64, 8, 2, 256, BF16, 0, 0, False, 0),
    ([1], [2100], 8, 40, 8, 96, F16, 0, 0, True, 0),
    ([1, 1], [5, 1500], 16, 2, 1, 128, F16, 0, 0, False, 1500),      # split, one sequence short of a part
    ([2, 0, 3, 1], [40, 9, 3, 77], 16, 5, 1, 128, F16, 1, 2, False, 0),
    ([5], [5], 8, 3, 1, 72, BF16, 0, 0, False, 0),
    ([3], [1000], 32, 9, 3, 64, F16, 0, 0, False, 0),
    ([70], [70], 16, 2, 2, 128, F16, 0, 0, False, 0),                # many rows from here on
    ([64, 1], [64, 300], 16, 4, 2, 64, BF16, 0, 0, False, 0),
    ([257], [300], 8, 1, 1, 128, F16, 0, 0, False, 0),
    ([130, 0, 40], [200, 5, 900], 32, 6, 2, 128, BF16, 2, 3, True, 0),
    ([90], [1111], 64, 8, 2, 256, F16, 0, 0, False, 0),
    ([65], [65], 16, 4, 4, 256, BF16, 0, 0, False, 0),
    ([100, 30], [130, 640], 128, 5, 1, 112, F16, 0, 0, False, 0),
    ([50], [2000], 16, 3, 3, 40, F16, 0, 0, False, 2000),
    ([40], [512], 8, 16, 2, 24, BF16, 0, 0, False, 0),
    ([33, 0, 7], [1500, 3, 1100], 16, 4, 2, 128, F16, 1, 1, False, 0),   # tiles of 128 rows, halves
    ([100], [1300], 32, 1, 1, 64, BF16, 0, 0, True, 0),
    ([25, 30], [2000, 1025], 8, 8, 2, 80, F16, 0, 0, False, 0),
    ([20], [1200], 16, 4, 1, 256, F16, 0, 0, False, 0),
]


def name(c):
    return f"n{len(c[0])}x{max(c[0])}_c{max(c[1])}_h{c[3]}-{c[4]}_d{c[5]}_p{c[2]}"


@pytest.mark.parametrize("case", ATTEND, ids=name)
def test_attend(case):
    n, ctx, page, heads, kv, dim, dtype, lead, trail, head_major, max_ctx = case
    say("case attend", case)
    s = Setup(n, ctx, page, heads, kv, dim, dtype, 5, lead, trail, head_major)
    want = s.want()
    out = torch.full_like(s.q, 55.0)
    got = s.cache.attend(s.seqs, s.q, out=out, max_ctx=max_ctx)
    torch.cuda.synchronize()
    assert got is out
    s.check(out, want, name(case))
    mine = ~np.isnan(want[0][:, 0, 0])
    assert (host(out)[~mine] == 55.0).all(), "a row of no sequence was written"
    again = s.cache.attend(s.seqs, s.q, max_ctx=max_ctx)
    assert torch.equal(again[torch.from_numpy(mine)], out[torch.from_numpy(mine)]), "not the same bits twice"


@pytest.mark.parametrize("scale", [1e-3, 0.5, 40.0])
@pytest.mark.parametrize("n,heads", [(1, 2), (80, 2), (200, 1)])
def test_attend_scales(scale, n, heads):
    """Weights from all equal to one key taking all."""
    say("case attend scale", scale, n)
    s = Setup([n], [400], 16, heads, 1, 64, F16, 6)
    want = s.want(scale)
    s.check(s.cache.attend(s.seqs, s.q, scale=scale), want, f"scale {scale}")


TREE = [([7], [7]), ([27, 0, 33], [40, 5, 33]), ([3, 5], [200, 700]), ([64], [1500]), ([40], [72]), ([27, 33], [1100, 90]), ([150], [190])]


@pytest.mark.parametrize("n,ctx", TREE)
@pytest.mark.parametrize("kind", ["tree", "random", "none", "short"])
@pytest.mark.parametrize("dim,heads,kv", [(128, 4, 2), (64, 3, 3)])
def test_attend_tree(n, ctx, kind, dim, heads, kv):
    say("case tree", n, ctx, kind, dim)
    s = Setup(n, ctx, 16, heads, kv, dim, BF16 if dim == 64 else F16, 7)
    rng = np.random.default_rng(8)
    words = 1 if kind == "short" else (max(n) + 31) // 32 + 1
    bits = np.zeros((s.tokens, words), np.uint32)
    for q in range(len(n)):
        a = s.new_start[q]
        for i in range(n[q]):
            up = {i}
            if kind == "tree":
                j = i
                while j:
                    j = (j - 1) // 2
                    up.add(j)
            elif kind == "none":
                up = set()
            else:
                up = {j for j in range(n[q]) if rng.random() < 0.4}
            for j in up:
                if j // 32 < words:
                    bits[a + i, j // 32] |= np.uint32(1 << (j % 32))
    want = s.want(tree=bits)
    tree = torch.from_numpy(bits.view(np.int32)).cuda()
    out = s.cache.attend(s.seqs, s.q, tree=tree)
    s.check(out, want, kind)
    if kind == "none":       # rows of pure prompts see nothing at all
        for q in range(len(n)):
            if n[q] == ctx[q]:
                assert (host(out)[s.new_start[q]: s.new_start[q + 1]] == 0).all()


@pytest.mark.parametrize("n,ctx,heads,kv", [([1, 1], [37, 300], 4, 2), ([3], [3], 2, 2), ([70, 33], [90, 333], 4, 2), ([200], [200], 1, 1), ([40, 40], [1090, 70], 4, 2)])
@pytest.mark.parametrize("value", [float("nan"), float("inf"), -65504.0])
def test_attend_unseen_slots_have_no_part(n, ctx, heads, kv, value):
    """Slots behind a sequence's end, pages of nobody, and later tokens of the
    same chunk hold NaN, infinities or the lowest value."""
    say("case unseen", n, ctx, value)
    s = Setup(n, ctx, 16, heads, kv, 128, F16, 9)
    clean = s.cache.attend(s.seqs, s.q).clone()
    for p in s.unused:
        s.kc[p], s.vc[p] = value, value
    for q in range(len(n)):
        if ctx[q] % 16:
            p = s.pages[q, ctx[q] // 16]
            s.kc[p, ctx[q] % 16:], s.vc[p, ctx[q] % 16:] = value, value
    got = s.cache.attend(s.seqs, s.q)
    assert torch.equal(got, clean)
    # the last new token of each sequence: only its own row sees it
    last = [int(s.new_start[q + 1]) - 1 for q in range(len(n)) if n[q] > 1]
    for q in range(len(n)):
        if n[q] > 1:
            p, sl = s.pages[q, (ctx[q] - 1) // 16], (ctx[q] - 1) % 16
            s.kc[p, sl], s.vc[p, sl] = value, value
    got = s.cache.attend(s.seqs, s.q)
    keep = torch.tensor([r not in last for r in range(s.tokens)], device="cuda")
    want = s.want()
    want[0][~keep.cpu().numpy()] = np.nan                 # (np.exp of an infinite difference)
    s.check(got, want, "rows before the last")
    if value != value and last:
        assert torch.isnan(got[last]).all(), "a row that sees NaN is NaN"


@pytest.mark.parametrize("n,ctx", [([1], [200]), ([90], [200]), ([90], [1200]), ([300], [400])])
def test_attend_infinite_value_that_is_seen(n, ctx):
    """An infinite v is infinite for the rows that see it (all weights here are positive) and nothing for the others."""
    say("case infinite value", n)
    s = Setup(n, ctx, 16, 2, 1, 64, F16, 10)
    slot = ctx[0] - n[0] // 2 - 1
    s.vc[s.pages[0, slot // 16], slot % 16, 0, 5] = float("inf")
    got = host(s.cache.attend(s.seqs, s.q))
    sees = np.arange(ctx[0] - n[0], ctx[0]) >= slot
    assert np.isposinf(got[sees][:, :, 5]).all() and np.isfinite(got[~sees]).all() and np.isfinite(np.delete(got, 5, 2)).all()


def test_attend_pages_that_are_not_there():
    say("case attend bad pages")
    for n, ctx in (([1, 1, 2], [40, 100, 20]), ([70, 3], [100, 90]), ([70, 30], [100, 1090]), ([300, 3], [300, 90])):
        s = Setup(n, ctx, 16, 4, 2, 128, F16, 11)
        s.pages[0, 1], s.pages[1, 3], s.pages[1, 0] = -1, s.n_pages, 2 ** 31 - 1
        s.seqs = sg.Sequences(ints(s.new_start), ints(ctx), ints(s.pages))
        s.check(s.cache.attend(s.seqs, s.q), s.want(), "missing pages")
        # nothing there at all: zeros
        s.pages[:] = -5
        seqs = sg.Sequences(ints(s.new_start), ints(ctx), ints(s.pages))
        assert (host(s.cache.attend(seqs, s.q)) == 0).all()


def test_attend_lengths_that_do_not_fit():
    """A context past its pages counts up to them; new tokens below slot 0 see nothing; a cache without pages."""
    say("case attend lengths")
    for n, ctx, fit in (([1, 4], [200, 2], [64, 2]), ([80, 90], [10 ** 9, 70], [64, 64]), ([200, 190], [10 ** 9, 70], [64, 64])):
        s = Setup(n, [40, 64], 16, 2, 2, 64, F16, 12, per_seq=4)
        s.pages[:] = np.arange(8).reshape(2, 4) % s.n_pages
        s.ctx = fit
        s.seqs = sg.Sequences(ints(s.new_start), ints(ctx), ints(s.pages))
        out = s.cache.attend(s.seqs, s.q)
        want = s.want()
        s.check(out, want)
        first = int(s.new_start[1])
        assert (host(out)[first: first + n[1] - fit[1]] == 0).all()
    empty = sg.PagedCache(0, 16, 2, 64)
    seqs = sg.Sequences(ints([0, 3]), ints([3]), torch.zeros(1, 0, dtype=torch.int32, device="cuda"))
    assert (host(empty.attend(seqs, torch.ones(3, 2, 64, dtype=F16, device="cuda"))) == 0).all()


def test_attend_strided_rows():
    say("case attend strided")
    s = Setup([3, 60], [50, 200], 16, 4, 2, 64, F16, 13)
    want = s.want()
    wide = torch.zeros(s.tokens, 9, 72, dtype=F16, device="cuda")
    wide[:, 2:6, 8:72] = s.q
    out = torch.empty(4, s.tokens, 64, dtype=F16, device="cuda").transpose(0, 1)
    s.cache.attend(s.seqs, wide[:, 2:6, 8:72], out=out)
    s.check(out, want, "strided")


def test_attend_far_into_a_large_cache():
    """Offsets past 2^32 elements, for keys and pages."""
    say("case large cache")
    kv, dim, page = 2, 128, 4096
    n_pages = (1 << 32) // (page * kv * dim) + 8
    k = torch.zeros(n_pages, page, kv, dim, dtype=F16, device="cuda")
    s = Setup([1, 70], [5000, 4500], page, 4, kv, dim, F16, 14)
    v = torch.zeros_like(k)
    far = [n_pages - 1, n_pages - 2, 1, n_pages - 3]
    pages = np.array([[far[0], far[1]], [far[2], far[3]]], np.int32)
    for q in range(2):
        for i in range(2):
            k[pages[q, i]], v[pages[q, i]] = s.kc[s.pages[q, i]], s.vc[s.pages[q, i]]
    cache = sg.PagedCache.from_tensors(k, v)
    seqs = sg.Sequences(ints(s.new_start), ints(s.ctx), ints(pages))
    assert torch.equal(cache.attend(seqs, s.q), s.cache.attend(s.seqs, s.q))
    cache.append(seqs, s.k, s.v)
    s.cache.append(s.seqs, s.k, s.v)
    for q in range(2):
        for i in range(2):
            assert torch.equal(k[pages[q, i]], s.kc[s.pages[q, i]]) and torch.equal(v[pages[q, i]], s.vc[s.pages[q, i]])


def test_attend_workspace_given():
    say("case workspace")
    s = Setup([1], [4000], 16, 8, 2, 128, F16, 15)
    need = s.cache.plan(s.seqs, 1, 8).workspace_bytes
    assert need > 0
    ws = torch.full((need + 64,), 255, dtype=torch.uint8, device="cuda")     # NaN in every word
    a = s.cache.attend(s.seqs, s.q, workspace=ws[:need])
    assert torch.equal(a, s.cache.attend(s.seqs, s.q))
    assert (ws[need:] == 255).all()
    with pytest.raises(sg.SgemvError):
        s.cache.attend(s.seqs, s.q, workspace=ws[: need - 16])


# ---------------------------------------------------------------- logits

LOGITS = [
    # rows, vocab, history lengths, bias lengths, masks, dtype, out dtype
    (1, 1, [0], [0], 0, F16, F16),
    (1, 32000, [300], [8], 1, F16, F32),
    (3, 4095, [0, 1, 900], [0, 5, 1], 2, F32, F32),
    (4, 4097, [7, 0, 3000, 64], [300, 0, 2, 9], 3, BF16, BF16),
    (16, 1003, [50] * 16, [3] * 16, 16, F16, F16),
    (2, 131073, [5000, 17], [0, 700], 1, BF16, F32),
]


def logits_case(rows, vocab, hist, bias, masks, dtype, seed=16):
    rng = np.random.default_rng(seed)
    x = torch.randn(rows, vocab, device="cuda", generator=torch.Generator(device="cuda").manual_seed(seed)) * 4
    kw = dict(repetition=1 + rng.random(rows), frequency=rng.random(rows) - 0.3, presence=rng.random(rows) - 0.3)
    kw = {k: v.astype(np.float32) for k, v in kw.items()}
    # ids repeat, and some are no tokens
    h = [np.where(rng.random(n) < 0.05, rng.choice([-1, vocab, 2 ** 31 - 1, -2 ** 31], n), rng.integers(0, min(vocab, 1 + n // 2 + 1), n)).astype(np.int64) for n in hist]
    prompt = np.array([int(rng.integers(-1, n + 3)) for n in hist], np.int32)
    b = [[(int(i), float(np.float32(a))) for i, a in zip(np.where(rng.random(n) < 0.1, -3, rng.integers(0, min(vocab, n + 2), n)), rng.standard_normal(n))] for n in bias]
    m = rng.random((masks, vocab)) < 0.5 if masks else None
    row = rng.integers(-1, masks + 1, rows).astype(np.int32) if masks else None
    return x.to(dtype), kw, h, prompt, b, m, row


def bits(m):
    n, vocab = m.shape
    pad = np.zeros((n, -(-vocab // 32) * 32), bool)
    pad[:, :vocab] = m
    w = (pad.reshape(n, -1, 32).astype(np.uint32) << np.arange(32, dtype=np.uint32)).sum(-1, dtype=np.uint64).astype(np.uint32)
    return torch.from_numpy(w.view(np.int32)).cuda()


def ragged(lists, dtype):
    start = ints(np.concatenate([[0], np.cumsum([len(x) for x in lists])]))
    return torch.tensor(np.concatenate([np.asarray(x, np.float64) for x in lists]).astype(np.int64 if dtype == torch.int32 else np.float64), device="cuda").to(dtype), start


@pytest.mark.parametrize("case", LOGITS, ids=lambda c: f"{c[0]}x{c[1]}")
@pytest.mark.parametrize("use", ["all", "penalties", "bias", "mask", "nothing"])
def test_logits(case, use):
    rows, vocab, hist, bias, masks, dtype, out_dtype = case
    say("case logits", case, use)
    x, kw, h, prompt, b, m, row = logits_case(rows, vocab, hist, bias, masks, dtype)
    args, want = {}, {}
    if use in ("all", "penalties"):
        args["history"], args["history_start"] = ragged(h, torch.int32)
        args["prompt_len"] = ints(prompt)
        args.update({k: torch.from_numpy(v).cuda() for k, v in kw.items()})
        want.update(history=h, prompt_len=prompt, **kw)
    if use in ("all", "bias"):
        args["bias_ids"], args["bias_start"] = ragged([[i for i, _ in r] for r in b], torch.int32)
        args["bias_values"], _ = ragged([[a for _, a in r] for r in b], F32)
        want["bias"] = b
    if use in ("all", "mask") and masks:
        args["masks"], args["mask_row"] = bits(m), ints(row)
        want["masks"] = [m[i] if 0 <= i < masks else None for i in row]
    out = torch.full((rows, vocab + 3), 9.0, dtype=out_dtype, device="cuda")[:, :vocab]
    before = host(x)
    sg.adjust_logits(x, out=out, **args)
    torch.cuda.synchronize()
    ref = odec.adjust_logits(before, **want)
    got = host(out)
    fine = np.isfinite(ref)
    assert np.array_equal(fine, np.isfinite(got)) and np.array_equal(got[~fine], ref[~fine])
    # every term a token meets, counted whole
    size = np.abs(before) * 2 + 1.3 * max(hist + [0]) + 1.0 + np.abs(np.concatenate([[0.0]] + [[a for _, a in r] for r in b])).max()
    assert (np.abs(got[fine] - ref[fine]) <= (6 * E * size + U[out_dtype] * np.abs(ref) + A[out_dtype])[fine]).all()
    assert np.array_equal(host(x), before)
    assert (host(out._base)[:, vocab:] == 9.0).all(), "written past a row"
    if out_dtype == dtype:
        y = x.clone()
        assert torch.equal(sg.adjust_logits(y, out=y, **args), out), "in place differs"


def test_logits_bias_given_twice():
    """The first place holds, wherever the copies are in the list."""
    say("case bias twice")
    ids = np.array([5] * 700 + [9, 5, 9, 9, 4099, 4099])
    vals = 1.0 + np.arange(len(ids)) * 0.5
    out = sg.adjust_logits(torch.zeros(1, 5000, device="cuda"), bias_ids=ints(ids), bias_values=torch.tensor(vals, dtype=F32, device="cuda"),
                           bias_start=ints([0, len(ids)]))
    want = np.zeros(5000)
    want[5], want[9], want[4099] = vals[0], vals[700], vals[704]
    assert np.array_equal(host(out)[0], want)


@pytest.mark.parametrize("n", [1, 2, 7, 256, 257, 1024, 1025, 3000])
@pytest.mark.parametrize("spread", [1, 40, 9000])
def test_logits_bias_lists_of_any_length(n, spread):
    """Copies in one part or over several, lists that the lanes hold and longer ones, in place too."""
    say("case bias lists", n, spread)
    rng = np.random.default_rng(n + spread)
    ids = [rng.integers(0, spread, k) for k in (n, 0, n)]
    vals = [rng.integers(-50, 50, k) * 0.25 for k in (n, 0, n)]
    x = torch.randint(-9, 9, (3, 9001), device="cuda").float()
    m = rng.random((1, 9001)) < 0.7
    h = [[3, 3, 5], list(range(50)), []]
    flat, start = ragged(ids, torch.int32)
    hist, hist_start = ragged(h, torch.int32)
    two = torch.full((3,), 2.0, device="cuda")
    args = dict(bias_ids=flat, bias_start=start, bias_values=ragged(vals, F32)[0], history=hist, history_start=hist_start, repetition=two, frequency=two,
                masks=bits(m), mask_row=ints([0, 0, -1]))
    ref = odec.adjust_logits(host(x), h, repetition=[2.0] * 3, frequency=[2.0] * 3, bias=[list(zip(i, v)) for i, v in zip(ids, vals)], masks=[m[0], m[0], None])
    assert np.array_equal(host(sg.adjust_logits(x, **args)), ref)          # every step is exact in these numbers
    assert np.array_equal(host(sg.adjust_logits(x, out=x, **args)), ref)


def test_logits_special_values():
    """NaN and infinities in masked places are gone, in others they follow the formula; a row may be left with nothing."""
    say("case logits special")
    inf, nan = float("inf"), float("nan")
    x = torch.tensor([[nan, inf, -inf, 1.0, nan, inf, -inf, -1.0, 65504.0, -65504.0]] * 3, device="cuda")
    m = np.ones((2, 10), bool)
    m[0, [0, 1, 2, 3]] = False
    m[1] = False
    hist = ints([1, 2, 5, 6, 8, 9] * 3)
    out = host(sg.adjust_logits(x, history=hist, history_start=ints([0, 6, 12, 18]), repetition=torch.full((3,), 2.0, device="cuda"),
                                masks=bits(m), mask_row=ints([0, 1, -1])))
    assert np.array_equal(out[0], [-inf, -inf, -inf, -inf, nan, inf, -inf, -1.0, 32752.0, -131008.0], equal_nan=True)
    assert (out[1] == -inf).all()
    assert np.array_equal(out[2], [nan, inf, -inf, 1.0, nan, inf, -inf, -1.0, 32752.0, -131008.0], equal_nan=True)


def test_logits_lists_that_do_not_fit():
    """Starts that point outside their list, or backwards, are cut to it."""
    say("case logits starts")
    x = torch.ones(3, 100, device="cuda")
    two = torch.full((3,), 2.0, device="cuda")
    hist, start = ints([1, 2, 3]), ints([-7, 1, 0, 99])
    out = host(sg.adjust_logits(x, history=hist, history_start=start, repetition=two, bias_ids=hist, bias_start=start, bias_values=two))
    want = np.ones((3, 100))
    want[0, 1] = want[2, 1] = want[2, 2] = want[2, 3] = 2.5
    assert np.array_equal(out, want)


# ------------------------------------------- tensors of another device

def test_tensors_on_the_cpu_are_refused_by_name():
    say("case cpu tensors")
    s = Setup([1, 3], [40, 70], 16, 4, 2, 64, F16, 23)
    cpu = lambda x: x.detach().cpu()
    rope, far = sg.Rope(64), sg.Rope(64, device="cpu")
    pos = ints([0, 1, 2, 3])
    tree = ints(np.zeros((4, 1)))
    there = sg.Sequences(cpu(s.seqs.new_start), cpu(s.seqs.ctx_len), cpu(s.seqs.pages))
    good = dict(seqs=s.seqs, k=s.k, v=s.v, rope=rope, q=s.q, q_out=torch.empty_like(s.q), positions=pos)
    for what, x in (("seqs", there), ("k", cpu(s.k)), ("v", cpu(s.v)), ("rope", far), ("q", cpu(s.q)), ("q_out", cpu(s.q)), ("positions", cpu(pos))):
        with pytest.raises(ValueError, match=f"{what} is on cpu"):
            s.cache.append(**{**good, what: x})
    work = torch.empty(1 << 20, dtype=torch.uint8, device="cuda")
    good = dict(seqs=s.seqs, q=s.q, tree=tree, out=torch.empty_like(s.q), workspace=work)
    for what, x in (("seqs", there), ("q", cpu(s.q)), ("tree", cpu(tree)), ("out", cpu(s.q)), ("workspace", cpu(work))):
        with pytest.raises(ValueError, match=f"{what} is on cpu"):
            s.cache.attend(**{**good, what: x})
    for what, args in (("x", (cpu(s.q), pos)), ("positions", (s.q, cpu(pos))), ("out", (s.q, pos, cpu(s.q)))):
        with pytest.raises(ValueError, match=f"{what} is on cpu"):
            rope.apply(*args)
    x = torch.zeros(2, 50, device="cuda")
    lists = dict(history=ints([1, 2]), history_start=ints([0, 1, 2]), prompt_len=ints([1, 1]), repetition=torch.ones(2, device="cuda"),
                 frequency=torch.ones(2, device="cuda"), presence=torch.ones(2, device="cuda"), bias_ids=ints([3]), bias_start=ints([0, 0, 1]),
                 bias_values=torch.ones(1, device="cuda"), masks=ints([[-1, -1]]), mask_row=ints([0, -1]))
    for what in lists:
        with pytest.raises(ValueError, match=what):
            sg.adjust_logits(x, **{**lists, what: cpu(lists[what])})
    with pytest.raises(ValueError, match="out"):
        sg.adjust_logits(x, out=cpu(x), **lists)


# ------------------------------------------- streams, graphs, use together

def test_other_stream_and_two_at_once():
    say("case streams")
    a = Setup([1, 1], [3000, 900], 16, 8, 2, 128, F16, 17)
    b = Setup([70], [700], 16, 4, 2, 64, BF16, 18)
    wa, wb = a.cache.attend(a.seqs, a.q), b.cache.attend(b.seqs, b.q)
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    got = []
    for _ in range(8):
        got.append((a.cache.attend(a.seqs, a.q, stream=s1), b.cache.attend(b.seqs, b.q, stream=s2)))
    s1.synchronize()
    s2.synchronize()
    assert all(torch.equal(x, wa) and torch.equal(y, wb) for x, y in got)


def test_captured_step_replays_with_new_lengths():
    """Append, attention and logits captured once; lengths, pages and inputs
    change between replays, and eager calls run in between."""
    say("case graph")
    heads, kv, dim, page, vocab = 8, 2, 128, 16, 5000
    s = Setup([1, 1], [1, 1], page, heads, kv, dim, F16, 19, per_seq=80, spare=200)
    s.pages[:] = np.random.default_rng(20).permutation(160).reshape(2, 80)
    s.seqs.pages.copy_(ints(s.pages))
    rope = sg.Rope(dim)
    x = torch.randn(2, vocab, device="cuda").half()
    hist, start = torch.zeros(64, dtype=torch.int32, device="cuda"), ints([0, 3, 9])
    rep = torch.full((2,), 1.5, device="cuda")
    kc0, vc0 = s.kc.clone(), s.vc.clone()

    def step():
        q = s.cache.append(s.seqs, s.k, s.v, rope=rope, q=s.q)
        return s.cache.attend(s.seqs, q, max_ctx=1280), sg.adjust_logits(x, history=hist, history_start=start, repetition=rep)

    step()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph, other = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        with torch.cuda.graph(graph, stream=side):
            out = step()
        with torch.cuda.graph(other, stream=side):
            out2 = step()
    torch.cuda.synchronize()
    for round_, ctx in enumerate([[1, 2], [17, 900], [1280, 64], [500, 1]]):
        s.seqs.ctx_len.copy_(ints(ctx))
        for t in (s.q, s.k, s.v, x):
            t.copy_(torch.randn(t.shape, device="cuda", generator=torch.Generator(device="cuda").manual_seed(round_)))
        hist.copy_(torch.randint(0, vocab, (64,), device="cuda"))
        s.kc.copy_(kc0)
        s.vc.copy_(vc0)
        eager = [t.clone() for t in step()]
        cache = s.kc.clone(), s.vc.clone()
        s.kc.copy_(kc0)
        s.vc.copy_(vc0)
        for g, o in ((graph, out), (other, out2), (graph, out)):
            g.replay()
            torch.cuda.synchronize()
            assert torch.equal(o[0], eager[0]) and torch.equal(o[1], eager[1])
        assert torch.equal(s.kc, cache[0]) and torch.equal(s.vc, cache[1])


def test_decode_step_between_the_gemvs():
    """A decoder layer's attention half and the choice of a token, on packed
    layers: the q, k, v products in one launch, the append, the attention, the
    o product, the vocabulary product and its penalties and masks; two beams
    over a prompt of 40 tokens, and every step against FP64 on its own inputs."""
    say("case decode step")
    heads, kv, dim, hidden, vocab, B = 4, 4, 64, 256, 3000, 2
    rng = synth.rng(77)
    def layer(N, K, nk):
        return sg.SparseGemvLayer.from_dense((0.06 * rng.standard_normal((N, K))).astype(np.float16), nk)
    wq, wk, wv, wo, wh = (layer(N, hidden, 2) for N in (hidden, hidden, hidden, hidden, vocab))
    cache = sg.PagedCache(12, 16, kv, dim)
    rope = sg.Rope(dim)
    prompt = torch.randn(40, kv, dim, device="cuda").half()
    pages = ints([[3, 1, 7], [3, 1, 5]])                       # the beams share the prompt's first two pages
    first = sg.Sequences(ints([0, 40]), ints([40]), ints([[3, 1, 7]]))
    cache.append(first, prompt, prompt * 0.5, rope=rope)
    cache.k[5], cache.v[5] = cache.k[7], cache.v[7]
    x = torch.randn(B, hidden, device="cuda").half()
    ctx = ints([40, 40])
    seqs = sg.Sequences(ints([0, 1, 2]), ctx, pages)
    history = [[1, 2], [2, 2]]
    allowed = rng.random((2, vocab)) < 0.01
    rep = torch.full((B,), 1.3, device="cuda")
    stream = torch.cuda.current_stream().cuda_stream
    for step in range(5):
        ctx += 1
        q, k, v = (torch.empty(B, heads, dim, dtype=F16, device="cuda") for _ in range(3))
        sg.run_group([(w.desc, w.blob.data_ptr(), x.data_ptr(), y.data_ptr()) for w, y in ((wq, q), (wk, k), (wv, v))], B, stream)
        q0 = host(q)
        cache.append(seqs, k, v, rope=rope, q=q, q_out=q)
        pos = [40 + step] * B
        turns = rope.turns.cpu().numpy()
        for got, src in ((host(q), q0), (host(cache.k[[7, 5], (40 + step) % 16]), host(k))):
            ref = odec.rope(src, pos, turns)
            mag = np.abs(src).max()
            assert (np.abs(got - ref) <= 2.0 ** -20 * 2 * mag + U[F16] * np.abs(ref) + A[F16]).all()
        a = cache.attend(seqs, q)
        out, mean, worst, keys = odec.attend(host(q), host(cache.k), host(cache.v), [0, 1, 2], [41 + step] * 2, pages.cpu().numpy(), dim ** -0.5)
        tol = mean * (3 * U[F16] + 2 * dim * E * worst[:, :, None] + 2 * keys[:, :, None] * E) + (41 + step) * A[F16] * 8 + A[F16]
        assert (np.abs(host(a) - out) <= tol).all()
        x = wo.run(a.reshape(B, hidden))
        logits = wh.run(x)
        ids, start = ragged(history, torch.int32)
        got = sg.adjust_logits(logits, history=ids, history_start=start, repetition=rep, masks=bits(allowed))
        ref = odec.adjust_logits(host(logits), history, repetition=rep.cpu().numpy(), masks=list(allowed))
        fine = np.isfinite(ref)
        assert np.array_equal(fine, np.isfinite(host(got)))
        assert (np.abs(host(got) - ref)[fine] <= (6 * E * 2 * np.abs(host(logits)))[fine]).all()
        best = got.argmax(1).tolist()
        assert all(allowed[b, t] for b, t in enumerate(best))
        history = [h + [t] for h, t in zip(history, best)]

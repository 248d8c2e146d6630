"""GPU parity of the cache in 8 bits and of attention through a window against
their FP64 oracle.

Tolerances count roundings as those of the 16-bit operators do (u the type's half
step, e = 2^-24):

* append: without rotary positions the codes and scales are the oracle's, bit
  for bit. With them a turned value is off by t = 2^-20 m (|x| + |y|) (counted
  with the 16-bit append), so its code may be that of a value t away: the decoded
  value is off by half a step of e4m3 there, 2^-4 (|ref| + t) or 2^-10 of the
  scale for subnormals, and t. A scale may differ where the largest value lies
  within t of a border.
* attention: the 16-bit attention's bound, on the values that codes and scales
  stand for.
"""
import numpy as np
import pytest

import sparse_weight_only_amd as sg
from gpu_util import say
from oracle import decode as odec
from test_gpu_decode import A, ATTEND, BF16, E, F16, TREE, U, Setup, host, ints, name

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _device():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    sg.lib()


def raw(x):
    return x.contiguous().view(torch.uint8).cpu().numpy()


class Setup8(Setup):
    """A Setup over a cache in 8 bits: random codes, a scale for each block and head."""

    def __init__(self, n, ctx, page, heads, kv, dim, dtype, seed=0, lead=0, trail=0, head_major=False, spare=2, per_seq=None, block=8,
                 spread=3):
        super().__init__(n, ctx, page, heads, kv, dim, dtype, seed, lead, trail, False, spare, per_seq)
        g = torch.Generator(device="cuda").manual_seed(seed + 1000)
        self.block = min(block, page)
        def codes():
            x = (100.0 * torch.randn(self.n_pages, page, kv, dim, device="cuda", generator=g)).clamp(-448, 448).to(torch.float8_e4m3fn)
            return x.transpose(1, 2).contiguous().transpose(1, 2) if head_major else x
        self.k8, self.v8 = codes(), codes()
        s = torch.randint(120 - spread, 121, (self.n_pages, page // self.block, kv, 2), device="cuda", generator=g)
        self.scales = s.to(torch.uint8).view(torch.float8_e8m0fnu)
        self.cache = sg.PagedCache8.from_tensors(self.k8, self.v8, self.scales)
        self.values()

    def values(self):
        """The cache's values, for the oracle and the tolerance, as they are now."""
        k, v, s = raw(self.k8).reshape(self.k8.shape), raw(self.v8).reshape(self.v8.shape), raw(self.scales)
        self.kc, self.vc = (torch.from_numpy(odec.values8(c, s, i)) for i, c in enumerate((k, v)))

    def want(self, scale=None, tree=None, window=0, sinks=0):
        return odec.attend(host(self.q), host(self.kc), host(self.vc), self.new_start, self.ctx, self.pages,
                           scale or self.dim ** -0.5, tree, window, sinks)


# ---------------------------------------------------------------- append

APPEND = [
    # n, ctx, page, block, heads, kv, dim, rot, interleaved, dtype, lead, trail
    ([1], [1], 8, 8, 1, 1, 16, 16, False, F16, 0, 0),
    ([1], [700], 16, 16, 32, 32, 128, 128, False, F16, 0, 0),
    ([3, 0, 5, 1], [3, 7, 60, 33], 16, 8, 4, 2, 64, 64, True, BF16, 0, 0),
    ([2, 9], [30, 9], 8, 8, 5, 5, 80, 20, False, F16, 1, 2),
    ([4, 40], [100, 45], 32, 32, 6, 3, 96, 24, True, BF16, 2, 1),
    ([1] * 70, list(range(1, 71)), 64, 32, 8, 1, 128, 96, False, F16, 0, 0),
    ([17], [17], 8, 8, 3, 3, 256, 2, False, BF16, 0, 3),
    ([400], [1000], 256, 128, 2, 1, 256, 256, True, F16, 0, 0),          # every lane of a workgroup, and its most sines
    ([130, 64], [135, 200], 128, 128, 3, 2, 128, 64, False, BF16, 0, 0),
    ([777], [777], 64, 64, 3, 2, 64, 64, False, F16, 1, 0),
    ([33, 1], [50, 17], 16, 16, 2, 2, 48, 48, False, F16, 0, 0),
]


def check_append(s, before, rope_args, q0, out, x_k, x_v, pos):
    """The cache, its scales and q after an append, against the oracle; x_k and x_v FP64 as stored, pos by row."""
    turns, inter, m = rope_args
    of = odec.slots(s.new_start, s.ctx)
    mine = np.array([r in of for r in range(s.tokens)])
    def slack(x):
        half = 0 if turns is None else len(turns)
        t = np.zeros(x.shape)
        if half:
            i0, i1 = (np.arange(half) * 2, np.arange(half) * 2 + 1) if inter else (np.arange(half), np.arange(half) + half)
            both = np.abs(x[..., i0]) + np.abs(x[..., i1])
            t[..., i0] = t[..., i1] = 2.0 ** -20 * m * both
        return t
    if out is not None:
        ref = odec.rope(q0, pos, turns, inter, m)
        ok = np.abs(host(out) - ref) <= slack(q0) + U[s.dtype] * np.abs(ref) + A[s.dtype]
        assert ok[mine].all()
        assert np.array_equal(host(out)[~mine], q0[~mine]) or (host(out)[~mine] == 77.0).all(), "a row of no sequence was written"
    k0, v0, s0 = before
    v_ref, s_ref = odec.append8(v0, s0, x_v, 1, s.new_start, s.ctx, s.pages)
    k_ref, s_ref = odec.append8(k0, s_ref, x_k if turns is None else odec.rope(x_k, pos, turns, inter, m), 0, s.new_start, s.ctx, s.pages)
    got_k, got_v, got_s = (raw(t).reshape(t.shape) for t in (s.k8, s.v8, s.scales))
    assert np.array_equal(got_v, v_ref) and np.array_equal(got_s[..., 1], s_ref[..., 1]), "V"
    if turns is None:
        assert np.array_equal(got_k, k_ref) and np.array_equal(got_s[..., 0], s_ref[..., 0]), "K"
        return
    # a border within the slack would be a coincidence of 2^-18 or so for each block: none in these cases
    assert np.array_equal(got_s[..., 0], s_ref[..., 0]), "scales of K"
    a, b = odec.values8(got_k, got_s, 0), odec.values8(k_ref, s_ref, 0)
    step = 2.0 ** (np.repeat(s_ref[..., 0].astype(int), s.block, 1) - 127)[..., None]
    near = np.abs(a - b) <= 2.0 ** -3 * np.abs(b) + 2.0 ** -9 * step
    assert near.all(), "codes of K more than one apart"
    # each new code is a nearest one of a value within the slack
    each = s.page
    for row, (q, _, slot) in of.items():
        if slot < 0 or slot // each >= s.pages.shape[1] or not 0 <= s.pages[q, slot // each] < s.n_pages:
            continue
        at = int(s.pages[q, slot // each]), slot % each
        ref, t = odec.rope(x_k[row:row + 1], [pos[row]], turns, inter, m)[0], slack(x_k[row:row + 1])[0]
        far = np.abs(a[at] - ref) - (t + np.maximum(2.0 ** -4 * (np.abs(ref) + t), 2.0 ** -10 * step[at]))
        assert (far <= 0).all(), (row, far.max())
    new = np.zeros(got_k.shape[:2], bool)
    for _, (q, _, slot) in of.items():
        if slot >= 0 and slot // each < s.pages.shape[1] and 0 <= s.pages[q, slot // each] < s.n_pages:
            new[s.pages[q, slot // each], slot % each] = True
    assert np.array_equal(got_k[~new], k_ref[~new]), "older codes"


def state(s):
    return tuple(raw(t).reshape(t.shape) for t in (s.k8, s.v8, s.scales))


@pytest.mark.parametrize("case", APPEND, ids=lambda c: f"n{len(c[0])}x{max(c[0])}_b{c[3]}_d{c[6]}_r{c[7]}_{'i' if c[8] else 'h'}")
@pytest.mark.parametrize("how", ["plain", "rope", "in place"])
def test_append8(case, how):
    n, ctx, page, block, heads, kv, dim, rot, inter, dtype, lead, trail = case
    say("case append8", case, how)
    s = Setup8(n, ctx, page, heads, kv, dim, dtype, 1, lead, trail, block=block, spread=6)
    # magnitudes that call for scales above and below the older ones
    s.v *= torch.exp2(torch.randint(-6, 7, (s.tokens, kv, 1), device="cuda").float()).to(dtype)
    of = odec.slots(s.new_start, ctx)
    pos = [of[r][2] if r in of else 0 for r in range(s.tokens)]
    before = state(s)
    k, v, q0 = host(s.k), host(s.v), host(s.q)
    if how == "plain":
        assert s.cache.append(s.seqs, s.k, s.v) is None
        check_append(s, before, (None, False, 1.0), None, None, k, v, pos)
        return
    rope = sg.Rope(rot, interleaved=inter, magnitude=1.25)
    out = s.q if how == "in place" else torch.full_like(s.q, 77.0)
    s.cache.append(s.seqs, s.k, s.v, rope=rope, q=s.q, q_out=out)
    check_append(s, before, (odec.rope_turns(rot), inter, 1.25), q0, out, k, v, pos)


def test_append8_token_by_token():
    """Block by block, tokens whose magnitudes rise and fall: scales grow with them and start anew with a block."""
    say("case append8 token by token")
    s = Setup8([1, 1], [1, 1], 16, 2, 2, 32, F16, 2, per_seq=4, spare=10, block=16)
    s.pages[:] = [[0, 1, 2, 3], [4, 5, 6, 7]]
    s.seqs.pages.copy_(ints(s.pages))
    rng = np.random.default_rng(3)
    for step in range(50):
        s.ctx = [step + 1, min(step + 7, 64)]
        s.seqs.ctx_len.copy_(ints(s.ctx))
        for t in (s.k, s.v):
            t.copy_(torch.from_numpy(rng.standard_normal(t.shape) * 2.0 ** rng.integers(-12, 8)).half())
        before = state(s)
        s.cache.append(s.seqs, s.k, s.v)
        check_append(s, before, (None, False, 1.0), None, None, host(s.k), host(s.v), None)
    assert len(set(raw(s.scales)[..., 0].reshape(-1).tolist())) > 4


@pytest.mark.parametrize("dtype", [F16, BF16])
def test_append8_special_values(dtype):
    say("case append8 special values", dtype)
    s = Setup8([9], [12], 16, 2, 2, 16, dtype, 4, block=8)
    big = torch.finfo(dtype).max
    s.k.zero_()
    s.v[0], s.v[1, 0, 0], s.v[1, 0, 1], s.v[1, 1, 2] = 0.0, float("inf"), float("nan"), -float("inf")
    s.v[2, 0, 3], s.v[6:, 1] = big, torch.finfo(dtype).tiny
    s.k[7] = -0.0
    before = state(s)
    s.cache.append(s.seqs, s.k, s.v)
    check_append(s, before, (None, False, 1.0), None, None, host(s.k), host(s.v), None)
    assert (raw(s.v8).reshape(s.v8.shape)[s.pages[0, 0], 4, 0, :2] & 127 == 127).all()


def test_append8_where_nothing_is_stored():
    """Pages that are not there, and slots below 0: q is turned all the same."""
    say("case append8 pages not there")
    s = Setup8([12, 9, 3], [40, 5, 3], 16, 4, 2, 64, F16, 5, block=16)
    s.pages[0, 1], s.pages[2, 0] = -1, s.n_pages
    s.seqs.pages.copy_(ints(s.pages))
    of = odec.slots(s.new_start, s.ctx)
    pos = [of[r][2] if r in of else 0 for r in range(s.tokens)]
    before, q0 = state(s), host(s.q)
    out = s.cache.append(s.seqs, s.k, s.v, rope=sg.Rope(64), q=s.q)
    check_append(s, before, (odec.rope_turns(64), False, 1.0), q0, out, host(s.k), host(s.v), pos)


def test_append8_strided_and_positions():
    say("case append8 strided")
    heads, kv, dim = 6, 2, 64
    s = Setup8([5, 2], [40, 2], 16, heads, kv, dim, BF16, 6, head_major=True, block=8)
    qkv = torch.randn(s.tokens, heads + 2 * kv, dim, device="cuda").to(BF16)
    s.q, s.k, s.v = qkv[:, :heads], qkv[:, heads: heads + kv], qkv[:, heads + kv:]
    pos = [1000000, -7, 3, 3, 2 ** 31 - 1, 0, 77]
    before, q0 = state(s), host(s.q)
    out = s.cache.append(s.seqs, s.k, s.v, rope=sg.Rope(32), q=s.q, positions=ints(pos))
    check_append(s, before, (odec.rope_turns(32), False, 1.0), q0, out, host(s.k), host(s.v), pos)


def test_append8_far_into_a_large_cache():
    """Offsets beyond 2^32 bytes."""
    say("case append8 far")
    page, kv, dim = 16, 2, 64
    pages = (1 << 32) // (page * kv * dim) + 3
    k, v = (torch.zeros(pages, page, kv, dim, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn) for _ in range(2))
    cache = sg.PagedCache8.from_tensors(k, v, torch.full((pages, 1, kv, 2), 31, dtype=torch.uint8, device="cuda").view(torch.float8_e8m0fnu))
    x = torch.randn(3, kv, dim, device="cuda").half()
    seqs = sg.Sequences(ints([0, 3]), ints([3]), ints([[pages - 1]]))
    cache.append(seqs, x, -x)
    got = odec.values8(raw(k[-1:]).reshape(1, page, kv, dim), raw(cache.scales[-1:]), 0)[0, :3]
    top = 2.0 ** (raw(cache.scales[-1:])[0, 0, :, 0].astype(int) - 127)
    assert (np.abs(got - host(x)) <= np.maximum(2.0 ** -4 * np.abs(host(x)), 2.0 ** -10 * top[None, :, None])).all()
    assert not k.view(torch.uint8)[0].any()
    q = torch.randn(3, kv, dim, device="cuda").half()
    out = cache.attend(seqs, q, window=2)
    vals = [odec.values8(raw(t[-1:]).reshape(1, page, kv, dim), raw(cache.scales[-1:]), i) for i, t in enumerate((k, v))]
    ref, mean, worst, keys = odec.attend(host(q), *vals, [0, 3], [3], np.array([[0]]), dim ** -0.5, window=2)
    tol = mean * (3 * U[F16] + 2 * dim * E * worst[:, :, None] + 2 * keys[:, :, None] * E) + 3 * A[F16] * np.abs(vals[1]).max() + A[F16]
    assert (np.abs(host(out) - ref) <= tol).all()


# ------------------------------------------------------------- attention

def fits(case):
    return case[5] % 16 == 0


@pytest.mark.parametrize("case", [c for c in ATTEND if fits(c)], ids=name)
@pytest.mark.parametrize("block", [8, 32])
def test_attend8(case, block):
    n, ctx, page, heads, kv, dim, dtype, lead, trail, head_major, max_ctx = case
    say("case attend8", case, block)
    s = Setup8(n, ctx, page, heads, kv, dim, dtype, 5, lead, trail, head_major, block=block)
    want = s.want()
    out = torch.full_like(s.q, 55.0)
    assert s.cache.attend(s.seqs, s.q, out=out, max_ctx=max_ctx) is out
    s.check(out, want, name(case))
    mine = ~np.isnan(want[0][:, 0, 0])
    assert (host(out)[~mine] == 55.0).all(), "a row of no sequence was written"
    again = s.cache.attend(s.seqs, s.q, max_ctx=max_ctx)
    assert torch.equal(again[torch.from_numpy(mine)], out[torch.from_numpy(mine)]), "not the same bits twice"


WINDOW = [(1, 0), (7, 3), (64, 0), (100, 40), (33, 500), (2 ** 31 - 1, 5)]


@pytest.mark.parametrize("case", [c for c in ATTEND if fits(c)][::2] + [ATTEND[1]], ids=name)
@pytest.mark.parametrize("window,sinks", WINDOW)
@pytest.mark.parametrize("kind", [Setup, Setup8])
def test_attend_window(case, window, sinks, kind):
    n, ctx, page, heads, kv, dim, dtype, lead, trail, head_major, max_ctx = case
    say("case window", case, window, sinks, kind.__name__)
    s = kind(n, ctx, page, heads, kv, dim, dtype, 6, lead, trail, head_major)
    want = odec.attend(host(s.q), host(s.kc), host(s.vc), s.new_start, s.ctx, s.pages, dim ** -0.5, None, window, sinks)
    out = torch.full_like(s.q, 55.0)
    s.cache.attend(s.seqs, s.q, out=out, max_ctx=max_ctx, window=window, sinks=sinks)
    s.check(out, want, name(case))
    mine = ~np.isnan(want[0][:, 0, 0])
    assert (host(out)[~mine] == 55.0).all(), "a row of no sequence was written"


@pytest.mark.parametrize("n,ctx", TREE)
@pytest.mark.parametrize("window,sinks", [(0, 0), (1, 0), (3, 2), (40, 0), (300, 70)])
@pytest.mark.parametrize("kind", [Setup, Setup8])
def test_attend_tree_window(n, ctx, window, sinks, kind):
    say("case tree window", n, ctx, window, sinks, kind.__name__)
    dim, heads, kv = (128, 4, 2) if len(n) % 2 else (64, 3, 3)
    s = kind(n, ctx, 16, heads, kv, dim, F16, 7)
    rng = np.random.default_rng(8)
    words = (max(n) + 31) // 32 + 1
    bits = np.zeros((s.tokens, words), np.uint32)
    for q in range(len(n)):
        for i in range(n[q]):
            up, j = {i}, i
            while j:
                j = (j - 1) // 2
                up.add(j)
            if i % 5 == 4:
                up = set(np.flatnonzero(rng.random(n[q]) < 0.3).tolist())
            for j in up:
                bits[s.new_start[q] + i, j // 32] |= np.uint32(1) << np.uint32(j % 32)
    want = odec.attend(host(s.q), host(s.kc), host(s.vc), s.new_start, s.ctx, s.pages, dim ** -0.5, bits, window, sinks)
    got = s.cache.attend(s.seqs, s.q, tree=ints(bits.view(np.int32)), window=window, sinks=sinks)
    s.check(got, want, f"tree {n} {ctx} {window} {sinks}")


@pytest.mark.parametrize("n,ctx,heads,kv", [([1], [300], 2, 2), ([3], [1500], 4, 2), ([60], [200], 2, 1), ([90], [1200], 4, 2), ([300], [700], 1, 1)])
def test_attend8_unseen_slots_have_no_part(n, ctx, heads, kv):
    """NaN codes behind the end and outside the window, and any scales in blocks that no token sees."""
    say("case attend8 unseen", n, ctx)
    s = Setup8(n, ctx, 16, heads, kv, 64, F16, 9, spare=3)
    first = ctx[0] - n[0]
    window, sinks = 50, 9
    got = s.cache.attend(s.seqs, s.q, window=window, sinks=sinks)
    plain = s.cache.attend(s.seqs, s.q)
    bad = np.zeros((s.n_pages, 16), bool)
    block = np.zeros((s.n_pages, 2), bool)
    bad[s.unused], block[s.unused] = True, True
    low = first + 1 - window
    for t in range(s.pages.shape[1] * 16):
        at = s.pages[0, t // 16], t % 16
        if t >= ctx[0] or sinks <= t < low:
            bad[at] = True
    hidden = bad.reshape(s.n_pages, 2, 8).all(2)
    for c in (s.k8, s.v8):
        c.view(torch.uint8)[torch.from_numpy(bad).cuda()] = 0x7F
    for e in (0, 254, 255):
        s.scales.view(torch.uint8)[torch.from_numpy(hidden).cuda()] = e
        again = s.cache.attend(s.seqs, s.q, window=window, sinks=sinks)
        assert not torch.isnan(again).any()
        want = odec.attend(host(s.q), np.nan_to_num(host(s.kc)), np.nan_to_num(host(s.vc)), s.new_start, s.ctx, s.pages, 0.125, None, window, sinks)
        s.check(again, want, f"scales of {e}")
    # pages out of the window may be given back
    gone = [i for i in range(s.pages.shape[1]) if 16 * i >= sinks and 16 * (i + 1) <= low]
    pages = s.pages.copy()
    pages[0, gone] = -1
    s.seqs.pages.copy_(ints(pages))
    assert torch.equal(s.cache.attend(s.seqs, s.q, window=window, sinks=sinks), again)
    assert not torch.isnan(got).any() and not torch.isnan(plain).any()


# the few-row kernel, its short tiles of more rows, tiles of 128 rows (windows of more than its 2048 or 4096 slots) and of 256
HIDDEN = [(1, 300, 2, 2, 64, 50, 9), (3, 1500, 4, 2, 128, 50, 9), (60, 200, 2, 1, 64, 50, 9), (30, 2700, 2, 1, 64, 2100, 5),
          (25, 5200, 4, 1, 128, 4300, 40), (90, 1200, 4, 2, 128, 50, 9), (300, 700, 1, 1, 256, 200, 70), (150, 900, 2, 1, 64, 100, 0)]


@pytest.mark.parametrize("n,ctx,heads,kv,dim,window,sinks", HIDDEN)
@pytest.mark.parametrize("tree", [False, True])
@pytest.mark.parametrize("kind,dtype", [(Setup, F16), (Setup, BF16), (Setup8, F16)])
def test_what_a_window_hides_has_no_part(n, ctx, heads, kv, dim, window, sinks, tree, kind, dtype):
    """Not numbers and infinities in every slot that no token sees, then anything in the table's entries of pages without another."""
    say("case hidden", n, ctx, window, sinks, tree, kind.__name__, dtype)
    s = kind([n], [ctx], 16, heads, kv, dim, dtype, 23, spare=3)
    old, bits = ctx - n, None
    low = old + 1 - window
    if tree:
        bits = np.zeros((n, (n + 31) // 32), np.uint32)
        path = []
        for i in range(n):
            up, j = {i}, i
            while j:
                j = (j - 1) // 2
                up.add(j)
            for j in up:
                bits[i, j // 32] |= np.uint32(1) << np.uint32(j % 32)
            path.append(len(up))
        low = min(old, old + min(path) - window)
    hide = np.ones((s.n_pages, 16), bool)
    for t in list(range(max(low, 0), ctx)) + list(range(min(sinks, ctx))):
        hide[s.pages[0, t // 16], t % 16] = False
    at = torch.from_numpy(hide).cuda()
    if kind is Setup8:
        for c in (s.k8, s.v8):
            c.view(torch.uint8)[at] = 0x7F
        clean = [np.nan_to_num(host(x)) for x in (s.kc, s.vc)]
    else:
        clean = [host(x) for x in (s.kc, s.vc)]
        odd = torch.tensor([float("nan"), float("inf"), -float("inf")], device="cuda", dtype=dtype)
        for c in (s.kc, s.vc):
            c[at] = odd[torch.randint(0, 3, c[at].shape, device="cuda")]
    want = odec.attend(host(s.q), *clean, s.new_start, s.ctx, s.pages, dim ** -0.5, bits, window, sinks)
    kw = dict(tree=None if bits is None else ints(bits.view(np.int32)), window=window, sinks=sinks)
    s.check(s.cache.attend(s.seqs, s.q, **kw), want, "hidden slots")
    pages = s.pages.copy()
    gone = [i for i in range(pages.shape[1]) if 16 * i >= sinks and 16 * (i + 1) <= low]
    pages[0, gone] = np.resize([-1, s.n_pages, 2 ** 31 - 1, -2 ** 31, s.unused[0]], len(gone))
    s.seqs.pages.copy_(ints(pages))
    s.check(s.cache.attend(s.seqs, s.q, **kw), want, "pages given back")


@pytest.mark.parametrize("n,ctx", [([1], [40]), ([20], [300]), ([150], [400])])
def test_attend8_nan_that_is_seen(n, ctx):
    say("case attend8 NaN", n, ctx)
    s = Setup8(n, ctx, 16, 2, 1, 64, F16, 10)
    s.v8.view(torch.uint8)[s.pages[0, 1], 3, 0, 5] = 0x7F
    got = host(s.cache.attend(s.seqs, s.q))
    assert np.isnan(got[:, :, 5]).all() and not np.isnan(np.delete(got, 5, 2)).any()


@pytest.mark.parametrize("n,ctx,dim", [([1], [700], 128), ([30], [300], 64), ([90], [1300], 128), ([300], [500], 256), ([260], [400], 64)])
@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("far", [14, 17, 45, 90])
def test_attend8_exponents_far_apart(n, ctx, dim, dtype, far):
    """Rows that see only blocks of small scales beside rows that see large ones."""
    say("case attend8 far exponents", n, ctx, dim, dtype, far)
    s = Setup8(n, ctx, 16, 2, 1, dim, dtype, 11, block=8)
    e = torch.full((s.n_pages, 2, 1, 2), 120 - far // 2, dtype=torch.uint8, device="cuda")
    up = 120 + (far + 1) // 2 if dtype == BF16 else 122
    e[..., 0] = 120
    if dtype == F16:
        e[..., 1] = up - min(far, 24)
    late = ctx[0] - n[0] // 2
    e[s.pages[0, late // 16], late % 16 // 8, 0, 1] = up        # seen by the last rows alone (or by the only one)
    e[s.pages[0, 0], 0, 0, 0] = 120 - min(far, 50)
    s.scales.view(torch.uint8).copy_(e)
    s.values()
    want = s.want()
    out, mean, worst, keys = want
    got = host(s.cache.attend(s.seqs, s.q))
    u, a = U[dtype], A[dtype]
    # half subnormals of the weights count by what the row itself sees: as those sums have them, n a max |v| of the row
    old = ctx[0] - n[0]
    big = np.array([max(np.abs(host(s.vc)[s.pages[0, t // 16], t % 16]).max() for t in (range(old + i + 1) if i % 7 == 0 or i == n[0] - 1 else [old + i]))
                    for i in range(n[0])])
    for i in range(n[0]):
        if not (i % 7 == 0 or i == n[0] - 1):
            continue
        tol = mean[i] * (3 * u + 2 * dim * E * worst[i][:, None] + 2 * keys[i][:, None] * E) + keys[i][:, None] * a * big[i] + a
        assert (np.abs(got[i] - out[i]) <= tol).all(), (i, (np.abs(got[i] - out[i]) - tol).max())


# rows of the many-row kernel: full tiles, and 128 rows of them (room for more than 4096 slots)
@pytest.mark.parametrize("n,dim,per", [(300, 64, None), (60, 64, 600), (300, 128, None), (60, 128, 600), (300, 256, None)])
@pytest.mark.parametrize("dtype,least,far,scale", [(F16, -62, 40, 2.0 ** 52), (F16, -75, 35, 2.0 ** 65), (BF16, -96, 130, 2.0 ** 86),
                                                   (BF16, -70, 10, 2.0 ** 60)])
def test_attend8_small_keys_under_a_large_scale(n, dim, per, dtype, least, far, scale):
    """Keys of the smallest scales, whose scores count since `scale` is large, in one block with keys of larger ones
    that only later rows see."""
    say("case attend8 large scale", n, dim, per, dtype, least, far, scale)
    s = Setup8([n], [n], 16, 2, 1, dim, dtype, 16, block=8, per_seq=per)
    assert s.cache.plan(s.seqs, n, 2).tile_rows == (128 if per and dim <= 128 else 256)
    late = 56                                              # slots 56 to 63 have the larger ones
    s.scales.view(torch.uint8)[..., 0] = 127 + least
    s.scales.view(torch.uint8)[s.pages[0, late // 16], late % 16 // 8, :, 0] = 127 + least + far
    if dtype == BF16:
        s.q[late:] *= 2.0 ** -60                           # scores that FP32 holds
    s.values()
    want = s.want(scale)
    assert want[2][:late].max() < 200                      # scores of a few units: their rows' tolerances are those of roundings
    s.check(s.cache.attend(s.seqs, s.q, scale=scale), want, f"{n} {dim} {dtype}")


# room for more than 4096 slots a sequence, which the launch goes by: the kernel for many rows, in its form for few tokens
ROOMY = [([60], [300], 16, 2, 1, 64, F16, 600), ([27, 33], [1100, 90], 16, 4, 2, 128, F16, 600), ([40], [40], 8, 3, 1, 128, BF16, 700),
         ([25, 30], [2000, 1025], 8, 8, 2, 80, F16, 700), ([20], [1200], 16, 4, 1, 256, F16, 400), ([60, 1, 0], [200, 3000, 7], 128, 3, 3, 96, BF16, 60),
         ([17], [17], 16, 1, 1, 16, F16, 600)]


@pytest.mark.parametrize("case", ROOMY, ids=lambda c: f"n{len(c[0])}x{max(c[0])}_d{c[5]}")
@pytest.mark.parametrize("block", [8, 16])
def test_attend8_tiles_of_128_rows(case, block):
    n, ctx, page, heads, kv, dim, dtype, per = case
    say("case attend8 tiles of 128", case, block)
    s = Setup8(n, ctx, page, heads, kv, dim, dtype, 13, per_seq=per, block=block, spread=6)
    assert s.cache.plan(s.seqs, s.tokens, heads).tile_rows == (128 if dim <= 128 else 256)
    s.check(s.cache.attend(s.seqs, s.q), s.want(), str(case))
    bits = np.zeros((s.tokens, 3), np.uint32)
    rng = np.random.default_rng(14)
    for q in range(len(n)):
        for i in range(n[q]):
            for j in [i] + np.flatnonzero(rng.random(n[q]) < 0.4).tolist():
                bits[s.new_start[q] + i, j // 32] |= np.uint32(1) << np.uint32(j % 32)
    s.check(s.cache.attend(s.seqs, s.q, tree=ints(bits.view(np.int32))), s.want(tree=bits), str(case) + " tree")
    # NaN where nobody looks, and exponents too far apart for one unit
    s.k8.view(torch.uint8)[torch.from_numpy(s.unused).cuda()] = 0x7F
    s.scales.view(torch.uint8)[s.pages[0, 0], 0, :, 1] = 60
    s.values()
    s.kc, s.vc = s.kc.nan_to_num(), s.vc.nan_to_num()
    s.check(s.cache.attend(s.seqs, s.q), s.want(), str(case) + " far exponents")


@pytest.mark.parametrize("kind,ctx,window", [(Setup, [2600, 150], 2100), (Setup8, [5000, 150], 4200)])
@pytest.mark.parametrize("tree", [False, True])
def test_window_tiles_of_128_rows(kind, ctx, window, tree):
    say("case window tiles of 128", kind.__name__, ctx, window, tree)
    s = kind([30, 20], ctx, 16, 2, 1, 64, F16, 15, per_seq=400)
    assert s.cache.plan(s.seqs, s.tokens, 2, window=window, sinks=5).tile_rows == 128
    bits = np.uint32(1) << (np.arange(50) % 30 % 20).astype(np.uint32) if tree else None
    bits = None if bits is None else (bits | np.uint32(3))[:, None]
    got = s.cache.attend(s.seqs, s.q, tree=None if bits is None else ints(bits.view(np.int32)), window=window, sinks=5)
    want = odec.attend(host(s.q), host(s.kc), host(s.vc), s.new_start, s.ctx, s.pages, 0.125, bits, window, 5)
    s.check(got, want, f"{ctx} {window}")


def test_attend8_cache_without_pages():
    say("case attend8 no pages")
    empty = torch.zeros(0, 16, 1, 64, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
    cache = sg.PagedCache8.from_tensors(empty, empty, torch.zeros(0, 2, 1, 2, dtype=torch.uint8, device="cuda").view(torch.float8_e8m0fnu))
    for n in (1, 200):
        seqs = sg.Sequences(ints([0, n]), ints([n + 5]), torch.zeros(1, 20, dtype=torch.int32, device="cuda"))
        q = torch.randn(n, 2, 64, device="cuda").half()
        for kw in ({}, dict(window=3, sinks=1)):
            out = torch.full_like(q, 9.0)
            assert not cache.attend(seqs, q, out=out, **kw).any()
        assert cache.append(seqs, q[:, :1], q[:, :1], rope=sg.Rope(64), q=q).shape == q.shape


def test_attend8_lengths_that_do_not_fit():
    say("case attend8 lengths")
    s = Setup8([3, 40], [50, 60], 16, 2, 1, 64, F16, 12, per_seq=4, spare=12)
    s.seqs.ctx_len.copy_(ints([10 ** 9, -5]))
    s.ctx = [10 ** 9, -5]
    for window, sinks in ((0, 0), (20, 3)):
        got = host(s.cache.attend(s.seqs, s.q, window=window, sinks=sinks))
        assert (got[3:] == 0).all() and np.isfinite(got[:3]).all()


def test_streams_and_workspace():
    say("case streams 8")
    a = Setup8([1, 1], [3000, 900], 16, 8, 2, 128, F16, 17)
    b = Setup8([70], [700], 16, 4, 2, 64, BF16, 18)
    wa, wb = a.cache.attend(a.seqs, a.q), b.cache.attend(b.seqs, b.q, window=90, sinks=3)
    room = torch.empty(a.cache.plan(a.seqs, 2, 8).workspace_bytes, dtype=torch.uint8, device="cuda")
    assert room.numel() > 0
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    got = []
    for _ in range(8):
        got.append((a.cache.attend(a.seqs, a.q, stream=s1, workspace=room), b.cache.attend(b.seqs, b.q, stream=s2, window=90, sinks=3)))
    s1.synchronize()
    s2.synchronize()
    assert all(torch.equal(x, wa) and torch.equal(y, wb) for x, y in got)
    with pytest.raises(sg.SgemvError):
        a.cache.attend(a.seqs, a.q, workspace=room[:-8])


def test_append8_lengths_that_do_not_fit():
    """A sequence longer than its row of the page table ends with that row; one below 0 has no slots."""
    say("case append8 lengths")
    a, b = (Setup8([5, 3], [64, 3], 16, 2, 2, 32, F16, 21, per_seq=4, spare=6, block=16) for _ in range(2))
    b.seqs.ctx_len.copy_(ints([10 ** 9, 3]))
    for s in (a, b):
        s.cache.append(s.seqs, s.k, s.v)
    assert all(np.array_equal(x, y) for x, y in zip(state(a), state(b)))
    before = state(a)
    a.seqs.ctx_len.copy_(ints([0, -9]))
    out = a.cache.append(a.seqs, a.k, a.v, rope=sg.Rope(32), q=a.q)
    assert all(np.array_equal(x, y) for x, y in zip(state(a), before)) and torch.isfinite(out).all()


# ------------------------------------------------------------ use together

def ragged(lists, dtype):
    start = np.concatenate([[0], np.cumsum([len(x) for x in lists])])
    return torch.tensor([v for x in lists for v in x], dtype=dtype, device="cuda"), ints(start)


def test_decode_step_in_8_bits():
    """A prompt and five steps of two beams: the append, the attention through a
    window, penalties and masks on logits, the choice of a token; every step
    against FP64 on its own inputs."""
    say("case decode step in 8 bits")
    heads, kv, dim, vocab, page, block = 4, 2, 64, 3000, 16, 8
    cache, rope = sg.PagedCache8(12, page, kv, dim, scale_slots=block), sg.Rope(dim)
    turns = odec.rope_turns(dim)
    window, sinks = 24, 3
    g = torch.Generator(device="cuda").manual_seed(3)
    prompt = torch.randn(40, kv, dim, device="cuda", generator=g).half()
    pages = np.array([[3, 1, 7, 4], [3, 1, 5, 6]])             # the beams share the prompt's whole pages
    cache.append(sg.Sequences(ints([0, 40]), ints([40]), ints(pages[:1])), prompt, prompt * 0.5, rope=rope)
    for t in (cache.k, cache.v, cache.scales):                 # and have copies of the one that goes on
        t.view(torch.uint8)[5] = t.view(torch.uint8)[7]
    seqs = sg.Sequences(ints([0, 1, 2]), ints([40, 40]), ints(pages))
    head = (0.3 * torch.randn(heads * dim, vocab, device="cuda", generator=g)).half()
    rng = np.random.default_rng(4)
    history, rep = [[1, 2], [2, 2]], torch.full((2,), 1.3, device="cuda")
    allowed = torch.from_numpy(rng.random((2, vocab)) < 0.05).cuda()
    words = torch.zeros(2, -(-vocab // 32) * 32, dtype=torch.int64, device="cuda")
    words[:, :vocab] = allowed
    words = (words.view(2, -1, 32) << torch.arange(32, device="cuda")).sum(-1)
    masks = words.where(words < 1 << 31, words - (1 << 32)).int()
    for step in range(5):
        seqs.ctx_len += 1
        q, k, v = (torch.randn(2, n, dim, device="cuda", generator=g).half() for n in (heads, kv, kv))
        before = [t.contiguous().view(torch.uint8).cpu().numpy() for t in (cache.k, cache.v, cache.scales)]
        q0 = host(q)
        cache.append(seqs, k, v, rope=rope, q=q, q_out=q)
        pos = [40 + step] * 2
        assert (np.abs(host(q) - odec.rope(q0, pos, turns)) <= 2.0 ** -19 * np.abs(q0).max() + U[F16] * np.abs(host(q)) + A[F16]).all()
        kk, vv, ss = (t.contiguous().view(torch.uint8).cpu().numpy() for t in (cache.k, cache.v, cache.scales))
        v_ref, s_ref = odec.append8(before[1], before[2], host(v), 1, [0, 1, 2], [41 + step] * 2, pages)
        assert np.array_equal(vv, v_ref) and np.array_equal(ss[..., 1], s_ref[..., 1])
        out = cache.attend(seqs, q, window=window, sinks=sinks)
        kd, vd = odec.values8(kk, ss, 0), odec.values8(vv, ss, 1)
        ref, mean, worst, keys = odec.attend(host(q), kd, vd, [0, 1, 2], [41 + step] * 2, pages, dim ** -0.5, None, window, sinks)
        tol = mean * (3 * U[F16] + 2 * dim * E * worst[:, :, None] + 2 * keys[:, :, None] * E) + keys[:, :, None] * A[F16] * 8 + A[F16]
        assert (np.abs(host(out) - ref) <= tol).all()
        ids, start = ragged(history, torch.int32)
        logits = sg.adjust_logits(out.reshape(2, -1) @ head, history=ids, history_start=start, repetition=rep, masks=masks)
        u = torch.tensor([0.2 + 0.15 * step, 0.9 - 0.1 * step], device="cuda")
        t, p = torch.tensor([0.7, 1.1], device="cuda"), torch.full((2,), 0.9, device="cuda")
        lp = torch.empty(2, device="cuda")
        got = sg.sample(logits, u, temperature=t, top_k=ints([40, 0]), top_p=p, logprob=lp)
        for b in range(2):
            want = odec.sample(host(logits)[b], float(u[b]), float(t[b]), (40, 0)[b], float(p[b]))
            assert want[2] > vocab * 2.0 ** -43 and int(got[b]) == want[0] and bool(allowed[b, int(got[b])])
            assert abs(float(lp[b]) - want[1]) <= 2.0 ** -23 * abs(want[1]) + 2.0 ** -23
        history = [h + [int(x)] for h, x in zip(history, got)]


def test_captured_step_in_8_bits():
    """The same four captured once and replayed while lengths and inputs change, eager calls in between."""
    say("case graph 8")
    heads, kv, dim, vocab = 8, 2, 128, 5000
    s = Setup8([1, 1], [1, 1], 16, heads, kv, dim, F16, 19, per_seq=80, spare=200, block=16)
    s.pages[:] = np.random.default_rng(20).permutation(160).reshape(2, 80)
    s.seqs.pages.copy_(ints(s.pages))
    rope, x = sg.Rope(dim), torch.randn(2, vocab, device="cuda").half()
    u, p, rep = torch.rand(2, device="cuda"), torch.full((2,), 0.95, device="cuda"), torch.full((2,), 1.5, device="cuda")
    hist, start = torch.zeros(64, dtype=torch.int32, device="cuda"), ints([0, 3, 9])
    now = [t.view(torch.uint8) for t in (s.k8, s.v8, s.scales)]
    first = [t.clone() for t in now]

    def step():
        q = s.cache.append(s.seqs, s.k, s.v, rope=rope, q=s.q)
        logits = sg.adjust_logits(x, history=hist, history_start=start, repetition=rep)
        return (s.cache.attend(s.seqs, q, max_ctx=1280), s.cache.attend(s.seqs, q, max_ctx=1280, window=200, sinks=4),
                sg.sample(logits, u, top_p=p))

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
        g = torch.Generator(device="cuda").manual_seed(round_)
        for t in (s.q, s.k, s.v, x):
            t.copy_(torch.randn(t.shape, device="cuda", generator=g))
        u.copy_(torch.rand(2, device="cuda", generator=g))
        hist.copy_(torch.randint(0, vocab, (64,), device="cuda", generator=g))
        for t, t0 in zip(now, first):
            t.copy_(t0)
        eager = [t.clone() for t in step()]
        cache = [t.clone() for t in now]
        for t, t0 in zip(now, first):
            t.copy_(t0)
        for gr, o in ((graph, out), (other, out2), (graph, out)):
            gr.replay()
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(o, eager))
            assert all(torch.equal(a, b) for a, b in zip(now, cache))

"""GPU parity of the choice of tokens with its FP64 oracle: tokens are whole
numbers and have to be equal. The kernel's exponentials are within 2^-45 and its
sums in whole multiples of 2^-43, so of n tokens a border is off by at most
(n + 1) 2^-43 of the sum (it is 1 at least: the largest p); a row whose borders
all lie further than that from where they would decide otherwise has one answer.
The test's inputs are chosen by the oracle alone: a row that has a border within
that distance is given another random number first, without the kernel's answer.
Shares are rounded to FP32 once: e |ref| and, of the logarithm's argument, 2^-40."""
import math

import numpy as np
import pytest

import sparse_weight_only_amd as sg
from gpu_util import say
from oracle import decode as odec
from test_gpu_decode import BF16, F16, F32, host, ints

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _device():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    sg.lib()


def per_row(v, rows, default):
    return [default] * rows if v is None else list(v)


def check(x, uniform, temperature=None, top_k=None, top_p=None, min_p=None):
    """x: a tensor [rows, vocab]; the rest: a list of a number for each row, or None."""
    rows, vocab = x.shape
    x64 = host(x)
    f32 = lambda v: None if v is None else np.asarray(v, np.float32)       # noqa: E731
    uniform, temperature, top_p, min_p = f32(uniform), f32(temperature), f32(top_p), f32(min_p)
    t, k, tp, mp = per_row(temperature, rows, 1.0), per_row(top_k, rows, 0), per_row(top_p, rows, 1.0), per_row(min_p, rows, 0.0)
    ref = []
    for r in range(rows):
        for again in range(20):
            a = odec.sample(x64[r], float(uniform[r]), float(t[r]), int(k[r]), float(tp[r]), float(mp[r]))
            if a[2] == 0 or a[2] > (vocab + 1) * 2.0 ** -43 or not 0 < uniform[r] < 1 or again == 19:
                break                                   # 0: equal weights, whose sums are exact on both sides
            uniform[r] = np.float32((uniform[r] + 0.3819) % 1.0)
        ref.append(a)
    dev = lambda v, d=torch.float32: None if v is None else torch.tensor(np.asarray(v), dtype=d, device="cuda")   # noqa: E731
    lp = torch.full((rows,), 9.0, device="cuda")
    got = sg.sample(x, dev(uniform), dev(temperature), dev(top_k, torch.int32), dev(top_p), dev(min_p), logprob=lp)
    ids, shares = [a[0] for a in ref], np.array([a[1] for a in ref])
    assert got.tolist() == ids, [(r, g, i, ref[r]) for r, (g, i) in enumerate(zip(got.tolist(), ids)) if g != i][:5]
    fine = np.isfinite(shares)
    assert np.array_equal(fine, np.isfinite(host(lp)))
    assert (np.abs(host(lp) - shares)[fine] <= 2.0 ** -24 * np.abs(shares)[fine] + vocab * 2.0 ** -43 * np.exp(-shares[fine]) + 2.0 ** -40).all()
    again = sg.sample(x, dev(uniform), dev(temperature), dev(top_k, torch.int32), dev(top_p), dev(min_p))
    assert torch.equal(again, got)
    return got


def logits(rows, vocab, dtype, seed=0, sigma=2.0, peaks=20):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = sigma * torch.randn(rows, vocab, device="cuda", generator=g)
    x += 5.0 * (torch.rand(rows, vocab, device="cuda", generator=g) < peaks / vocab)
    return x.to(dtype)


def uniforms(rows, seed=0):
    return np.random.default_rng(seed).random(rows).astype(np.float32)


SHAPES = [(1, 1), (2, 2), (3, 5), (2, 255), (2, 257), (3, 1023), (2, 4097), (4, 32000), (2, 50257), (1, 128003), (1, 200001)]


@pytest.mark.parametrize("rows,vocab", SHAPES)
@pytest.mark.parametrize("dtype", [F32, F16, BF16])
@pytest.mark.parametrize("how", ["all", "top_k", "top_p", "min_p", "together", "greedy"])
def test_sample(rows, vocab, dtype, how):
    say("case sample", rows, vocab, dtype, how)
    x, u = logits(rows, vocab, dtype, vocab), uniforms(rows, vocab)
    rng = np.random.default_rng(rows)
    t = rng.uniform(0.3, 1.5, rows)
    k, p, m = rng.integers(1, min(vocab, 60) + 1, rows), rng.uniform(0.1, 0.99, rows), rng.uniform(0.001, 0.2, rows)
    kw = dict(all={}, top_k=dict(top_k=k), top_p=dict(top_p=p), min_p=dict(min_p=m), together=dict(top_k=k, top_p=p, min_p=m),
              greedy=dict(temperature=np.zeros(rows), top_k=k))[how]
    check(x, u, **{**dict(temperature=t), **kw})


@pytest.mark.parametrize("k", [1, 2, 63, 64, 65, 300, 1000, 1024, 1025, 3000, 31999, 32000, 32001, 2 ** 31 - 1])
def test_many_and_few_candidates(k):
    say("case sample k", k)
    for dtype in (F32, BF16):
        check(logits(2, 32000, dtype, 3), uniforms(2, k), top_k=[k, k], top_p=[0.999, 0.5])
        check(logits(2, 32000, dtype, 4), uniforms(2, k + 1), temperature=[30.0, 1.0], top_k=[k, 0], top_p=[0.98, 0.9999])


@pytest.mark.parametrize("vocab", [7, 1000, 40000])
@pytest.mark.parametrize("dtype", [F32, F16])
def test_ties(vocab, dtype):
    """Equal logits count by id: at the border of top_k, of top_p, and everywhere."""
    say("case sample ties", vocab, dtype)
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randint(0, 4, (6, vocab), device="cuda", generator=g).to(dtype)
    for seed in range(3):
        u = uniforms(6, seed)
        check(x, u, top_k=[1, 2, 3, max(1, vocab // 7), vocab // 2, vocab - 1])
        check(x, u, top_p=[0.1, 0.3, 0.5, 0.7, 0.9, 0.99], temperature=[0.7] * 6)
        check(x, u, top_k=[vocab // 2] * 6, top_p=[0.11, 0.31, 0.51, 0.71, 0.91, 0.97])
    flat = torch.full((4, vocab), -3.5, dtype=dtype, device="cuda")
    check(flat, [0.0, 0.3, 0.7, 0.9999], top_p=[0.5, 0.25, 1.0, 0.75])
    check(flat, [0.0, 0.3, 0.7, 0.9999], top_k=[3, 5, 1, vocab])
    both = torch.zeros(2, vocab, device="cuda")
    both[:, ::2] = -0.0
    check(both, [0.4, 0.8], top_k=[max(1, vocab // 2), 3])


@pytest.mark.parametrize("dtype", [torch.float32, torch.float16])
@pytest.mark.parametrize("vocab", [8193, 32761, 50021])
def test_more_than_are_listed(vocab, dtype):
    # min_p leaves thousands of tokens: with top_p, with many of the largest, and alone
    say("case sample long lists", vocab, dtype)
    x, u = logits(6, vocab, dtype, vocab, peaks=0), uniforms(6, vocab + 1)
    check(x, u, min_p=[1e-7] * 6)
    check(x, u, min_p=[1e-7] * 6, top_p=[0.3, 0.6, 0.9, 0.97, 0.99, 0.5])
    check(x, u, min_p=[1e-7] * 6, top_k=[5000, 8192, 2000, 769, 40, 8000], temperature=[0.5, 3.0, 20.0, 1.0, 1.0, 100.0])


@pytest.mark.parametrize("vocab", [5003, 30522, 32000, 50257, 100277])
@pytest.mark.parametrize("dtype", [F32, F16, BF16])
def test_top_k_where_lanes_have_no_logit(vocab, dtype):
    """Lengths and masks that leave some lanes without a token, or with none but far ones."""
    say("case sample empty lanes", vocab, dtype)
    far = -6e4 if dtype == F16 else -1e9
    x = logits(9, vocab, dtype, vocab + 1)
    g = torch.Generator(device="cuda").manual_seed(vocab)
    some = torch.rand(9, vocab, device="cuda", generator=g)
    x[1, : vocab // 2] = -math.inf
    x[2].masked_fill_(some[2] < 0.9, -math.inf)
    x[3].masked_fill_(some[3] < 0.9, far)
    x[4].masked_fill_(some[4] < 0.95, torch.finfo(dtype).min)
    x[5, -vocab // 30:] = far
    x[6] = (-10.0 ** (torch.arange(vocab, device="cuda") % (4 if dtype == F16 else 38))).to(dtype).where(some[6] < 0.5, x[6])
    x[7].masked_fill_(some[7] < 0.9, math.nan)
    x[8] -= 4000.0
    for k in (1, 50, 300, 768):
        check(x, uniforms(9, k), top_k=[k] * 9)
        check(x, uniforms(9, k + 1), top_k=[k] * 9, top_p=[0.9] * 9, temperature=[1.5] * 9)
    check(x, uniforms(9, 9), top_k=[50] * 9, min_p=[1e-4] * 9)


def test_largest_vocabulary():
    """2^20 tokens: of equal logits the sums reach 2^63."""
    say("case sample 2^20")
    n = 1 << 20
    check(torch.full((3, n), 7.25, dtype=F16, device="cuda"), [0.99999, 0.5, 0.1], top_p=[0.25, 1.0, 0.75], top_k=[0, 700000, n])
    check(logits(2, n, BF16, 11), uniforms(2, 3), top_p=[0.7, 1.0], temperature=[1.1, 0.9])
    with pytest.raises(sg.SgemvError):
        sg.sample(torch.zeros(1, n + 1, device="cuda"), torch.zeros(1, device="cuda"))


def test_special_values():
    say("case sample special values")
    inf, nan = math.inf, math.nan
    x = torch.full((12, 500), -inf, device="cuda")
    x[1, 77] = -5.0
    x[2] = nan
    x[3, 400], x[3, 10] = 2.0, nan
    x[4, [3, 9, 450]] = inf
    x[4, 100] = 5.0
    x[5] = torch.finfo(F32).min
    x[6, 0], x[6, 499] = 3e38, -3e38
    x[7, [5, 6, 7]] = torch.tensor([1e-40, 2e-40, 3e-40], device="cuda")
    x[8, 498:] = 1.0
    x[9, ::2] = 0.0
    x[10, 499] = -inf
    x[10, 13] = nan
    x[10, 14] = -1e30
    x[11] = torch.linspace(-700, 0, 500)
    u = [0.1, 0.9, 0.5, 0.5, 0.7, 0.35, 0.999, 0.5, 0.5, 0.75, 0.0, 0.6]
    check(x, u)
    check(x, u, temperature=[0.0] * 12)
    check(x, u, top_k=[2] * 12, top_p=[0.9] * 12, min_p=[0.01] * 12)
    check(x, u, temperature=[0.01] * 12, top_p=[0.5] * 12)
    check(x, u, temperature=[1e-30] * 12)
    check(x[5:12], u[5:12], temperature=[1e30] * 7, top_p=[0.999] * 7)


def test_arguments_out_of_range():
    """They mean what the documentation says, row by row."""
    say("case sample arguments")
    nan, inf = math.nan, math.inf
    x = logits(8, 3000, F32, 6).expand(8, 3000).contiguous()
    x[:] = x[0]
    u = [-1.0, 0.0, 1.0, 7.0, nan, 0.999999, -inf, inf]
    check(x, u, top_p=[0.5] * 8)
    u = uniforms(8, 5)
    check(x, u, top_p=[0.0, -1.0, 1.0, 2.0, nan, inf, -inf, 1e-30])
    check(x, u, min_p=[0.0, -1.0, 1.0, 2.0, nan, inf, -inf, 1e-30])
    check(x, u, top_k=[0, -1, -2 ** 31, 2 ** 31 - 1, 1, 3000, 3001, 2999])
    check(x, u, temperature=[0.0, -1.0, nan, -inf, 1e-38, 1.0, 2.0, 0.5])


def test_strides_and_outputs():
    say("case sample strides")
    wide = logits(9, 4099, F16, 7)
    x = wide[::2, 3:4002]
    check(x, uniforms(5, 1), top_k=[40] * 5)
    y = logits(1, 999, F32, 8).expand(6, 999)
    check(y, uniforms(6, 2), top_p=[0.9] * 6)
    ids = torch.full((7,), -9, dtype=torch.int32, device="cuda")
    u = torch.rand(5, device="cuda")
    assert sg.sample(x, u, out=ids[1:6]) is not None
    assert ids[0] == -9 and ids[6] == -9 and (ids[1:6] >= 0).all()
    empty = sg.sample(x[:0], u[:0])
    assert empty.shape == (0,)


def test_shares_are_met():
    """20000 draws over 6 tokens: each one's count within five standard deviations."""
    say("case sample shares")
    x = torch.tensor([[0.3, -1.0, 1.2, 0.0, 2.0, -30.0]], device="cuda").expand(20000, 6)
    g = torch.Generator(device="cuda").manual_seed(5)
    ids = sg.sample(x, torch.rand(20000, device="cuda", generator=g), temperature=torch.full((20000,), 0.8, device="cuda"))
    p = np.exp((host(x)[0] - 2.0) / 0.8)
    p /= p.sum()
    n = np.bincount(ids.cpu().numpy(), minlength=6)
    assert (np.abs(n - 20000 * p) <= 5 * np.sqrt(20000 * p * (1 - p)) + 1).all()


def test_tensors_on_the_cpu_are_refused_by_name():
    x, u = torch.zeros(2, 50, device="cuda"), torch.zeros(2, device="cuda")
    for what, v in (("uniform", torch.zeros(2)), ("temperature", torch.zeros(2)), ("top_k", torch.zeros(2, dtype=torch.int32)), ("top_p", torch.zeros(2)),
                    ("min_p", torch.zeros(2)), ("out", torch.zeros(2, dtype=torch.int32)), ("logprob", torch.zeros(2))):
        with pytest.raises(ValueError, match=what):
            sg.sample(x, **{**dict(uniform=u), what: v})


def test_captured_and_on_another_stream():
    say("case sample graph")
    x, u = logits(4, 32000, F32, 9), torch.rand(4, device="cuda")
    p = torch.full((4,), 0.9, device="cuda")
    k = ints([50, 0, 3, 2000])
    def step():
        lp = torch.empty(4, device="cuda")
        return sg.sample(x, u, top_p=p, top_k=k, logprob=lp), lp
    step()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side), torch.cuda.graph(graph, stream=side):
        out = step()
    for seed in range(4):
        x.copy_(logits(4, 32000, F32, seed))
        u.copy_(torch.rand(4, device="cuda", generator=torch.Generator(device="cuda").manual_seed(seed)))
        p.fill_(0.5 + 0.1 * seed)
        eager = step()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out[0], eager[0]) and torch.equal(out[1], eager[1])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = sg.sample(x, u, top_p=p, top_k=k, stream=side)
    side.synchronize()
    assert torch.equal(got, eager[0])

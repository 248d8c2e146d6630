"""The cache in 8 bits and attention through a window on the CPU: the oracle's
own pins, the windows' index arithmetic under sanitizers, launch plans, and what
the entry points refuse before any HIP call."""
import ctypes
import math
import os
import subprocess

import numpy as np
import pytest

import sparse_weight_only_amd as sg
from oracle import decode as odec
from sparse_weight_only_amd import _build, decode as D
from sparse_weight_only_amd.sgemv import SGEMV_EALIGN, SGEMV_EINVAL, SGEMV_ESIZE
from test_decode_host import BASE, cache, code, rows, seqs, turn

torch = pytest.importorskip("torch")


# ------------------------------------------------------------- the oracle

def test_oracle_codes_are_torchs():
    codes = np.arange(256, dtype=np.uint8)
    want = torch.from_numpy(codes).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(odec.of_e4m3(codes), want, equal_nan=True)
    x = np.random.default_rng(0).standard_normal(20000) * np.exp(np.random.default_rng(1).uniform(-9, 4.5, 20000))
    ties = (odec.E4M3[:-1] + odec.E4M3[1:]) / 2
    x = np.concatenate([np.clip(x, -448, 448), ties, -ties, odec.E4M3, [448.0, -448.0, -0.0]]).astype(np.float32)
    assert np.array_equal(odec.to_e4m3(x), torch.from_numpy(x).to(torch.float8_e4m3fn).view(torch.uint8).numpy())
    assert odec.to_e4m3([math.nan, math.inf, -math.inf]).tolist() == [0x7F] * 3


def test_oracle_exponents():
    for a, e in ((0.0, -96), (448.0, 0), (448.0001, 1), (224.0, -1), (1.0, -8), (3.5, -7), (3.5001, -6), (1e-40, -96), (3e38, 120)):
        assert odec.exponent8(a) == e, (a, e)


def test_oracle_append8_by_hand():
    # blocks of 8 slots; slot 0 holds 448 2^-7 = 3.5, then 7 comes (needs 2^-6), then 1 in a new block
    codes, scales = np.zeros((1, 16, 1, 1), np.uint8), np.full((1, 2, 1, 2), 99, np.uint8)
    pages = np.array([[0]])
    c, s = odec.append8(codes, scales, np.array([[[3.5]]]), 0, [0, 1], [1], pages)
    assert odec.of_e4m3(c[0, 0, 0, 0]) == 448 and s[0, 0, 0].tolist() == [120, 99]
    c, s = odec.append8(c, s, np.array([[[7.0]]]), 0, [0, 1], [2], pages)
    assert odec.of_e4m3(c[0, :2, 0, 0]).tolist() == [224, 448] and s[0, 0, 0, 0] == 121
    c, s = odec.append8(c, s, np.array([[[0.01]]]), 0, [0, 1], [3], pages)
    assert s[0, 0, 0, 0] == 121 and abs(odec.values8(c, s, 0)[0, 2, 0, 0] - 0.01) <= 0.01 / 16
    c, s = odec.append8(c, s, np.array([[[1.0]]]), 0, [0, 1], [9], pages)
    assert s[0, 1, 0, 0] == 119 and odec.values8(c, s, 0)[0, [0, 1, 8], 0, 0].tolist() == [3.5, 7.0, 1.0]
    # of no page, and below slot 0
    for n, ctx, table in (([0, 1], [9], [[5]]), ([0, 2], [1], [[0]])):
        d, u = odec.append8(c, s, np.full((n[1], 1, 1), 2.0), 1, n, ctx, np.array(table))
        assert (d != c).sum() == (1 if table == [[0]] else 0)


def test_oracle_window_by_hand():
    k = np.zeros((1, 8, 1, 1))
    v = np.arange(8.0).reshape(1, 8, 1, 1)
    def of(n, ctx, **kw):
        return odec.attend(np.zeros((n, 1, 1)), k, v, [0, n], [ctx], np.array([[0]]), 1.0, **kw)[0][:, 0, 0]
    assert of(1, 8, window=3).tolist() == [6.0]
    assert of(1, 8, window=2, sinks=1).tolist() == [13 / 3]
    assert of(2, 8, window=1, sinks=9).tolist() == [3.0, 3.5]
    # slots 0..4 are old; token 2 sees new tokens 0 and 2: one of its window of three is left
    tree = np.array([[0], [0], [5]])
    assert of(3, 8, window=3, tree=tree).tolist() == [(2 + 3 + 4) / 3, (2 + 3 + 4) / 3, (4 + 5 + 7) / 3]
    assert of(3, 8, window=1, sinks=1, tree=tree).tolist() == [2.0, 2.0, (0 + 5 + 7) / 3]


# ------------------------------------------------------- index arithmetic

def test_window_arithmetic_under_sanitizers():
    from sparse_weight_only_amd import _build_san
    exe = _build_san.WINDOW_CHECK
    newest = max(os.path.getmtime(f) for f in (_build_san.WINDOW_SRC, os.path.join(_build.CSRC, "decode_index.hpp")))
    if not os.path.exists(exe) or os.path.getmtime(exe) < newest:
        _build_san.build_index_check()
    r = subprocess.run([exe], stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.startswith("ok"), r.stdout[-3000:]


# ------------------------------------------------------------- C refusals

def cache8(**kw):
    a = dict(k=BASE, v=BASE, scales=BASE, k_page=16 * 2 * 64, k_slot=2 * 64, k_head=64, v_page=16 * 2 * 64, v_slot=2 * 64, v_head=64,
             pages=6, page_size=16, heads=2, head_dim=64, scale_slots=16)
    a.update(kw)
    return D.Cache8(**a)


def call(name, *args):
    """The status of an entry point; structures by reference."""
    args = [ctypes.byref(a) if isinstance(a, ctypes.Structure) else a for a in args]
    return getattr(sg.lib(), name)(*args)


def attend8(c=None, s=None, q=None, out=None, scale=0.1, tree=None, words=0, window=0, sinks=0, max_ctx=0, ws=None, room=0):
    return call("sgemv_attend8", c or cache8(), s or seqs(), q or rows(), out or rows(), scale, tree, words, window, sinks, max_ctx, ws, room, None)


def attend_window(c=None, s=None, q=None, out=None, scale=0.1, tree=None, words=0, window=9, sinks=0, max_ctx=0, ws=None, room=0):
    return call("sgemv_attend_window", c or cache(), s or seqs(), q or rows(), out or rows(), scale, tree, words, window, sinks, max_ctx, ws, room,
                None)


def append8(c=None, s=None, r=None, pos=None, q=None, q_out=None, k=None, v=None):
    return call("sgemv_append8", c or cache8(), s or seqs(), r, pos, q, q_out, k or rows(), v or rows(), None)


@pytest.mark.parametrize("bad,want", [
    (dict(pages=-1), SGEMV_EINVAL), (dict(page_size=4), SGEMV_EINVAL), (dict(page_size=24), SGEMV_EINVAL), (dict(page_size=1 << 17), SGEMV_EINVAL),
    (dict(heads=0), SGEMV_EINVAL), (dict(head_dim=56), SGEMV_EINVAL), (dict(head_dim=0), SGEMV_EINVAL), (dict(head_dim=272), SGEMV_EINVAL),
    (dict(scale_slots=4), SGEMV_EINVAL), (dict(scale_slots=0), SGEMV_EINVAL), (dict(scale_slots=12), SGEMV_EINVAL), (dict(scale_slots=32), SGEMV_EINVAL),
    (dict(scale_slots=256, page_size=256), SGEMV_EINVAL), (dict(k_page=8), SGEMV_EINVAL), (dict(v_slot=-128), SGEMV_EINVAL),
    (dict(v_head=72), SGEMV_EINVAL), (dict(k_slot=136), SGEMV_EINVAL), (dict(k=0), SGEMV_EINVAL), (dict(v=0), SGEMV_EINVAL), (dict(scales=0), SGEMV_EINVAL),
    (dict(k=BASE + 8), SGEMV_EALIGN), (dict(v=BASE + 2), SGEMV_EALIGN), (dict(scales=BASE + 1), SGEMV_EALIGN),
    (dict(k_page=-1024), SGEMV_EINVAL), (dict(k_page=1 << 62), SGEMV_EINVAL)])
def test_cache8_refused(bad, want):
    assert append8(cache8(**bad)) == want
    assert attend8(cache8(**bad)) == want
    assert call("sgemv_attend8_plan", cache8(**bad), seqs(), 5, 2, 0, 0, 0, D.AttendPlan()) == want


def test_strides_that_do_not_fit_the_kernels_are_refused():
    assert attend8(cache8(k_slot=1 << 28, k_page=1 << 35)) == SGEMV_ESIZE
    assert attend8(cache8(v_page=1 << 31)) == SGEMV_ESIZE
    assert append8(cache8(k_slot=0)) == SGEMV_EINVAL            # written slots may not overlap


@pytest.mark.parametrize("window,sinks", [(-1, 0), (0, 1), (0, -1), (5, -1)])
def test_windows_refused(window, sinks):
    assert attend8(window=window, sinks=sinks) == SGEMV_EINVAL
    assert attend_window(window=window, sinks=sinks) == SGEMV_EINVAL
    assert call("sgemv_attend8_plan", cache8(), seqs(), 5, 2, window, sinks, 0, D.AttendPlan()) == SGEMV_EINVAL
    assert call("sgemv_attend_window_plan", cache(), seqs(), 5, 2, window, sinks, 0, D.AttendPlan()) == SGEMV_EINVAL


def test_operands_that_do_not_fit_are_refused():
    E = SGEMV_EINVAL
    for f in (attend8, attend_window):
        for other in (dict(tokens=4), dict(heads=1), dict(head_dim=48), dict(dtype=D.BF16)):
            assert f(out=rows(**other)) == E
        for scale in (0.0, -1.0, math.nan, math.inf, 2e30):
            assert f(scale=scale) == E
        assert f(q=rows(heads=3), out=rows(heads=3)) == E
        assert f(q=rows(dtype=D.F32), out=rows(dtype=D.F32)) == E
        assert f(tree=BASE, words=-1) == E and f(words=1) == E and f(tree=BASE + 2, words=1) == SGEMV_EALIGN
        assert f(max_ctx=-1) == E
        assert f(s=seqs(count=-1)) == E and f(s=seqs(ctx_len=BASE + 1)) == SGEMV_EALIGN
        big = seqs(pages_per_seq=1000, pages_stride=1000)
        far = dict(s=big, window=9000)
        assert f(**far) == E and f(**far, ws=BASE, room=16) == SGEMV_ESIZE and f(**far, ws=BASE + 8, room=1 << 30) == SGEMV_EALIGN
    # 16 bits: the queries' type is the cache's
    assert attend_window(q=rows(dtype=D.BF16), out=rows(dtype=D.BF16)) == E
    r = turn()
    assert append8(r=r, q=rows()) == E and append8(r=r, q_out=rows()) == E and append8(q=rows(), q_out=rows()) == E
    assert append8(k=rows(heads=3), v=rows(heads=3)) == E and append8(v=rows(tokens=4)) == E
    assert append8(k=rows(dtype=D.BF16)) == E and append8(k=rows(dtype=D.F32), v=rows(dtype=D.F32)) == E
    assert append8(k=rows(head_dim=48), v=rows(head_dim=48)) == E
    assert append8(r=r, q=rows(tokens=4), q_out=rows(tokens=4)) == E and append8(r=r, q=rows(dtype=D.BF16), q_out=rows(dtype=D.BF16)) == E
    assert append8(r=r, q=rows(heads=6), q_out=rows(heads=4)) == E
    assert append8(r=r, q=rows(), q_out=rows(head_stride=0)) == E
    assert append8(r=turn(rot_dim=66)) == E and append8(r=turn(turns=BASE + 4)) == SGEMV_EALIGN and append8(r=r, pos=BASE + 2) == SGEMV_EALIGN
    many = rows(tokens=1 << 24, head_stride=64, token_stride=128)
    assert append8(k=many, v=many) == SGEMV_ESIZE
    assert append8(s=seqs(pages=0)) == E


def test_null_structures_are_refused():
    s, r, pl = seqs(), rows(), D.AttendPlan()
    assert call("sgemv_append8", None, s, None, None, None, None, r, r, None) == SGEMV_EINVAL
    assert call("sgemv_append8", cache8(), None, None, None, None, None, r, r, None) == SGEMV_EINVAL
    assert call("sgemv_append8", cache8(), s, None, None, None, None, r, None, None) == SGEMV_EINVAL
    for name, c in (("sgemv_attend8", cache8()), ("sgemv_attend_window", cache())):
        for args in ((None, s, r, r), (c, None, r, r), (c, s, None, r), (c, s, r, None)):
            assert call(name, *args, 0.1, None, 0, 5, 0, 0, None, 0, None) == SGEMV_EINVAL
        assert call(name + "_plan", c, s, 5, 2, 5, 0, 0, None) == SGEMV_EINVAL
        assert call(name + "_plan", None, s, 5, 2, 5, 0, 0, pl) == SGEMV_EINVAL
        assert call(name + "_plan", c, None, 5, 2, 5, 0, 0, pl) == SGEMV_EINVAL


def test_nothing_to_do_is_no_launch():
    # without a GPU a launch would report SGEMV_EHIP
    no_seqs, none = seqs(count=0, new_start=0, ctx_len=0, pages=0), rows(tokens=0, data=0)
    assert append8(s=no_seqs) == 0 and append8(k=none, v=none) == 0
    assert attend8(s=no_seqs) == 0 and attend8(q=none, out=none) == 0
    assert attend_window(s=no_seqs) == 0 and attend_window(q=none, out=none) == 0


def test_plans():
    """A window shapes the launch as a context of its length does."""
    s = seqs(pages_per_seq=8192, pages_stride=8192)
    def plan(name, c, *a):
        pl = D.AttendPlan()
        assert call(name, c, s, *a, pl) == 0
        return pl.as_dict()
    whole, as16 = plan("sgemv_attend8_plan", cache8(), 3, 8, 0, 0, 0), plan("sgemv_attend_plan", cache(), 3, 8, 0)
    assert whole == as16 and whole["splits"] > 1
    near = plan("sgemv_attend8_plan", cache8(), 3, 8, 1000, 4, 0)
    assert near == plan("sgemv_attend_window_plan", cache(), 3, 8, 1000, 4, 0)
    assert near["splits"] < whole["splits"] and near["splits"] <= 1005 // 64 + 1
    assert plan("sgemv_attend8_plan", cache8(), 3, 8, 2 ** 31 - 1, 2 ** 31 - 1, 0) == whole
    assert plan("sgemv_attend_window_plan", cache(), 3, 8, 0, 0, 0) == as16


# ---------------------------------------------------------------- binding

def test_windows_past_32_bits_are_not_cut():
    """A window or sinks of more than 32 bits is all there is, and one far below 0 is refused, not what its low bits say."""
    s = sg.Sequences(*(torch.zeros(n, dtype=torch.int32) for n in ((2,), (1,), (1, 40960))))
    for cache_ in (sg.PagedCache(4, 16, 2, 64, device="cpu"), sg.PagedCache8(4, 16, 2, 64, device="cpu")):
        def splits(**kw):
            return cache_.plan(s, 1, 2, **kw).splits
        whole = splits(window=2 ** 31 - 1)
        assert whole == splits() > splits(window=5)
        for n in (2 ** 31, 2 ** 32 + 5, 10 ** 30):
            assert splits(window=n) == splits(window=5, sinks=n) == whole, n
            for kw in (dict(window=-n), dict(window=5, sinks=-n), dict(sinks=n)):
                with pytest.raises(sg.SgemvError) as e:
                    splits(**kw)
                assert e.value.code == SGEMV_EINVAL
        for seen in ((2 ** 32 + 5, 0), (7, 2 ** 32), (-2 ** 32 + 5, 0)):      # what attend() passes on is what plan() does
            given = cache_._attend(*seen)[2]
            assert all(-2 ** 31 <= g < 2 ** 31 and (g < 0) == (n < 0) and (g == n or abs(n) >= 2 ** 31) for g, n in zip(given, seen))


def test_binding_refuses_what_it_cannot_pass_on():
    b8 = lambda *shape: torch.zeros(shape, dtype=torch.uint8).view(torch.float8_e4m3fn)    # noqa: E731
    e8 = lambda *shape: torch.zeros(shape, dtype=torch.uint8).view(torch.float8_e8m0fnu)   # noqa: E731
    k = b8(4, 16, 2, 64)
    ok = sg.PagedCache8.from_tensors(k, k, e8(4, 2, 2, 2))
    assert ok.args.scale_slots == 8 and ok.args.k_slot == 128 and ok.args.k_page == 2048
    for args in ((k.view(torch.uint8), k, e8(4, 2, 2, 2)), (k, b8(4, 16, 2, 32), e8(4, 2, 2, 2)), (k[0], k[0], e8(4, 2, 2, 2)),
                 (k.transpose(2, 3), k.transpose(2, 3), e8(4, 2, 64, 2)), (k, k, e8(4, 2, 2)), (k, k, e8(4, 3, 2, 2)), (k, k, e8(4, 2, 2, 1)),
                 (k, k, e8(5, 2, 2, 2)), (k, k, e8(4, 2, 2, 2).view(torch.uint8)), (k, k, e8(4, 2, 2, 4)[..., ::2]), (k, k, e8(4, 0, 2, 2))):
        with pytest.raises(ValueError):
            sg.PagedCache8.from_tensors(*args)
    for n in (0, 24, -8):
        with pytest.raises(ValueError):
            sg.PagedCache8(4, 16, 2, 64, n, device="cpu")
    made = sg.PagedCache8(4, 16, 2, 64, device="cpu")
    assert made.args.scale_slots == 16 and made.k.dtype == torch.float8_e4m3fn and made.scales.shape == (4, 1, 2, 2)
    head_major = b8(4, 2, 16, 64).transpose(1, 2)
    assert sg.PagedCache8.from_tensors(head_major, head_major, e8(4, 2, 2, 2)).args.k_head == 16 * 64
    s = sg.Sequences(*(torch.zeros(n, dtype=torch.int32) for n in ((2,), (1,), (1, 4))))
    q = torch.zeros(1, 2, 64, dtype=torch.float16)
    for f in (lambda: made.attend(s, q), lambda: made.append(s, q, q), lambda: made.attend(s, q, window=4)):
        with pytest.raises(ValueError, match="not on a GPU"):
            f()
    assert made.plan(s, 1, 2).splits == 1 and made.plan(s, 1, 2, window=3, sinks=1).splits == 1
    with pytest.raises(sg.SgemvError) as e:
        made.plan(s, 1, 2, sinks=1)
    assert e.value.code == SGEMV_EINVAL

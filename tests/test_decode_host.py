"""The decode-step operators on the CPU: their FP64 oracle's own pins, the
frequency table, the index arithmetic under sanitizers, launch plans, and what
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

torch = pytest.importorskip("torch")


# ------------------------------------------------------------- the oracle

def test_oracle_rope_is_a_complex_turn():
    rng = np.random.default_rng(0)
    turns = odec.rope_turns(6, base=100.0)
    x = rng.standard_normal((4, 2, 8))
    pos = [0, 1, 17, -5]
    for inter in (False, True):
        y = odec.rope(x, pos, turns, inter, 1.5)
        i0, i1 = ([0, 2, 4], [1, 3, 5]) if inter else ([0, 1, 2], [3, 4, 5])
        z = 1.5 * (x[..., i0] + 1j * x[..., i1]) * np.exp(2j * np.pi * np.array(pos)[:, None, None] * turns)
        assert np.allclose(y[..., i0], z.real, atol=1e-13) and np.allclose(y[..., i1], z.imag, atol=1e-13)
        assert np.array_equal(y[..., 6:], x[..., 6:])
    assert np.array_equal(odec.rope(x, [0] * 4, turns), x)


def test_oracle_attend_by_hand():
    # one head of two columns, page size 2: slots 0..2 of sequence 0 in pages 1, 0
    k = np.zeros((2, 2, 1, 2))
    v = np.zeros((2, 2, 1, 2))
    k[1, 0, 0], k[1, 1, 0], k[0, 0, 0] = [1, 0], [0, 1], [1, 1]
    v[1, 0, 0], v[1, 1, 0], v[0, 0, 0] = [4, 0], [0, 8], [2, 2]
    q = np.array([[[math.log(3.0), 0.0]], [[0.0, 0.0]]])
    pages = np.array([[1, 0]])
    out, _, _, keys = odec.attend(q, k, v, [0, 2], [3], pages, 1.0)
    # token 0 (slot 1): weights 3, 1; token 1 (slot 2): equal weights
    assert np.allclose(out[0, 0], [3.0, 2.0]) and np.allclose(out[1, 0], [2.0, 10 / 3])
    assert keys.tolist() == [[2], [3]]
    # candidates that see the old slot 0 and themselves only
    out, _, _, _ = odec.attend(q, k, v, [0, 2], [3], pages, 1.0, tree=np.array([[1], [2]]))
    assert np.allclose(out[0, 0], [3.0, 2.0]) and np.allclose(out[1, 0], [3.0, 1.0])
    out, _, _, _ = odec.attend(q, k, v, [0, 2], [3], np.array([[-1, 7]]), 1.0)
    assert np.array_equal(out, np.zeros_like(out))


def test_oracle_logits_by_hand():
    x = np.array([[2.0, -2.0, 1.0, 0.0, 5.0]])
    y = odec.adjust_logits(x, [[0, 1, 1, 0, 4, 9, -1]], [3], [2.0], [0.5], [0.25], [[(2, 1.0), (2, 7.0)]], [[1, 1, 1, 1, 0]])
    # behind the prompt: 0 and 4 once each; 9 and -1 are no tokens
    assert y.tolist() == [[1.0 - 0.75, -4.0, 2.0, 0.0, -np.inf]]


# ------------------------------------------------------- frequency table

@pytest.mark.parametrize("args", [(2, 10000.0, 1.0, 0.0, 1.0, 32.0), (128, 10000.0, 8.0, 0.0, 1.0, 32.0),
                                  (64, 500000.0, 8.0, 8192.0, 1.0, 4.0), (256, 1e6, 40.0, 4096.0, 1.0, 32.0), (34, 10.0, 0.5, 7.0, -1.0, 0.5)])
def test_rope_table(args):
    rot, base, factor, context, low, high = args
    got = sg.rope_table(rot, base, factor, context, low, high)
    want = odec.rope_turns(rot, base, factor, context, low, high)
    # pow, a division and up to five more FP64 operations, each within an ulp or two
    assert got.shape == (rot // 2,) and np.all(np.abs(got - want) <= 2.0 ** -48 * np.abs(want))


@pytest.mark.parametrize("args", [(3,), (0,), (258,), (-2,), (8, 0.0), (8, -1.0), (8, math.inf), (8, math.nan), (8, 1e4, 0.0), (8, 1e4, math.nan),
                                  (8, 1e4, 2.0, -1.0), (8, 1e4, 2.0, math.inf), (8, 1e4, 2.0, 10.0, 4.0, 4.0), (8, 1e4, 2.0, 10.0, math.nan, 4.0)])
def test_rope_table_refusals(args):
    with pytest.raises(sg.SgemvError) as e:
        sg.rope_table(*args)
    assert e.value.code == SGEMV_EINVAL


# ------------------------------------------------------- index arithmetic

def test_index_arithmetic_under_sanitizers():
    from sparse_weight_only_amd import _build_san
    exe = _build_san.INDEX_CHECK
    newest = max(os.path.getmtime(f) for f in (_build_san.INDEX_SRC, os.path.join(_build.CSRC, "decode_index.hpp")))
    if not os.path.exists(exe) or os.path.getmtime(exe) < newest:
        _build_san.build_index_check()
    r = subprocess.run([exe], stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.startswith("ok"), r.stdout[-3000:]


# ------------------------------------------------------------- C refusals

BASE = 1 << 20     # an aligned address that nothing reads


def cache(**kw):
    a = dict(k=BASE, v=BASE, k_page=16 * 2 * 64, k_slot=2 * 64, k_head=64, v_page=16 * 2 * 64, v_slot=2 * 64, v_head=64,
             pages=10, page_size=16, heads=2, head_dim=64, dtype=D.F16)
    a.update(kw)
    return D.Cache(**a)


def seqs(**kw):
    a = dict(new_start=BASE, ctx_len=BASE, pages=BASE, pages_stride=4, count=3, pages_per_seq=4)
    a.update(kw)
    return D.Seqs(**a)


def rows(heads=2, **kw):
    a = dict(data=BASE, token_stride=heads * 64, head_stride=64, tokens=5, heads=heads, head_dim=64, dtype=D.F16)
    a.update(kw)
    return D.Rows(**a)


def turn(**kw):
    a = dict(turns=BASE, rot_dim=64, interleaved=0, magnitude=1.0)
    a.update(kw)
    return D.RopeArgs(**a)


def code(f, *a):
    with pytest.raises(sg.SgemvError) as e:
        f(*a)
    return e.value.code


BAD_ROWS = [(dict(tokens=-1), SGEMV_EINVAL), (dict(heads=0), SGEMV_EINVAL), (dict(head_dim=60), SGEMV_EINVAL), (dict(head_dim=264), SGEMV_EINVAL),
            (dict(head_dim=0), SGEMV_EINVAL), (dict(dtype=D.F32), SGEMV_EINVAL), (dict(dtype=7), SGEMV_EINVAL), (dict(token_stride=100), SGEMV_EINVAL),
            (dict(head_stride=68), SGEMV_EINVAL), (dict(token_stride=-64), SGEMV_EINVAL), (dict(data=0), SGEMV_EINVAL), (dict(data=BASE + 8), SGEMV_EALIGN),
            (dict(token_stride=1 << 62), SGEMV_EINVAL), (dict(tokens=1 << 30), SGEMV_ESIZE)]


@pytest.mark.parametrize("bad,want", BAD_ROWS)
def test_rows_refused(bad, want):
    pos = BASE
    assert code(D.rope, turn(rot_dim=8), pos, rows(**bad), rows()) in (want, SGEMV_EINVAL)
    assert code(D.rope, turn(rot_dim=8), pos, rows(**bad), rows(**bad)) == want
    assert code(D.append, cache(), seqs(), turn(), 0, None, None, rows(**bad), rows(**bad)) in (want, SGEMV_EINVAL)
    assert code(D.attend, cache(), seqs(), rows(**bad), rows(**bad), 0.1) == want


def test_written_rows_may_not_overlap():
    for bad in (dict(head_stride=0), dict(head_stride=56), dict(token_stride=0)):
        assert code(D.rope, turn(), BASE, rows(), rows(**bad)) == SGEMV_EINVAL
        assert code(D.attend, cache(), seqs(), rows(), rows(**bad), 0.1) == SGEMV_EINVAL


@pytest.mark.parametrize("bad,want", [
    (dict(pages=-1), SGEMV_EINVAL), (dict(page_size=4), SGEMV_EINVAL), (dict(page_size=24), SGEMV_EINVAL), (dict(page_size=1 << 17), SGEMV_EINVAL),
    (dict(heads=0), SGEMV_EINVAL), (dict(head_dim=12), SGEMV_EINVAL), (dict(dtype=D.F32), SGEMV_EINVAL), (dict(k_page=4), SGEMV_EINVAL),
    (dict(v_slot=-128), SGEMV_EINVAL), (dict(v_head=33), SGEMV_EINVAL), (dict(k=0), SGEMV_EINVAL), (dict(v=0), SGEMV_EINVAL),
    (dict(k=BASE + 2), SGEMV_EALIGN), (dict(v=BASE + 8), SGEMV_EALIGN)])
def test_cache_refused(bad, want):
    assert code(D.append, cache(**bad), seqs(), turn(), 0, None, None, rows(), rows()) == want
    assert code(D.attend, cache(**bad), seqs(), rows(), rows(), 0.1) == want
    assert code(D.attend_plan, cache(**bad), seqs(), 5, 2) == want


@pytest.mark.parametrize("bad,want", [
    (dict(count=-1), SGEMV_EINVAL), (dict(pages_per_seq=-1), SGEMV_EINVAL), (dict(new_start=0), SGEMV_EINVAL), (dict(ctx_len=0), SGEMV_EINVAL),
    (dict(pages=0), SGEMV_EINVAL), (dict(pages_stride=-4), SGEMV_EINVAL), (dict(new_start=BASE + 2), SGEMV_EALIGN), (dict(ctx_len=BASE + 1), SGEMV_EALIGN),
    (dict(pages=BASE + 3), SGEMV_EALIGN)])
def test_seqs_refused(bad, want):
    assert code(D.append, cache(), seqs(**bad), turn(), 0, None, None, rows(), rows()) == want
    assert code(D.attend, cache(), seqs(**bad), rows(), rows(), 0.1) == want


@pytest.mark.parametrize("bad,want", [
    (dict(rot_dim=0), SGEMV_EINVAL), (dict(rot_dim=66), SGEMV_EINVAL), (dict(rot_dim=7), SGEMV_EINVAL), (dict(turns=0), SGEMV_EINVAL),
    (dict(interleaved=2), SGEMV_EINVAL), (dict(magnitude=0.0), SGEMV_EINVAL), (dict(magnitude=math.nan), SGEMV_EINVAL),
    (dict(magnitude=math.inf), SGEMV_EINVAL), (dict(turns=BASE + 4), SGEMV_EALIGN)])
def test_rope_refused(bad, want):
    assert code(D.rope, turn(**bad), BASE, rows(), rows()) == want
    assert code(D.append, cache(), seqs(), turn(**bad), 0, rows(), rows(), rows(), rows()) == want


def test_operands_that_do_not_fit_are_refused():
    c, s, r = cache(), seqs(), turn()
    E = SGEMV_EINVAL
    assert code(D.rope, r, 0, rows(), rows()) == E                                  # no positions
    assert code(D.rope, r, BASE + 2, rows(), rows()) == SGEMV_EALIGN
    for other in (dict(tokens=4), dict(heads=1), dict(head_dim=56), dict(dtype=D.BF16)):
        assert code(D.rope, r, BASE, rows(), rows(**other)) == E
        assert code(D.attend, c, s, rows(), rows(**other), 0.1) == E
    assert code(D.append, c, s, r, 0, rows(), None, rows(), rows()) == E            # q without q_out
    assert code(D.append, c, s, r, 0, None, rows(), rows(), rows()) == E
    assert code(D.append, c, s, None, 0, rows(), rows(), rows(), rows()) == E       # q without a rope
    assert code(D.append, c, s, r, 0, None, None, None, rows()) == E
    assert code(D.append, c, s, r, 0, None, None, rows(heads=3), rows(heads=3)) == E
    assert code(D.append, c, s, r, 0, None, None, rows(), rows(tokens=4)) == E
    assert code(D.append, c, s, r, 0, None, None, rows(dtype=D.BF16), rows(dtype=D.BF16)) == E
    assert code(D.append, c, s, r, 0, rows(tokens=4), rows(tokens=4), rows(), rows()) == E
    assert code(D.append, c, s, r, 2, None, None, rows(), rows()) == SGEMV_EALIGN
    assert code(D.append, cache(k_slot=0), s, r, 0, None, None, rows(), rows()) == E
    assert code(D.attend, c, s, rows(heads=3), rows(heads=3), 0.1) == E             # not a multiple of the cache's heads
    assert code(D.attend, c, s, rows(dtype=D.BF16), rows(dtype=D.BF16), 0.1) == E
    for scale in (0.0, -1.0, math.nan, math.inf, 2e30):
        assert code(D.attend, c, s, rows(), rows(), scale) == E
    assert code(D.attend, c, s, rows(), rows(), 0.1, BASE, -1) == E
    assert code(D.attend, c, s, rows(), rows(), 0.1, 0, 1) == E
    assert code(D.attend, c, s, rows(), rows(), 0.1, BASE + 2, 1) == SGEMV_EALIGN
    assert code(D.attend, c, s, rows(), rows(), 0.1, 0, 0, -1) == E


def test_workspace_refused():
    c, s = cache(), seqs(pages_per_seq=1000, pages_stride=1000)
    need = D.attend_plan(c, s, 5, 2).workspace_bytes
    assert need > 0 and need % 8 == 0
    assert code(D.attend, c, s, rows(), rows(), 0.1) == SGEMV_EINVAL
    assert code(D.attend, c, s, rows(), rows(), 0.1, 0, 0, 0, BASE, need - 1) == SGEMV_ESIZE
    assert code(D.attend, c, s, rows(), rows(), 0.1, 0, 0, 0, BASE + 8, need) == SGEMV_EALIGN


def test_nothing_to_do_is_no_launch():
    # without a GPU a launch would report SGEMV_EHIP
    c, s, none = cache(), seqs(count=0, new_start=0, ctx_len=0, pages=0), rows(tokens=0, data=0)
    D.rope(turn(), 0, none, none)
    D.append(c, s, turn(), 0, rows(), rows(), rows(), rows())
    D.append(c, seqs(), turn(), 0, None, None, none, none)
    D.attend(c, s, rows(), rows(), 0.1)
    D.attend(c, seqs(), none, none, 0.1)
    assert D.attend_plan(c, s, 5, 2).as_dict()["grid"] == 0
    lg = D.Logits(rows=0, vocab=5, dtype=D.F32, out_dtype=D.F32)
    assert sg.lib().sgemv_adjust_logits(ctypes.byref(lg), None) == 0


@pytest.mark.parametrize("tokens,heads,kv,dim,count,per_seq,max_ctx", [
    (1, 2, 2, 64, 1, 4, 0), (1, 8, 2, 128, 1, 8192, 0), (1, 8, 2, 128, 1, 8192, 300), (64, 32, 32, 128, 64, 100, 0), (4096, 32, 8, 128, 1, 256, 0),
    (100, 8, 1, 256, 3, 4096, 0), (300, 3, 1, 80, 300, 7, 0), (27, 8, 2, 128, 1, 400, 0), (27, 8, 2, 128, 1, 40, 0)])
def test_plan(tokens, heads, kv, dim, count, per_seq, max_ctx):
    c = cache(heads=kv, head_dim=dim, k_page=16 * kv * dim, v_page=16 * kv * dim, k_slot=kv * dim, v_slot=kv * dim, k_head=dim, v_head=dim)
    pl = D.attend_plan(c, seqs(count=count, pages_per_seq=per_seq, pages_stride=per_seq), tokens, heads, max_ctx)
    slots = tokens * (heads // kv) // pl.tile_rows + count
    assert pl.grid == slots * kv * pl.splits and 1 <= pl.splits <= 256 and pl.block in (256, 512)
    assert pl.lds_bytes <= 160 * 1024
    assert pl.workspace_bytes == (tokens * heads * pl.splits * (dim + 2) * 4 if pl.splits > 1 else 0)
    # a part of the context is worth a workgroup: two blocks of the few-row kernel, four of the other
    ctx = min(max_ctx or 1 << 30, 16 * per_seq)
    assert pl.splits == 1 or ctx // pl.splits >= (64 if pl.tile_rows == 16 else 256)


LOGITS = dict(x=BASE, out=BASE, x_stride=100, out_stride=100, rows=3, vocab=100, dtype=D.F32, out_dtype=D.F32)


@pytest.mark.parametrize("bad,want", [
    (dict(rows=-1), SGEMV_EINVAL), (dict(rows=65536), SGEMV_ESIZE), (dict(vocab=0), SGEMV_EINVAL), (dict(dtype=3), SGEMV_EINVAL),
    (dict(out_dtype=D.F16), SGEMV_EINVAL), (dict(dtype=D.F16, out_dtype=D.BF16), SGEMV_EINVAL), (dict(x=0), SGEMV_EINVAL), (dict(out=0), SGEMV_EINVAL),
    (dict(x=BASE + 2), SGEMV_EALIGN), (dict(out=BASE + 2), SGEMV_EALIGN), (dict(out_stride=99), SGEMV_EINVAL), (dict(x_stride=-100), SGEMV_EINVAL),
    (dict(dtype=D.F16), SGEMV_EINVAL),                                     # in place into another type
    (dict(x_stride=104), SGEMV_EINVAL),                                    # in place with another stride
    (dict(hist_ids=BASE, n_hist=4), SGEMV_EINVAL), (dict(hist_start=BASE, n_hist=4), SGEMV_EINVAL), (dict(hist_start=BASE, hist_ids=BASE, n_hist=-1), SGEMV_EINVAL),
    (dict(hist_start=BASE + 2, hist_ids=BASE, n_hist=4), SGEMV_EALIGN), (dict(repetition=BASE), SGEMV_EINVAL), (dict(prompt_len=BASE), SGEMV_EINVAL),
    (dict(bias_ids=BASE, bias_values=BASE, n_bias=3), SGEMV_EINVAL), (dict(bias_start=BASE, bias_ids=BASE, n_bias=3), SGEMV_EINVAL),
    (dict(bias_start=BASE, bias_ids=BASE, bias_values=BASE + 1, n_bias=3), SGEMV_EALIGN),
    (dict(masks=BASE, n_masks=0, mask_row=BASE), SGEMV_EINVAL), (dict(masks=BASE, n_masks=2, mask_stride=3, mask_row=BASE), SGEMV_EINVAL),
    (dict(masks=BASE, n_masks=2, mask_stride=4), SGEMV_EINVAL), (dict(n_masks=2), SGEMV_EINVAL), (dict(mask_row=BASE), SGEMV_EINVAL),
    (dict(masks=BASE + 2, n_masks=2, mask_stride=4, mask_row=BASE), SGEMV_EALIGN)])
def test_logits_refused(bad, want):
    g = D.Logits(**{**LOGITS, **bad})
    assert sg.lib().sgemv_adjust_logits(ctypes.byref(g), None) == want


def test_null_structures_are_refused():
    L, c, s, r = sg.lib(), cache(), seqs(), rows()
    E, ref = SGEMV_EINVAL, ctypes.byref
    assert L.sgemv_rope_table(8, 1e4, 1.0, 0.0, 1.0, 32.0, None) == E
    assert L.sgemv_rope(None, BASE, ref(r), ref(r), None) == E and L.sgemv_rope(ref(turn()), BASE, None, ref(r), None) == E
    assert L.sgemv_append(None, ref(s), ref(turn()), None, None, None, ref(r), ref(r), None) == E
    assert L.sgemv_append(ref(c), None, ref(turn()), None, None, None, ref(r), ref(r), None) == E
    assert L.sgemv_attend_plan(ref(c), ref(s), 5, 2, 0, None) == E
    assert L.sgemv_attend(None, ref(s), ref(r), ref(r), 0.1, None, 0, 0, None, 0, None) == E
    assert L.sgemv_attend(ref(c), None, ref(r), ref(r), 0.1, None, 0, 0, None, 0, None) == E
    assert L.sgemv_attend(ref(c), ref(s), None, ref(r), 0.1, None, 0, 0, None, 0, None) == E
    assert L.sgemv_adjust_logits(None, None) == E


# ------------------------------------------------- the binding's refusals

def t(*shape, dtype=torch.float16):
    return torch.zeros(shape, dtype=dtype)


def ints(*shape):
    return t(*shape, dtype=torch.int32)


def test_packed_structures():
    for structure, pack in ((D.Rows, D._pack_rows), (D.Logits, D._pack_logits)):
        values = [(7 << 33) + 3 * i if t is not ctypes.c_int32 else 5 - 2 * i for i, (_, t) in enumerate(structure._fields_)]
        packed = pack(*values)
        assert len(packed) == ctypes.sizeof(structure)
        got = structure.from_buffer_copy(packed)
        assert [getattr(got, f) for f, _ in structure._fields_] == values


def test_binding_refuses_what_it_cannot_pass_on():
    c = sg.PagedCache(4, 16, 2, 64, device="cpu")
    s = sg.Sequences(ints(3), ints(2), ints(2, 4))
    with pytest.raises(ValueError, match="not on a GPU"):
        c.attend(s, t(5, 4, 64))
    with pytest.raises(ValueError, match="not on a GPU"):
        c.append(s, t(5, 2, 64), t(5, 2, 64))
    with pytest.raises(ValueError, match="not on a GPU"):
        sg.adjust_logits(t(2, 50))
    with pytest.raises(ValueError, match="columns"):
        c.attend(s, t(5, 64, 4).transpose(1, 2))
    with pytest.raises(ValueError, match="need a rope"):
        c.append(s, t(5, 2, 64), t(5, 2, 64), q=t(5, 4, 64))
    with pytest.raises(ValueError, match="tree"):
        c.attend(s, t(5, 4, 64), tree=ints(4, 1))
    with pytest.raises(ValueError, match="int32"):
        c.attend(s, t(5, 4, 64), tree=t(5, 1, dtype=torch.int64))
    with pytest.raises(ValueError, match="new_start"):
        sg.Sequences(ints(2), ints(2), ints(2, 4))
    with pytest.raises(ValueError, match="pages"):
        sg.Sequences(ints(3), ints(2), ints(3, 4))
    with pytest.raises(ValueError, match="shape or type"):
        sg.PagedCache.from_tensors(t(4, 16, 2, 64), t(4, 16, 2, 64, dtype=torch.bfloat16))
    with pytest.raises(ValueError, match="no operator"):
        sg.PagedCache(4, 16, 2, 64, dtype=torch.float64, device="cpu")
    with pytest.raises(sg.SgemvError):
        sg.Rope(7, device="cpu")


@pytest.mark.parametrize("kw", [
    dict(history=ints(4)), dict(history_start=ints(3)), dict(history=ints(4), history_start=ints(2)), dict(history=t(4, dtype=torch.int64), history_start=ints(3)),
    dict(repetition=t(2)), dict(repetition=t(3, dtype=torch.float32)), dict(bias_ids=ints(2)), dict(bias_ids=ints(2), bias_start=ints(3), bias_values=t(3, dtype=torch.float32)),
    dict(masks=ints(2, 1)), dict(masks=ints(2, 2), mask_row=ints(3)), dict(mask_row=ints(2)), dict(out=t(2, 49)), dict(prompt_len=ints(3))])
def test_binding_refuses_logits_arguments(kw):
    with pytest.raises(ValueError):
        sg.adjust_logits(t(2, 50), **kw)

"""The operators between the GEMVs of a decode step, on torch tensors.

``PagedCache.append`` (rotary positions and the append to a paged cache),
``PagedCache.attend`` (attention of the new tokens over it), ``Rope.apply``
(rotary positions alone) and ``adjust_logits`` (penalties, biases and grammar
masks) check their tensors, marshal them into the C ABI's structures
(``include/sgemv.h``) and enqueue on the current stream or on ``stream``.
Everything is computed by the library; lengths, page tables and positions are
read on the device when the kernels run, so a captured call can be replayed
while they change. Tensors that a call makes (outputs, scratch) belong to the
stream that it runs on.
"""
from __future__ import annotations

import ctypes
import struct

import numpy as np

from .sgemv import SgemvError, _check, _ptr, lib, SGEMV_EALIGN, SGEMV_EINVAL, SGEMV_ESIZE  # noqa: F401

F16, BF16, F32 = 0, 1, 2
_P, _I32, _I64 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64


class Rows(ctypes.Structure):
    """Rows of tokens x heads x columns (mirrors sgemv_rows)."""
    _fields_ = [("data", _P), ("token_stride", _I64), ("head_stride", _I64),
                ("tokens", _I32), ("heads", _I32), ("head_dim", _I32), ("dtype", _I32)]


class Cache(ctypes.Structure):
    """A paged cache (mirrors sgemv_cache)."""
    _fields_ = [("k", _P), ("v", _P), ("k_page", _I64), ("k_slot", _I64), ("k_head", _I64),
                ("v_page", _I64), ("v_slot", _I64), ("v_head", _I64),
                ("pages", _I32), ("page_size", _I32), ("heads", _I32), ("head_dim", _I32), ("dtype", _I32)]


class Seqs(ctypes.Structure):
    """Sequences and their new tokens (mirrors sgemv_seqs)."""
    _fields_ = [("new_start", _P), ("ctx_len", _P), ("pages", _P), ("pages_stride", _I64),
                ("count", _I32), ("pages_per_seq", _I32)]


class RopeArgs(ctypes.Structure):
    """Rotary positions (mirrors sgemv_rope_t)."""
    _fields_ = [("turns", _P), ("rot_dim", _I32), ("interleaved", _I32), ("magnitude", ctypes.c_float)]


class AttendPlan(ctypes.Structure):
    """What sgemv_attend enqueues (mirrors sgemv_attend_plan_t)."""
    _fields_ = [("workspace_bytes", _I64), ("grid", _I64), ("lds_bytes", _I64),
                ("block", _I32), ("tile_rows", _I32), ("block_keys", _I32), ("splits", _I32)]

    def as_dict(self) -> dict:
        return {f: getattr(self, f) for f, _ in self._fields_}


class Logits(ctypes.Structure):
    """Penalties, biases and masks on rows of logits (mirrors sgemv_logits)."""
    _fields_ = [("x", _P), ("out", _P), ("x_stride", _I64), ("out_stride", _I64),
                ("hist_start", _P), ("hist_ids", _P), ("n_hist", _I64), ("prompt_len", _P),
                ("repetition", _P), ("frequency", _P), ("presence", _P),
                ("bias_start", _P), ("bias_ids", _P), ("bias_values", _P), ("n_bias", _I64),
                ("masks", _P), ("mask_stride", _I64), ("mask_row", _P),
                ("n_masks", _I32), ("rows", _I32), ("vocab", _I32), ("dtype", _I32), ("out_dtype", _I32)]


def rope_table(rot_dim: int, base: float = 10000.0, factor: float = 1.0, context: float = 0.0, low: float = 1.0,
               high: float = 32.0) -> np.ndarray:
    """Turns per position of each rotated pair (float64 [rot_dim / 2]); see sgemv_rope_table."""
    if not 2 <= rot_dim <= 256 or rot_dim % 2:
        _check(SGEMV_EINVAL, "sgemv_rope_table")
    out = np.empty(rot_dim // 2, dtype=np.float64)
    _check(lib().sgemv_rope_table(rot_dim, base, factor, context, low, high, _ptr(out)), "sgemv_rope_table")
    return out


def rope(rope_args: RopeArgs, positions_dev: int, x: Rows, out: Rows, stream: int = 0) -> None:
    """Enqueue rotary positions alone (raw device pointers in the structures)."""
    _check(lib().sgemv_rope(_ref(rope_args), positions_dev, _ref(x), _ref(out), stream), "sgemv_rope")


def append(cache: Cache, seqs: Seqs, rope_args, positions_dev: int, q, q_out, k: Rows, v: Rows, stream: int = 0) -> None:
    """Enqueue the append of new tokens to a cache (raw device pointers in the structures; None for what is absent)."""
    _check(lib().sgemv_append(_ref(cache), _ref(seqs), _ref(rope_args), positions_dev, _ref(q), _ref(q_out), _ref(k), _ref(v), stream), "sgemv_append")


def attend_plan(cache: Cache, seqs: Seqs, tokens: int, heads: int, max_ctx: int = 0) -> AttendPlan:
    """The launch sgemv_attend would make; no GPU needed (device pointers are not read)."""
    pl = AttendPlan()
    _check(lib().sgemv_attend_plan(_ref(cache), _ref(seqs), tokens, heads, max_ctx, _ref(pl)), "sgemv_attend_plan")
    return pl


def attend(cache: Cache, seqs: Seqs, q: Rows, out: Rows, scale: float, tree_dev: int = 0, tree_words: int = 0,
           max_ctx: int = 0, workspace_dev: int = 0, workspace_bytes: int = 0, stream: int = 0) -> None:
    """Enqueue the attention of new tokens over a cache (raw device pointers)."""
    _check(lib().sgemv_attend(_ref(cache), _ref(seqs), _ref(q), _ref(out), scale, tree_dev, tree_words, max_ctx, workspace_dev, workspace_bytes,
                              stream), "sgemv_attend")


_byref = ctypes.byref


def _ref(x):
    return None if x is None else _byref(x)


def _packer(structure):
    """A function from a structure's fields to its bytes, which cost a quarter of what the structure does."""
    codes = {_P: "P", _I64: "q", _I32: "i"}
    return struct.Struct("@" + "".join(codes[t] for _, t in structure._fields_) + "0q").pack


_pack_rows, _pack_logits = _packer(Rows), _packer(Logits)

# torch and what is looked up in it on every call, set by _init (the library's
# host side is used without torch)
torch = _types = _raw_stream = _current_device = None


def _init():
    global torch, _types, _raw_stream, _current_device
    import torch as t
    _types = {t.float16: F16, t.bfloat16: BF16, t.float32: F32}
    # the raw current stream without building a Stream object, which costs more than the rest of a call's checks
    _raw_stream = getattr(t._C, "_cuda_getCurrentRawStream", None) or (lambda i: t.cuda.current_stream(i).cuda_stream)
    _current_device = getattr(t._C, "_cuda_getDevice", None) or t.cuda.current_device
    torch = t


def _type(dtype) -> int:
    try:
        return _types[dtype]
    except KeyError:
        raise ValueError(f"no operator for {dtype}") from None


def _rows(x, what: str) -> bytes:
    """The bytes of a Rows."""
    try:
        t, h, d = x.shape
    except ValueError:
        raise ValueError(f"{what} must be [tokens, heads, head_dim]") from None
    st, sh, sd = x.stride()
    if sd != 1 and d > 1:
        raise ValueError(f"{what} must have contiguous columns")
    dtype = _types.get(x.dtype)
    if dtype is None:
        dtype = _type(x.dtype)
    return _pack_rows(x.data_ptr(), st, sh, t, h, d, dtype)


def _on(device, **tensors) -> None:
    # a call asks each tensor's get_device() first, at half the cost, and comes here to say which one differs
    for what, x in tensors.items():
        if x is not None and x.device != device:
            raise ValueError(f"{what} is on {x.device}, not on {device}")


def _ints(x, what: str, shape=None) -> None:
    if x.dtype != torch.int32 or not x.is_contiguous() or (shape is not None and x.shape != shape):
        raise ValueError(f"{what} must be a contiguous int32 tensor" + (f" of shape {list(shape)}" if shape is not None else ""))


def _enter(device, stream):
    """Makes a call's device and stream current (kernels are launched on the
    current device, and tensors made meanwhile belong to the stream): the raw
    stream, and what to leave again, None where both were current already."""
    if device.type != "cuda":
        raise ValueError(f"tensors are on {device}, not on a GPU")
    i = device.index
    if stream is None:
        if _current_device() == i:
            return _raw_stream(i), None
        ctx = torch.cuda.device(i)
        ctx.__enter__()
        return _raw_stream(i), ctx
    if stream.device != device:
        raise ValueError(f"the stream is on {stream.device}, the tensors on {device}")
    ctx = torch.cuda.stream(stream)
    ctx.__enter__()
    return stream.cuda_stream, ctx


def _leave(ctx) -> None:
    if ctx is not None:
        ctx.__exit__(None, None, None)


class Rope:
    """Rotary positions: the frequency table (on ``device``), pairing and magnitude.

    ``factor`` stretches for contexts longer than trained: every frequency
    divided by it, or, with ``context`` (the trained length), blended by the
    turns a pair makes over it, from ``low`` (divided) to ``high`` (kept).
    """

    def __init__(self, rot_dim: int, base: float = 10000.0, interleaved: bool = False, factor: float = 1.0,
                 context: float = 0.0, low: float = 1.0, high: float = 32.0, magnitude: float = 1.0, device="cuda"):
        _init()
        self.turns = torch.from_numpy(rope_table(rot_dim, base, factor, context, low, high)).to(device)
        self.args = RopeArgs(self.turns.data_ptr(), rot_dim, int(bool(interleaved)), magnitude)
        self._ref, self._index = _byref(self.args), self.turns.get_device()

    def apply(self, x, positions, out=None, stream=None):
        """x [tokens, heads, head_dim] turned at ``positions`` (int32 [tokens]) into ``out`` (a new tensor; x itself is fine)."""
        _ints(positions, "positions", (x.shape[0],))
        _on(self.turns.device, x=x, positions=positions, out=out)
        xr = _rows(x, "x")
        s, ctx = _enter(x.device, stream)
        try:
            if out is None:
                out = torch.empty(x.shape, dtype=x.dtype, device=x.device)
            code = lib().sgemv_rope(self._ref, positions.data_ptr(), xr, _rows(out, "out"), s)
        finally:
            _leave(ctx)
        if code:
            _check(code, "sgemv_rope")
        return out


class Sequences:
    """Sequences and their new tokens, as int32 tensors on the GPU.

    new_start [count + 1]: the first new token of each sequence in the packed
    rows, and their end; ctx_len [count]: tokens of each sequence, new ones
    included; pages [count, pages_per_seq]: its pages in the cache. The
    tensors are read when a kernel runs and may be rewritten between calls.
    """

    def __init__(self, new_start, ctx_len, pages):
        _init()
        count = ctx_len.shape[0]
        _ints(ctx_len, "ctx_len", (count,))
        _ints(new_start, "new_start", (count + 1,))
        if pages.dtype != torch.int32 or pages.dim() != 2 or pages.shape[0] != count or (pages.shape[1] > 1 and pages.stride(1) != 1):
            raise ValueError("pages must be an int32 tensor of shape [count, pages_per_seq] with contiguous rows")
        _on(ctx_len.device, new_start=new_start, pages=pages)
        self.new_start, self.ctx_len, self.pages = new_start, ctx_len, pages
        self.device = ctx_len.device
        self.args = Seqs(new_start.data_ptr(), ctx_len.data_ptr(), pages.data_ptr(), pages.stride(0), count, pages.shape[1])
        self._ref, self._index = _byref(self.args), ctx_len.get_device()


class PagedCache:
    """Keys and values of many sequences in pages of ``page_size`` slots
    (a power of two, 8 or more): ``k`` and ``v`` are [pages, page_size,
    heads, head_dim], FP16 or BF16."""

    def __init__(self, pages: int, page_size: int, heads: int, head_dim: int, dtype=None, device="cuda"):
        _init()
        shape = (pages, page_size, heads, head_dim)
        self._set(*(torch.zeros(shape, dtype=dtype or torch.float16, device=device) for _ in range(2)))

    @classmethod
    def from_tensors(cls, k, v) -> "PagedCache":
        """A cache over tensors of the caller's, of any strides with
        contiguous columns (a head-major cache is passed transposed)."""
        _init()
        self = cls.__new__(cls)
        self._set(k, v)
        return self

    def _set(self, k, v):
        for what, x in (("k", k), ("v", v)):
            if x.dim() != 4 or (x.shape[3] > 1 and x.stride(3) != 1):
                raise ValueError(f"{what} must be [pages, page_size, heads, head_dim] with contiguous columns")
        if k.shape != v.shape or k.dtype != v.dtype:
            raise ValueError("k and v differ in shape or type")
        _on(k.device, v=v)
        self.k, self.v, self.device = k, v, k.device
        self.args = Cache(k.data_ptr(), v.data_ptr(), *k.stride()[:3], *v.stride()[:3], *k.shape, _type(k.dtype))
        self._ref, self._index = _byref(self.args), k.get_device()

    def append(self, seqs: Sequences, k, v, rope: Rope = None, q=None, q_out=None, positions=None, stream=None):
        """Store the new tokens' k (turned by ``rope``) and v, [tokens, heads,
        head_dim], in their slots; q [tokens, query heads, head_dim] turned
        into ``q_out`` (a new tensor; q itself is fine), which is returned.
        ``positions`` (int32 [tokens]): instead of the tokens' slots."""
        if rope is None and (q is not None or positions is not None):
            raise ValueError("q and positions need a rope")
        if q is None and q_out is not None:
            raise ValueError("q_out needs q")
        dev, i = self.device, self._index
        at = qr = qo = None
        if positions is not None:
            _ints(positions, "positions", (k.shape[0],))
            at = positions.data_ptr()
        if (k.get_device() != i or v.get_device() != i or seqs._index != i or (q is not None and q.get_device() != i)
                or (q_out is not None and q_out.get_device() != i) or (rope is not None and rope._index != i)
                or (at is not None and positions.get_device() != i)):
            _on(dev, k=k, v=v, q=q, q_out=q_out, positions=positions, seqs=seqs, rope=rope and rope.turns)
        if q is not None:
            qr = _rows(q, "q")
        kr, vr = _rows(k, "k"), _rows(v, "v")
        s, ctx = _enter(dev, stream)
        try:
            if q is not None:
                if q_out is None:
                    q_out = torch.empty(q.shape, dtype=q.dtype, device=dev)
                qo = _rows(q_out, "q_out")
            code = lib().sgemv_append(self._ref, seqs._ref, None if rope is None else rope._ref, at, qr, qo, kr, vr, s)
        finally:
            _leave(ctx)
        if code:
            _check(code, "sgemv_append")
        return q_out

    def plan(self, seqs: Sequences, tokens: int, heads: int, max_ctx: int = 0) -> AttendPlan:
        """The launch that ``attend`` would make (its workspace_bytes, its splits)."""
        return attend_plan(self.args, seqs.args, tokens, heads, max_ctx)

    def attend(self, seqs: Sequences, q, scale: float = None, tree=None, out=None, max_ctx: int = 0, workspace=None,
               stream=None):
        """Attention of the new tokens q [tokens, query heads, head_dim] over
        the cache, which holds them already. scale: 1/sqrt(head_dim) unless
        given. tree (int32 [tokens, words]): bit j of a row says whether it
        sees new token j of its sequence; without it a token sees the slots up
        to its own. max_ctx: the longest context to expect (shapes the launch
        only). workspace: a uint8 tensor of ``plan(...).workspace_bytes`` or
        more, not shared with calls that may run at the same time; made if
        not given. Rows of no sequence stay as they are in a given ``out``
        and are undefined in a new one."""
        dev, i = self.device, self._index
        words = at = 0
        if tree is not None:
            _ints(tree, "tree")
            if tree.dim() != 2 or tree.shape[0] != q.shape[0]:
                raise ValueError("tree must be [tokens, words]")
            # a tree without words has no address, which would mean no tree; nothing is read of it
            words, at = tree.shape[1], tree.data_ptr() or seqs.new_start.data_ptr()
        if workspace is not None and (workspace.dtype != torch.uint8 or not workspace.is_contiguous()):
            raise ValueError("workspace must be a contiguous uint8 tensor")
        if (q.get_device() != i or seqs._index != i or (out is not None and out.get_device() != i)
                or (tree is not None and tree.get_device() != i) or (workspace is not None and workspace.get_device() != i)):
            _on(dev, q=q, seqs=seqs, tree=tree, out=out, workspace=workspace)
        qr = _rows(q, "q")
        tokens, heads, dim = q.shape
        s, ctx = _enter(dev, stream)
        try:
            if out is None:
                out = torch.empty(q.shape, dtype=q.dtype, device=dev)
            L, c, sq = lib(), self._ref, seqs._ref
            if workspace is None:
                pl = AttendPlan()
                code = L.sgemv_attend_plan(c, sq, tokens, heads, max_ctx, _byref(pl))
                if code:
                    _check(code, "sgemv_attend_plan")
                if pl.workspace_bytes:
                    workspace = torch.empty(pl.workspace_bytes, dtype=torch.uint8, device=dev)
            scratch, room = (0, 0) if workspace is None else (workspace.data_ptr(), workspace.numel())
            code = L.sgemv_attend(c, sq, qr, _rows(out, "out"), dim ** -0.5 if scale is None else scale, at, words, max_ctx,
                                  scratch, room, s)
        finally:
            _leave(ctx)
        if code:
            _check(code, "sgemv_attend")
        return out


def adjust_logits(x, out=None, history=None, history_start=None, prompt_len=None, repetition=None, frequency=None,
                  presence=None, bias_ids=None, bias_values=None, bias_start=None, masks=None, mask_row=None, stream=None):
    """Penalties, biases and grammar masks on logits x [rows, vocab] (FP16, BF16 or FP32).

    out: x's type or FP32 (a new FP32 tensor unless given; x itself is fine).
    history (int32, all rows' ids one after the other), history_start (int32
    [rows + 1]) and prompt_len (int32 [rows]: ids that are the prompt's, for
    ``repetition`` only); repetition, frequency, presence: float32 [rows];
    bias_ids, bias_values, bias_start: a ragged list as the history; masks
    (int32 [n, (vocab + 31) / 32]): bit v of a mask set where token v is
    allowed; mask_row (int32 [rows]): each row's mask, -1 for none."""
    if torch is None:
        _init()
    dev, card = x.device, x.get_device()
    rows, vocab = x.shape if x.dim() == 2 else (-1, -1)
    sx, cx = x.stride() if rows >= 0 else (0, 0)
    if rows < 0 or (cx != 1 and vocab > 1):
        raise ValueError("x must be [rows, vocab] with contiguous rows")
    if out is not None and (out.shape != x.shape or (out.stride(1) != 1 and vocab > 1) or out.device != dev):
        raise ValueError(f"out must have the shape of x, and contiguous rows, on {dev}")

    def at(t, what, n, dtype):
        if t.dtype != dtype or t.shape != n or not t.is_contiguous() or t.get_device() != card:
            raise ValueError(f"{what} must be a contiguous {dtype} tensor of shape {list(n)} on {dev}")
        return t.data_ptr()

    i32, f32 = torch.int32, torch.float32
    one, ends = (rows,), (rows + 1,)
    hist_start = hist_ids = n_hist = prompt = rep = freq = pres = 0
    b_start = b_ids = b_values = n_bias = mask_at = mask_stride = mask_rows = n_masks = 0
    if history is not None or history_start is not None:
        if history is None or history_start is None:
            raise ValueError("history and history_start belong together")
        n = history.numel()
        hist_ids, hist_start, n_hist = at(history, "history", (n,), i32), at(history_start, "history_start", ends, i32), n
    if prompt_len is not None:
        prompt = at(prompt_len, "prompt_len", one, i32)
    if repetition is not None:
        rep = at(repetition, "repetition", one, f32)
    if frequency is not None:
        freq = at(frequency, "frequency", one, f32)
    if presence is not None:
        pres = at(presence, "presence", one, f32)
    if bias_ids is not None or bias_values is not None or bias_start is not None:
        if bias_ids is None or bias_values is None or bias_start is None:
            raise ValueError("bias_ids, bias_values and bias_start belong together")
        n = bias_ids.numel()
        b_ids, b_values, n_bias = at(bias_ids, "bias_ids", (n,), i32), at(bias_values, "bias_values", (n,), f32), n
        b_start = at(bias_start, "bias_start", ends, i32)
    if masks is not None:
        words = (vocab + 31) // 32
        if masks.dtype != i32 or masks.dim() != 2 or masks.shape[1] != words or (words > 1 and masks.stride(1) != 1) or masks.device != dev:
            raise ValueError(f"masks must be an int32 tensor of shape [n, {words}] with contiguous rows on {dev}")
        if mask_row is not None:
            mask_rows = at(mask_row, "mask_row", one, i32)
        # empty tensors have no address, which would mean that there are none: rows without their masks, masks without
        # their rows
        if rows and masks.shape[0] == 0:
            raise ValueError(f"masks holds no mask for {rows} rows")
        if rows or mask_row is None:
            mask_at, mask_stride, n_masks = masks.data_ptr(), masks.stride(0), masks.shape[0]
    elif mask_row is not None:
        raise ValueError("mask_row needs masks")
    s, ctx = _enter(dev, stream)
    try:
        if out is None:
            out = torch.empty(x.shape, dtype=f32, device=dev)
        g = _pack_logits(x.data_ptr(), out.data_ptr(), sx, out.stride(0), hist_start, hist_ids, n_hist, prompt, rep, freq, pres,
                         b_start, b_ids, b_values, n_bias, mask_at, mask_stride, mask_rows, n_masks, rows, vocab, _type(x.dtype),
                         _type(out.dtype))
        code = lib().sgemv_adjust_logits(g, s)
    finally:
        _leave(ctx)
    if code:
        _check(code, "sgemv_adjust_logits")
    return out

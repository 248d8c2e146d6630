"""The operators between the GEMVs of a decode step, on torch tensors.

``PagedCache.append`` (rotary positions and the append to a paged cache),
``PagedCache.attend`` (attention of the new tokens over it, all of it or through
a window), the same of ``PagedCache8``, which holds 8 bits, ``Rope.apply``
(rotary positions alone), ``adjust_logits`` (penalties, biases and grammar
masks) and ``sample`` (the choice of tokens) check their tensors, marshal them into the C ABI's structures
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
_ALL = 2 ** 31 - 1                       # of slots: more than there can be


class Rows(ctypes.Structure):
    """Rows of tokens x heads x columns (mirrors sgemv_rows)."""
    _fields_ = [("data", _P), ("token_stride", _I64), ("head_stride", _I64),
                ("tokens", _I32), ("heads", _I32), ("head_dim", _I32), ("dtype", _I32)]


class Cache(ctypes.Structure):
    """A paged cache (mirrors sgemv_cache)."""
    _fields_ = [("k", _P), ("v", _P), ("k_page", _I64), ("k_slot", _I64), ("k_head", _I64),
                ("v_page", _I64), ("v_slot", _I64), ("v_head", _I64),
                ("pages", _I32), ("page_size", _I32), ("heads", _I32), ("head_dim", _I32), ("dtype", _I32)]


class Cache8(ctypes.Structure):
    """A paged cache in 8 bits (mirrors sgemv_cache8)."""
    _fields_ = [("k", _P), ("v", _P), ("scales", _P), ("k_page", _I64), ("k_slot", _I64), ("k_head", _I64),
                ("v_page", _I64), ("v_slot", _I64), ("v_head", _I64),
                ("pages", _I32), ("page_size", _I32), ("heads", _I32), ("head_dim", _I32), ("scale_slots", _I32)]


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


class Sampling(ctypes.Structure):
    """The choice of a token for rows of logits (mirrors sgemv_sampling)."""
    _fields_ = [("x", _P), ("x_stride", _I64), ("uniform", _P), ("temperature", _P), ("top_k", _P), ("top_p", _P), ("min_p", _P),
                ("ids", _P), ("logprob", _P), ("rows", _I32), ("vocab", _I32), ("dtype", _I32)]


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


_pack_rows, _pack_logits, _pack_sampling = _packer(Rows), _packer(Logits), _packer(Sampling)

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


def _slots(window: int, sinks: int):
    """Numbers of slots as the C ABI takes them. ctypes would keep the low 32 bits of larger ones, which are more than any
    context has, and of negative ones, which the library refuses."""
    if 0 <= window <= _ALL and 0 <= sinks <= _ALL:
        return window, sinks
    return tuple(max(-1, min(n, _ALL)) for n in (window, sinks))


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

    def _append(self):
        return lib().sgemv_append, "sgemv_append"

    def _attend(self, window, sinks):
        """The entry points of an attention, and what they take behind the arguments that all have."""
        L = lib()
        if window or sinks:
            return L.sgemv_attend_window_plan, L.sgemv_attend_window, _slots(window, sinks), "sgemv_attend_window"
        return L.sgemv_attend_plan, L.sgemv_attend, (), "sgemv_attend"

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
            call, name = self._append()
            code = call(self._ref, seqs._ref, None if rope is None else rope._ref, at, qr, qo, kr, vr, s)
        finally:
            _leave(ctx)
        if code:
            _check(code, name)
        return q_out

    def plan(self, seqs: Sequences, tokens: int, heads: int, max_ctx: int = 0, window: int = 0, sinks: int = 0) -> AttendPlan:
        """The launch that ``attend`` would make (its workspace_bytes, its splits)."""
        call, _, more, name = self._attend(window, sinks)
        pl = AttendPlan()
        _check(call(self._ref, seqs._ref, tokens, heads, *more, max_ctx, _byref(pl)), name + "_plan")
        return pl

    def attend(self, seqs: Sequences, q, scale: float = None, tree=None, out=None, max_ctx: int = 0, workspace=None,
               stream=None, window: int = 0, sinks: int = 0):
        """Attention of the new tokens q [tokens, query heads, head_dim] over
        the cache, which holds them already. scale: 1/sqrt(head_dim) unless
        given. tree (int32 [tokens, words]): bit j of a row says whether it
        sees new token j of its sequence; without it a token sees the slots up
        to its own. window: of those only the last ``window``, and the first
        ``sinks`` of the sequence (0: all), which keep the positions they were
        appended at; with a tree the new tokens that a token sees come off
        its window first, and none of them is left out.
        max_ctx: the longest context to expect (shapes the launch
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
            plan, call, more, name = self._attend(window, sinks)
            c, sq = self._ref, seqs._ref
            if workspace is None:
                pl = AttendPlan()
                code = plan(c, sq, tokens, heads, *more, max_ctx, _byref(pl))
                if code:
                    _check(code, name + "_plan")
                if pl.workspace_bytes:
                    workspace = torch.empty(pl.workspace_bytes, dtype=torch.uint8, device=dev)
            scratch, room = (0, 0) if workspace is None else (workspace.data_ptr(), workspace.numel())
            code = call(c, sq, qr, _rows(out, "out"), dim ** -0.5 if scale is None else scale, at, words, *more, max_ctx,
                        scratch, room, s)
        finally:
            _leave(ctx)
        if code:
            _check(code, name)
        return out


class PagedCache8(PagedCache):
    """A paged cache in 8 bits: ``k`` and ``v`` are float8_e4m3fn [pages,
    page_size, heads, head_dim], in units of ``scales``, float8_e8m0fnu [pages,
    page_size / scale_slots, heads, 2] (K's and V's): ``scale_slots`` slots (a
    power of two, 8 to 128) share a power of two for each head. Appended rows
    and queries are FP16 or BF16. A block of ``scale_slots`` slots that gets new
    tokens is one sequence's alone: sequences that share a prefix share whole
    blocks of it."""

    def __init__(self, pages: int, page_size: int, heads: int, head_dim: int, scale_slots: int = None, device="cuda"):
        _init()
        n = min(32, page_size) if scale_slots is None else scale_slots
        if n < 1 or page_size % n:
            raise ValueError(f"pages of {page_size} slots have no whole number of blocks of {n}")
        bits = torch.zeros((2, pages, page_size, heads, head_dim), dtype=torch.uint8, device=device)
        scales = torch.full((pages, page_size // n, heads, 2), 31, dtype=torch.uint8, device=device)
        self._set(*bits.view(torch.float8_e4m3fn), scales.view(torch.float8_e8m0fnu))

    @classmethod
    def from_tensors(cls, k, v, scales) -> "PagedCache8":
        """A cache over tensors of the caller's: ``k`` and ``v`` of any strides
        with contiguous columns, ``scales`` contiguous."""
        _init()
        self = cls.__new__(cls)
        self._set(k, v, scales)
        return self

    def _set(self, k, v, scales):
        for what, x in (("k", k), ("v", v)):
            if x.dim() != 4 or (x.shape[3] > 1 and x.stride(3) != 1) or x.dtype != torch.float8_e4m3fn:
                raise ValueError(f"{what} must be a float8_e4m3fn tensor [pages, page_size, heads, head_dim] with contiguous columns")
        if k.shape != v.shape:
            raise ValueError("k and v differ in shape")
        pages, page, heads, dim = k.shape
        n = scales.shape[1] if scales.dim() == 4 else 0
        if (n < 1 or page % n or scales.shape != (pages, n, heads, 2) or scales.dtype != torch.float8_e8m0fnu
                or not scales.is_contiguous()):
            raise ValueError("scales must be a contiguous float8_e8m0fnu tensor [pages, page_size / scale_slots, heads, 2]")
        _on(k.device, v=v, scales=scales)
        self.k, self.v, self.scales, self.device = k, v, scales, k.device
        self.args = Cache8(k.data_ptr(), v.data_ptr(), scales.data_ptr(), *k.stride()[:3], *v.stride()[:3], *k.shape, page // n)
        self._ref, self._index = _byref(self.args), k.get_device()

    def _append(self):
        return lib().sgemv_append8, "sgemv_append8"

    def _attend(self, window, sinks):
        L = lib()
        return L.sgemv_attend8_plan, L.sgemv_attend8, _slots(window, sinks), "sgemv_attend8"


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


def sample(x, uniform, temperature=None, top_k=None, top_p=None, min_p=None, out=None, logprob=None, stream=None):
    """A token for each row of logits x [rows, vocab] (FP16, BF16 or FP32): int32 [rows].

    uniform (float32 [rows]): random numbers in [0, 1), the only source of
    chance. Of a row's tokens, whose p is exp((x - max) / temperature), those of
    ``min_p`` and more are kept, of these the ``top_k`` largest, of these the
    fewest largest that sum to ``top_p`` of them; equal logits count by id. The
    token is the first by id up to which the kept p sum to more than uniform
    times their sum. temperature, top_p, min_p: float32 [rows]; top_k: int32
    [rows]; temperature 0 or less takes the largest logit, top_k 0 or less, top_p
    1 or more and min_p 0 or less leave all. out (int32 [rows]): the tokens;
    logprob (float32 [rows]): the logarithm of each one's share of what is kept.
    A row of -inf and NaN alone gets -1 and -inf."""
    if torch is None:
        _init()
    dev, card = x.device, x.get_device()
    if x.dim() != 2 or (x.stride(1) != 1 and x.shape[1] > 1):
        raise ValueError("x must be [rows, vocab] with contiguous rows")
    rows, vocab = x.shape
    one, f32, i32 = (rows,), torch.float32, torch.int32

    def at(t, what, dtype):
        if t is None:
            return 0
        if t.dtype != dtype or t.shape != one or not t.is_contiguous() or t.get_device() != card:
            raise ValueError(f"{what} must be a contiguous {dtype} tensor of shape {list(one)} on {dev}")
        return t.data_ptr()

    u = at(uniform, "uniform", f32)
    rest = at(temperature, "temperature", f32), at(top_k, "top_k", i32), at(top_p, "top_p", f32), at(min_p, "min_p", f32)
    ids, lp = at(out, "out", i32), at(logprob, "logprob", f32)
    dtype = _type(x.dtype)
    s, ctx = _enter(dev, stream)
    try:
        if out is None:
            out = torch.empty(one, dtype=i32, device=dev)
            ids = out.data_ptr()
        code = lib().sgemv_sample(_pack_sampling(x.data_ptr(), x.stride(0), u, *rest, ids, lp, rows, vocab, dtype), s)
    finally:
        _leave(ctx)
    if code:
        _check(code, "sgemv_sample")
    return out

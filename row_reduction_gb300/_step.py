"""Binding of the operators around a decoder's cache (``include/mt_decoder.h``):
the pages of a step's tokens, attention over the cached codes, and the norms
behind a block and before the next one.

Devices, streams, graphs and autograd are as in :mod:`._decoder`: tensors of
one call are on one device, the work runs there on ``stream``, nothing
synchronises, calls can be captured, and autograd records nothing
(:func:`block_norm_backward` is the gradient of :func:`block_norm`).
"""
from __future__ import annotations

import ctypes
import struct
from collections import namedtuple

from . import _decoder as _d
from ._binding import _check
from ._decoder import (_F, _I32, _I64, _P, _cache, _dense, _first, _heads,
                       _On, _opt, _rows, _tensor, _three)

MT_NORM_AFTER, MT_NORM_BEFORE = 1, 2


class MtCacheExtendCall(ctypes.Structure):
    """``mt_cache_extend_call_t``."""
    _fields_ = [("table", _P), ("table_stride", _I64), ("lengths", _P),
                ("counts", _P), ("free_pages", _P), ("free_count", _P),
                ("offsets", _P), ("slots", _P), ("positions", _P),
                ("new_lengths", _P), ("new_free_count", _P), ("rows", _I64),
                ("pages", _I32), ("sequences", _I32), ("free_size", _I32),
                ("page_size", _I32)]


class MtAttentionCall(ctypes.Structure):
    """``mt_attention_call_t``."""
    _fields_ = ([("q", _P), ("out", _P), ("lse", _P)] +
                [(n, _I64) for n in ("q_row", "q_head", "out_row",
                                     "out_head")] +
                [(n, _P) for n in ("k_codes", "v_codes", "k_scales",
                                   "v_scales", "table")] +
                [("table_stride", _I64)] +
                [(n, _P) for n in ("offsets", "starts", "first", "last",
                                   "slopes")] +
                [("rows", _I64), ("slots", _I64)] +
                [(n, _I32) for n in ("sequences", "pages", "page_size",
                                     "q_heads", "k_heads", "dim", "group",
                                     "format", "window")] +
                [("scale", _F), ("cap", _F), ("reserved", _I32)])


class MtBlockNormCall(ctypes.Structure):
    """``mt_block_norm_call_t``."""
    _fields_ = ([(n, _P) for n in ("x", "residual", "gate", "weight",
                                   "next_weight", "h", "y")] +
                [(n, _I64) for n in ("x_stride", "residual_stride",
                                     "gate_stride", "h_stride", "y_stride",
                                     "rows")] +
                [("cols", _I32), ("norms", _I32), ("eps", _F),
                 ("residual_scale", _F)])


class MtBlockNormBack(ctypes.Structure):
    """``mt_block_norm_back_t``."""
    _fields_ = ([(n, _P) for n in ("dy", "dh", "x", "h", "gate", "weight",
                                   "next_weight", "dx", "dresidual", "dgate",
                                   "dgate_sum", "dweight",
                                   "dnext_weight")] +
                [(n, _I64) for n in ("dy_stride", "dh_stride", "x_stride",
                                     "h_stride", "gate_stride", "dx_stride",
                                     "dresidual_stride", "dgate_stride",
                                     "rows")] +
                [("cols", _I32), ("norms", _I32), ("eps", _F),
                 ("residual_scale", _F)])


_lib = None


def _step_lib():
    global _lib
    if _lib is None:
        L = _d._decoder_lib()
        ptr, size = ctypes.POINTER, ctypes.c_size_t
        for name, args in {
                "mt_cache_extend": [ptr(MtCacheExtendCall), _P],
                "mt_cache_attention": [_I32, ptr(MtAttentionCall), _P, size,
                                       _P],
                "mt_cache_attention_workspace": [_I32, ptr(MtAttentionCall),
                                                 ptr(size)],
                "mt_block_norm": [_I32, ptr(MtBlockNormCall), _P],
                "mt_block_norm_backward": [_I32, ptr(MtBlockNormBack), _P,
                                           size, _P],
                "mt_block_norm_backward_workspace": [
                    _I32, ptr(MtBlockNormBack), ptr(size)]}.items():
            fn = getattr(L, name)
            fn.argtypes, fn.restype = args, ctypes.c_int
        _lib = L
    return _lib


# ---- the C ABI, one function per entry point (raw addresses) -----------------
def mt_cache_extend(call, stream):
    _check(_step_lib().mt_cache_extend(ctypes.byref(call), stream),
           "mt_cache_extend")


def mt_cache_attention(dtype, call, workspace, workspace_bytes, stream):
    _check(_step_lib().mt_cache_attention(
        dtype, ctypes.byref(call), workspace, workspace_bytes, stream),
        "mt_cache_attention")


def mt_cache_attention_workspace(dtype, call):
    n = ctypes.c_size_t()
    _check(_step_lib().mt_cache_attention_workspace(
        dtype, ctypes.byref(call), ctypes.byref(n)),
        "mt_cache_attention_workspace")
    return n.value


def mt_block_norm(dtype, call, stream):
    _check(_step_lib().mt_block_norm(dtype, ctypes.byref(call), stream),
           "mt_block_norm")


def mt_block_norm_backward(dtype, call, workspace, workspace_bytes, stream):
    _check(_step_lib().mt_block_norm_backward(
        dtype, ctypes.byref(call), workspace, workspace_bytes, stream),
        "mt_block_norm_backward")


def mt_block_norm_backward_workspace(dtype, call):
    n = ctypes.c_size_t()
    _check(_step_lib().mt_block_norm_backward_workspace(
        dtype, ctypes.byref(call), ctypes.byref(n)),
        "mt_block_norm_backward_workspace")
    return n.value


# ---- tensors -----------------------------------------------------------------
# The C structures in one go, native alignment.
_EXTEND = struct.Struct("@Pq9Pq4i")
_ATTENTION = struct.Struct("@3P4q5Pq5P2q9i2fi")
_NORM = struct.Struct("@7P6q2i2f")
_NORM_BACK = struct.Struct("@13P9q2i2f")


def _pack(form, *values):
    """A call's structure."""
    try:
        return form.pack(*values)
    except (struct.error, OverflowError) as e:
        raise ValueError(f"an argument is out of its type's range: {e}") \
            from None


def _call(name, *args):
    st = _calls[name](*args)
    if st != _d.MT_OK:
        raise _d.MTError(st, name)


class _Calls(dict):
    """The entry points on packed structures, found on first use."""

    def __missing__(self, name):
        _step_lib()
        fn = getattr(ctypes.CDLL(_d.LIB_PATH), name)  # the same library
        size, text = ctypes.c_size_t, ctypes.c_char_p
        fn.argtypes = {"mt_cache_extend": [text, _P],
                       "mt_cache_attention": [_I32, text, _P, size, _P],
                       "mt_cache_attention_workspace": [_I32, text, _P],
                       "mt_block_norm": [_I32, text, _P],
                       "mt_block_norm_backward": [_I32, text, _P, size, _P],
                       "mt_block_norm_backward_workspace": [_I32, text, _P],
                       }[name]
        fn.restype = ctypes.c_int
        self[name] = fn
        return fn


_calls = _Calls()


def _workspace(name, dt, call, like):
    """(tensor, address, bytes) of a call's workspace."""
    n = ctypes.c_size_t()
    _call(name, dt, call, ctypes.addressof(n))
    if n.value == 0:
        return None, None, 0
    t = _d._torch.empty(n.value, dtype=_d._torch.uint8, device=like.device)
    return t, t.data_ptr(), n.value


def _on(index, stream, run):
    """run(handle) on the call's device and stream."""
    if stream is None and _d._torch._C._cuda_getDevice() == index:
        return run(_d._torch._C._cuda_getCurrentRawStream(index))
    with _On(index, stream) as handle:
        return run(handle)


def _length(t, name, dtype):
    """Values of a vector (the rest is checked with its address)."""
    sh = getattr(t, "shape", None)
    if sh is None or len(sh) != 1 or not t.is_cuda:
        _tensor(t, name, dtype, (None,))
    return sh[0]


def _table(table, sequences, index):
    """(address, row stride, width) of a page table."""
    try:
        sh, st = table.shape, table.stride()
        if (table.dtype is _d._torch.int32 and len(sh) == 2 and
                (sequences is None or sh[0] == sequences) and
                table.get_device() == index >= 0 and
                (sh[1] <= 1 or st[1] == 1)):
            return table.data_ptr(), st[0] if sh[0] > 1 else sh[1], sh[1]
    except AttributeError:
        pass
    _tensor(table, "table", _d._torch.int32, (sequences, None),
            None if index < 0 else index)
    raise ValueError("table must be [sequences, pages] with dense rows")


# ---- pages of a step ---------------------------------------------------------
CacheStep = namedtuple("CacheStep", ["offsets", "slots", "positions",
                                     "lengths", "free_count"])
CacheStep.__doc__ = """What :func:`cache_extend` gives: offsets int32
[sequences + 1] of the packed batch, slots int64 [rows] and positions int32
[rows] of its rows, the sequences' new lengths int32 [sequences] and the new
free_count int32 [1]."""


def cache_extend(table, lengths, counts, free_pages, free_count, page_size,
                 rows, out=None, stream=None):
    """Makes room for the next counts[s] tokens of each sequence, which holds
    lengths[s] (int32 [sequences] both): pages that it needs beyond the ones
    it has are taken from the end of the first free_count[0] (int32 [1]) of
    free_pages (int32), in the order of the sequences, and written into its
    row of table [sequences, pages] (int32), in place.  Returns a
    :class:`CacheStep`: where the step's rows, packed sequence by sequence,
    stand, for :func:`cache_write`, :func:`rotary` and :func:`cache_attention`
    (whose starts are the old lengths); rows behind the batch, up to `rows`,
    get slot -1 (with fewer rows than the counts add up to, only so many are
    written out).  A sequence for which there are not enough pages, in the list
    or in the table's width, gets none: its length stays and its rows have
    slot -1.  The lists themselves stay: pass the new lengths and free_count
    to the next call.  out: a CacheStep to write to."""
    if _d._torch is None:
        _d._setup()
    torch = _d._torch
    i32, i64 = torch.int32, torch.int64
    n = _length(lengths, "lengths", i32)
    index = lengths.get_device()
    at, stride, pages = _table(table, n, index)
    lens = _dense(lengths, "lengths", i32, (n,), index)
    more = _dense(counts, "counts", i32, (n,), index)
    size = _length(free_pages, "free_pages", i32)
    free = _dense(free_pages, "free_pages", i32, (size,), index)
    left = _dense(free_count, "free_count", i32, (1,), index)

    def run(handle):
        if out is None:
            # one block for the int32 ones: addresses by their places in it
            flat = torch.empty(rows + 2 * n + 2, dtype=i32,
                               device=lengths.device)
            place, offsets, lengths_, count = flat.split_with_sizes(
                (rows, n + 1, n, 1))
            slots = torch.empty(rows, dtype=i64, device=flat.device)
            step = CacheStep(offsets, slots, place, lengths_, count)
            p = flat.data_ptr()
            q = p + 4 * rows
            places = (q, slots.data_ptr(), p, q + 4 * (n + 1),
                      q + 4 * (2 * n + 1))
        else:
            step = CacheStep(*out)
            places = (_dense(step.offsets, "offsets", i32, (n + 1,), index),
                      _dense(step.slots, "slots", i64, (rows,), index),
                      _dense(step.positions, "positions", i32, (rows,),
                             index),
                      _dense(step.lengths, "new lengths", i32, (n,), index),
                      _dense(step.free_count, "new free_count", i32, (1,),
                             index))
        _call("mt_cache_extend",
              _pack(_EXTEND, at, stride, lens, more, free, left, *places, rows,
                    pages, n, size, page_size), handle)
        return step
    return _on(index, stream, run)


# ---- attention over the cache ------------------------------------------------
def cache_attention(q, k_cache, v_cache, table, offsets, starts, page_size,
                    scale=None, cap=None, slopes=None, window=None,
                    first=None, last=None, out=None, return_lse=False,
                    stream=None):
    """Attention of the queries q [rows, q_heads, dim] over the keys and values
    that k_cache and v_cache hold, each (codes, scales) as from
    :func:`cache_alloc`.  q_heads is a multiple of the cache's heads; q may be
    a strided view.  Heads of 64 (one or two groups), 80, 96 (one), 128 (one, two
    or four) and 256 (one, two or eight) in a cache whose codes begin at 32 bytes
    and scales at 16 go to matrix instructions; other heads take far longer.

    Rows offsets[s] .. offsets[s+1]-1 belong to sequence s and stand at
    positions starts[s], starts[s]+1, ... of it; its page p is table[s, p]
    (all int32, as in :func:`cache_slots`).  A row sees the keys from 0 to its
    own position: with `window` the last so many of them only, with `first`
    (int32 [rows]) from first[row] on (a document's mask), with `last` (int32
    [rows]) to last[row] in place of its position (a prefix's mask; at most to
    the end of what the sequence holds with these rows).

    Scores are scale * q.k (scale None: dim ** -0.5), then with `cap`
    cap * tanh(score / cap), then with `slopes` (float32 [q_heads]) less
    slopes[head] times the distance in positions.  Returns [rows, q_heads,
    dim], zeros for a row that sees nothing, and with return_lse also the
    logarithm of the sum of the exponentials of its scores (float32 [rows,
    q_heads], then -inf).  What a row does not see has no effect on it, but that
    codes which are NaN themselves (cache_write stores none) must not stand in
    slots that a row of its sequence sees.  out: where to write, not q; rows outside the batch
    (offsets[0] .. offsets[-1]) are left as they were (in new outputs:
    zeros)."""
    dt, index = _first(q, "q")
    torch = _d._torch
    dtype, shape = q.dtype, _three(q, "q")
    rows, q_heads, dim = shape
    x, xr, xh = _heads(q, "q", dtype, shape, index)
    kc, ks, like = _cache(k_cache, "k_cache", None, index)
    vc, vs, _ = _cache(v_cache, "v_cache", like, index)
    slots, heads, width = like[1]
    if width != dim:
        raise ValueError(f"q has heads of {dim}, the cache of {width}")
    if heads == 0 or q_heads == 0 or q_heads % heads:
        raise ValueError(f"{q_heads} query heads are no multiple of the "
                         f"cache's {heads}")
    i32 = torch.int32
    n = _length(starts, "starts", i32)
    at, stride, pages = _table(table, n, index)
    offs = _dense(offsets, "offsets", i32, (n + 1,), index)
    from_ = _dense(starts, "starts", i32, (n,), index)
    lo = _opt(first, "first", i32, (rows,), index)
    hi = _opt(last, "last", i32, (rows,), index)
    sl = _opt(slopes, "slopes", torch.float32, (q_heads,), index)
    if cap is not None and not cap >= 2.0 ** -126:
        raise ValueError(f"cap must be above 0 (from 2^-126 on), got {cap}")
    if window is not None and window < 1:
        raise ValueError(f"window must be at least 1, got {window}")
    if scale is None:
        scale = dim ** -0.5

    def run(handle):
        if out is None:
            y = torch.zeros(shape, dtype=dtype, device=q.device)
            o, orow, oh = y.data_ptr(), q_heads * dim, dim
        else:
            y = out
            o, orow, oh = _heads(y, "out", dtype, shape, index)
        lse = torch.full((rows, q_heads), -torch.inf, device=q.device) \
            if return_lse else None
        call = _pack(
            _ATTENTION, x, o, 0 if lse is None else lse.data_ptr(), xr, xh,
            orow, oh, kc, vc, ks, vs, at, stride, offs, from_, lo, hi, sl, rows, slots, n,
            pages, page_size, q_heads, heads, dim, dim // like[2][2],
            _d._FORMATS[like[0]], min(window or 0, 2 ** 31 - 1), scale,
            cap or 0.0, 0)
        held, address, size = _workspace("mt_cache_attention_workspace", dt,
                                         call, q)
        _call("mt_cache_attention", dt, call, address, size, handle)
        return (y, lse) if return_lse else y
    return _on(index, stream, run)


# ---- norms around a block ------------------------------------------------------
_NORMS = {"after": MT_NORM_AFTER, "before": MT_NORM_BEFORE,
          "both": MT_NORM_AFTER | MT_NORM_BEFORE}


def _kind(norms, weight, next_weight):
    kind = _NORMS.get(norms)
    if kind is None:
        raise ValueError(f"norms must be one of {sorted(_NORMS)}, got "
                         f"{norms!r}")
    if weight is not None and not kind & MT_NORM_AFTER:
        raise ValueError("weight belongs to the norm behind the block")
    if next_weight is not None and not kind & MT_NORM_BEFORE:
        raise ValueError("next_weight belongs to the norm before the next "
                         "block")
    return kind


def _matrix(t, name, dtype, shape, index):
    """(address, row stride) of a matrix with dense rows."""
    try:
        st = t.stride()
        if (st[1] == 1 and t.dtype is dtype and t.shape == shape and
                t.get_device() == index):
            return t.data_ptr(), st[0]
    except (AttributeError, IndexError):
        pass
    at, stride, width = _rows(t, name, dtype, shape[0], index)
    if width != shape[1]:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got "
                         f"{tuple(t.shape)}")
    return at, stride


def _dense_like(t, shape, stride):
    """A new dense matrix of t's shape, type and device (empty_like, the
    quicker call, where t is dense)."""
    if stride == shape[1]:
        return _d._torch.empty_like(t)
    return _d._torch.empty(shape, dtype=t.dtype, device=t.device)


def _gate(gate, dtype, shape, index):
    """(address, row stride) of a gate: [cols] or [rows, cols]."""
    if gate is None:
        return 0, 0
    if gate.dim() == 1:
        return _dense(gate, "gate", dtype, shape[1:], index), 0
    return _matrix(gate, "gate", dtype, shape, index)


def block_norm(x, residual, weight=None, gate=None, next_weight=None,
               norms="both", residual_scale=1.0, eps=1e-6, out=None,
               h_out=None, stream=None):
    """A block's output x [rows, cols] joins the residual stream, and the
    stream goes through the norm before the next block:

        u = rmsnorm(x) * weight                 (norms "after" or "both")
        h = residual_scale * residual + gate * u
        y = rmsnorm(h) * next_weight            (norms "before" or "both")

    gate: [cols], or [rows, cols], or None (ones).  Weights may be None
    (ones).  Returns (y, h), with norms "after" h alone.  out and h_out: where
    to write y and h; either may be x or residual."""
    dt, index = _first(x, "x")
    dtype, shape = x.dtype, x.shape
    if len(shape) != 2:
        raise ValueError(f"x must be [rows, cols], got {tuple(shape)}")
    kind = _kind(norms, weight, next_weight)
    px, xs = _matrix(x, "x", dtype, shape, index)
    pr, rs = _matrix(residual, "residual", dtype, shape, index)
    pg, gs = _gate(gate, dtype, shape, index)
    pw = _opt(weight, "weight", dtype, shape[1:], index)
    pn = _opt(next_weight, "next_weight", dtype, shape[1:], index)
    before = kind & MT_NORM_BEFORE
    if out is not None and not before:
        raise ValueError("out is y's, which norms 'after' does not have: "
                         "give h_out")

    def run(handle):
        h, y = h_out, out
        py = ys = 0
        if h is None:
            h = _dense_like(x, shape, xs)
            ph, hs = h.data_ptr(), shape[1]
        else:
            ph, hs = _matrix(h, "h_out", dtype, shape, index)
        if before and y is None:
            y = _dense_like(x, shape, xs)
            py, ys = y.data_ptr(), shape[1]
        elif before:
            py, ys = _matrix(y, "out", dtype, shape, index)
        _call("mt_block_norm", dt, _pack(
            _NORM, px, pr, pg, pw, pn, ph, py, xs, rs, gs, hs, ys, shape[0],
            shape[1], kind, eps, residual_scale), handle)
        return (y, h) if before else h
    return _on(index, stream, run)


def block_norm_backward(dy, dh, x, h, weight=None, gate=None,
                        next_weight=None, norms="both", residual_scale=1.0,
                        eps=1e-6, out=None, stream=None):
    """Gradients of :func:`block_norm`: dy and dh are those of y and h (dh
    None: zeros; dy None with norms "after"), h its output (not needed, and
    None, with norms "after"), x its input (not needed with norms "before"
    and no gate), the rest as it was given.  Returns the gradients of x, the
    residual, and, where they were given, of gate (FP32 and summed over rows
    for a gate [cols]), weight and next_weight (FP32).  out: (dx, dresidual)
    to write to; each may be one of dy, dh, x and h."""
    kind = _kind(norms, weight, next_weight)
    after, before = kind & MT_NORM_AFTER, kind & MT_NORM_BEFORE
    if before:
        if dy is None or h is None:
            raise ValueError("the norm before the next block needs dy and h")
    elif dy is not None:
        raise ValueError("dy belongs to the norm before the next block")
    elif dh is None:
        raise ValueError("without the norm before the next block dh is "
                         "needed")
    else:
        h = None
    if x is None and (after or gate is not None):
        raise ValueError("x is needed")
    one = dy if before else dh
    dt, index = _first(one, "dy" if before else "dh")
    torch = _d._torch
    dtype, shape, f32 = one.dtype, one.shape, torch.float32
    if len(shape) != 2:
        raise ValueError(f"gradients must be [rows, cols], got "
                         f"{tuple(shape)}")
    pdy, dys = _matrix(dy, "dy", dtype, shape, index) if before else (0, 0)
    pdh, dhs = (0, 0) if dh is None else \
        _matrix(dh, "dh", dtype, shape, index)
    px, xs = (0, 0) if x is None else _matrix(x, "x", dtype, shape, index)
    ph, hs = (0, 0) if h is None else _matrix(h, "h", dtype, shape, index)
    pg, gs = _gate(gate, dtype, shape, index)
    pw = _opt(weight, "weight", dtype, shape[1:], index)
    pn = _opt(next_weight, "next_weight", dtype, shape[1:], index)
    stride = dys if before else dhs

    def run(handle):
        dx, dres = (None, None) if out is None else out
        cols = shape[1]
        if dx is None:
            dx = _dense_like(one, shape, stride)
            pdx, dxs = dx.data_ptr(), cols
        else:
            pdx, dxs = _matrix(dx, "out (dx)", dtype, shape, index)
        if dres is None:
            dres = _dense_like(one, shape, stride)
            pdr, drs = dres.data_ptr(), cols
        else:
            pdr, drs = _matrix(dres, "out (dresidual)", dtype, shape, index)
        got, sums, pdg, dgs = [dx, dres], [0, 0, 0], 0, 0
        wide = gate is not None and gate.dim() == 2
        if wide:
            dgate = _dense_like(one, shape, stride)
            pdg, dgs = dgate.data_ptr(), cols
            got.append(dgate)
        for i, t in enumerate((None if wide else gate, weight, next_weight)):
            if t is not None:
                d = torch.empty(cols, dtype=f32, device=one.device)
                sums[i] = d.data_ptr()
                got.append(d)
        call = _pack(
            _NORM_BACK, pdy, pdh, px, ph, pg, pw, pn, pdx, pdr, pdg, *sums, dys, dhs, xs,
            hs, gs, dxs, drs, dgs, shape[0], shape[1], kind, eps,
            residual_scale)
        held, address, size = _workspace("mt_block_norm_backward_workspace",
                                         dt, call, one)
        _call("mt_block_norm_backward", dt, call, address, size, handle)
        return tuple(got)
    return _on(index, stream, run)

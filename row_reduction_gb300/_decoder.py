"""Binding of the decoder's row operators (``include/mt_decoder.h``): rotary
positions, the quantised cache and the logits.

The ``mt_*`` functions call the C functions of the same name; the functions
under them check tensors, allocate outputs and fill the calls.  Tensors of one
call are on one device and the work runs there, on ``stream`` (a
``torch.cuda.Stream``, a raw handle, or ``None`` for that device's current
stream); what a call allocates belongs to the stream it runs on.  Nothing
synchronises, and every call can be captured into a CUDA graph.
"""
from __future__ import annotations

import ctypes
from collections import namedtuple

from ._binding import DTYPE_IDS, _check, lib as _base_lib

MT_ROTARY_PLAIN, MT_ROTARY_LINEAR, MT_ROTARY_NTK = 0, 1, 2
MT_ROTARY_YARN, MT_ROTARY_BANDS = 3, 4
MT_CACHE_E4M3, MT_CACHE_INT8 = 0, 1
MT_LOGITS, MT_LOGITS_SOFTMAX, MT_LOGITS_LOG_SOFTMAX = 0, 1, 2

# Symbols declared in include/mt_decoder.h.
DECODER_EXPORTS = (
    "mt_rotary_frequencies", "mt_rotary_turns", "mt_rotary",
    "mt_rotary_backward", "mt_rotary_backward_workspace", "mt_cache_write",
    "mt_cache_read", "mt_cache_slots", "mt_process_logits",
)

_P, _I64, _I32, _F, _D = (ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32,
                          ctypes.c_float, ctypes.c_double)


class MtRotaryScaling(ctypes.Structure):
    """``mt_rotary_scaling_t``."""
    _fields_ = [("type", _I32), ("reserved", _I32), ("factor", _D),
                ("original_length", _D), ("low", _D), ("high", _D)]


class MtRotaryHeads(ctypes.Structure):
    """``mt_rotary_heads_t``."""
    _fields_ = ([(n, _P) for n in ("x", "dy", "y", "weight", "dweight")] +
                [(n, _I64) for n in ("x_token", "x_head", "dy_token",
                                     "dy_head", "y_token", "y_head")] +
                [("heads", _I32), ("reserved", _I32)])


class MtRotaryCall(ctypes.Structure):
    """``mt_rotary_call_t``."""
    _fields_ = [("q", MtRotaryHeads), ("k", MtRotaryHeads),
                ("positions", _P), ("turns", _P), ("tokens", _I64),
                ("position_bytes", _I32), ("dim", _I32),
                ("rotary_dim", _I32), ("interleaved", _I32), ("norm", _I32),
                ("eps", _F), ("scale", _F), ("reserved", _I32)]


class MtCacheRows(ctypes.Structure):
    """``mt_cache_rows_t``."""
    _fields_ = [("codes", _P), ("scales", _P), ("rows", _P),
                ("token_stride", _I64), ("head_stride", _I64)]


class MtCacheCall(ctypes.Structure):
    """``mt_cache_call_t``."""
    _fields_ = [("k", MtCacheRows), ("v", MtCacheRows), ("slot", _P),
                ("tokens", _I64), ("slots", _I64), ("heads", _I32),
                ("dim", _I32), ("group", _I32), ("format", _I32)]


class MtLogitsCall(ctypes.Structure):
    """``mt_logits_call_t``."""
    _fields_ = [("x", _P), ("y", _P), ("rows", _I64), ("x_stride", _I64),
                ("y_stride", _I64), ("vocab", _I32), ("mode", _I32),
                ("tokens", _P), ("tokens_stride", _I64), ("history", _I32),
                ("biases", _I32), ("lengths", _P), ("prompt_lengths", _P),
                ("repetition", _P), ("frequency", _P), ("presence", _P),
                ("bias_ids", _P), ("bias", _P), ("mask", _P),
                ("mask_stride", _I64), ("temperature", _P)]


_lib = None


def _decoder_lib():
    global _lib
    if _lib is None:
        L = _base_lib()
        ptr, st = ctypes.POINTER, ctypes.c_int
        for name, args in {
                "mt_rotary_frequencies": [_I32, _D, ptr(MtRotaryScaling),
                                          ptr(_D), ptr(_D)],
                "mt_rotary_turns": [ptr(_D), _I32, ptr(ctypes.c_uint64)],
                "mt_rotary": [st, ptr(MtRotaryCall), _P],
                "mt_rotary_backward": [st, ptr(MtRotaryCall), _P,
                                       ctypes.c_size_t, _P],
                "mt_rotary_backward_workspace": [ptr(MtRotaryCall),
                                                 ptr(ctypes.c_size_t)],
                "mt_cache_write": [st, ptr(MtCacheCall), _P],
                "mt_cache_read": [st, ptr(MtCacheCall), _P],
                "mt_cache_slots": [_P, _I64, _I32, _P, _P, _I32, _I32, _I64,
                                   _P, _P],
                "mt_process_logits": [st, ptr(MtLogitsCall), _P]}.items():
            fn = getattr(L, name)
            fn.argtypes, fn.restype = args, st
        _lib = L
    return _lib


# ---- the C ABI, one function per entry point (raw addresses) -----------------
def mt_rotary_frequencies(rotary_dim, base, scaling=None):
    """(frequencies in radians per position, factor on rotated values)."""
    n = max(0, rotary_dim // 2)
    freqs, factor = (_D * max(1, n))(), _D()
    _check(_decoder_lib().mt_rotary_frequencies(
        rotary_dim, base, ctypes.byref(scaling) if scaling else None, freqs,
        ctypes.byref(factor)), "mt_rotary_frequencies")
    return list(freqs)[:n], factor.value


def mt_rotary_turns(freqs):
    """Frequencies as fractions of a turn, in units of 2^-64 turns."""
    n = len(freqs)
    turns = (ctypes.c_uint64 * max(1, n))()
    _check(_decoder_lib().mt_rotary_turns((_D * max(1, n))(*freqs), n, turns),
           "mt_rotary_turns")
    return list(turns)[:n]


def mt_rotary(dtype, call, stream):
    _check(_decoder_lib().mt_rotary(dtype, ctypes.byref(call), stream),
           "mt_rotary")


def mt_rotary_backward(dtype, call, workspace, workspace_bytes, stream):
    _check(_decoder_lib().mt_rotary_backward(
        dtype, ctypes.byref(call), workspace, workspace_bytes, stream),
        "mt_rotary_backward")


def mt_rotary_backward_workspace(call):
    n = ctypes.c_size_t()
    _check(_decoder_lib().mt_rotary_backward_workspace(
        ctypes.byref(call), ctypes.byref(n)), "mt_rotary_backward_workspace")
    return n.value


def mt_cache_write(dtype, call, stream):
    _check(_decoder_lib().mt_cache_write(dtype, ctypes.byref(call), stream),
           "mt_cache_write")


def mt_cache_read(dtype, call, stream):
    _check(_decoder_lib().mt_cache_read(dtype, ctypes.byref(call), stream),
           "mt_cache_read")


def mt_cache_slots(table, table_stride, pages_per_sequence, offsets, starts,
                   sequences, page_size, rows, slot, stream):
    _check(_decoder_lib().mt_cache_slots(
        table, table_stride, pages_per_sequence, offsets, starts, sequences,
        page_size, rows, slot, stream), "mt_cache_slots")


def mt_process_logits(dtype, call, stream):
    _check(_decoder_lib().mt_process_logits(dtype, ctypes.byref(call),
                                            stream), "mt_process_logits")


# ---- tensors -----------------------------------------------------------------
_DTYPES = None


def _dtype_id(t, name):
    global _DTYPES
    if _DTYPES is None:
        import torch
        _DTYPES = {torch.float32: DTYPE_IDS["f32"],
                   torch.float16: DTYPE_IDS["f16"],
                   torch.bfloat16: DTYPE_IDS["bf16"]}
    got = _DTYPES.get(t.dtype)
    if got is None:
        raise TypeError(f"{name} must be float32, float16 or bfloat16, got "
                        f"{t.dtype}")
    return got


def _tensor(t, name, dtype=None, shape=None, like=None):
    """Checks one tensor: CUDA, its type, its shape (None entries are free)
    and the device of `like`."""
    import torch
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name}: expected a CUDA tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if like is not None and t.device != like.device:
        raise ValueError(f"{name} is on {t.device}, not on {like.device}")
    if shape is not None:
        if t.dim() != len(shape) or any(
                w is not None and g != w for g, w in zip(t.shape, shape)):
            raise ValueError(f"{name} must have shape "
                             f"{tuple(shape)}, got {tuple(t.shape)}")
    return t


def _dense(t, name, dtype, shape, like):
    _tensor(t, name, dtype, shape, like)
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


def _heads_view(t, name, dtype=None, shape=None, like=None):
    """A [tokens, heads, dim] tensor whose last dimension is dense."""
    _tensor(t, name, dtype, shape, like)
    if t.dim() != 3:
        raise ValueError(f"{name} must be [tokens, heads, dim]")
    if t.shape[2] > 1 and t.stride(2) != 1:
        raise ValueError(f"{name}: the last dimension must be dense")
    return t


class _On:
    """Runs a call on a tensor's device and on `stream`: allocations inside
    belong to that stream, `handle` is its raw handle."""

    def __init__(self, device, stream):
        import torch
        if stream is None:
            self.stream = None
            self.handle = torch.cuda.current_stream(device).cuda_stream
        elif isinstance(stream, int):
            self.stream = torch.cuda.ExternalStream(stream, device=device)
            self.handle = stream
        else:
            if stream.device != device:
                raise ValueError(f"stream is on {stream.device}, the tensors "
                                 f"are on {device}")
            self.stream, self.handle = stream, stream.cuda_stream
        if self.stream is not None:
            self.context = torch.cuda.stream(self.stream)
        elif torch.cuda.current_device() != device.index:
            self.context = torch.cuda.device(device)
        else:
            self.context = None

    def __enter__(self):
        if self.context is not None:
            self.context.__enter__()
        return self.handle

    def __exit__(self, *exc):
        if self.context is not None:
            self.context.__exit__(*exc)
        return False


# ---- rotary positions -------------------------------------------------------
class RotaryFrequencies(namedtuple("RotaryFrequencies",
                                   ["turns", "scale", "rotary_dim"])):
    """Frequencies of `rotary_dim`/2 pairs: `turns` (int64 CUDA tensor, in
    units of 2^-64 turns per position) and the factor `scale` on rotated
    values.  Made once (:func:`rotary_frequencies`) and used by every call."""
    __slots__ = ()


_SCALINGS = {"linear": MT_ROTARY_LINEAR, "ntk": MT_ROTARY_NTK,
             "yarn": MT_ROTARY_YARN, "bands": MT_ROTARY_BANDS}


def rotary_frequencies(rotary_dim, base=10000.0, scaling=None, freqs=None,
                       scale=None, device="cuda"):
    """The frequencies of :func:`rotary`.

    scaling: None, or a dict with "type" and the ratio "factor" of the long
    context to the one trained on: "linear"; "ntk"; "yarn" and "bands" with
    "original_length" and the bounds "low" and "high" in turns (yarn 1 and
    32, bands 1 and 4 where not given).  freqs: frequencies of your own
    (rotary_dim/2 radians per position) in place of base and scaling.
    scale: factor on rotated values in place of the scaling's own."""
    import torch
    if freqs is not None:
        if scaling is not None:
            raise ValueError("give freqs or scaling, not both")
        freqs, factor = [float(f) for f in freqs], 1.0
        if rotary_dim < 2 or len(freqs) * 2 != rotary_dim:
            raise ValueError(f"rotary_dim {rotary_dim} needs "
                             f"{rotary_dim // 2} frequencies, got "
                             f"{len(freqs)}")
    else:
        s = None
        if scaling is not None:
            known = {"type", "factor", "original_length", "low", "high"}
            if set(scaling) - known:
                raise ValueError(f"unknown scaling keys "
                                 f"{sorted(set(scaling) - known)}")
            kind = scaling.get("type")
            if kind not in _SCALINGS:
                raise ValueError(f"scaling type must be one of "
                                 f"{sorted(_SCALINGS)}, got {kind!r}")
            s = MtRotaryScaling(
                type=_SCALINGS[kind], factor=scaling["factor"],
                original_length=scaling.get("original_length", 0.0),
                low=scaling.get("low", 1.0),
                high=scaling.get("high", 32.0 if kind == "yarn" else 4.0))
        freqs, factor = mt_rotary_frequencies(rotary_dim, base, s)
    turns = [t - 2 ** 64 if t >= 2 ** 63 else t
             for t in mt_rotary_turns(freqs)]
    return RotaryFrequencies(
        torch.tensor(turns, dtype=torch.int64, device=device),
        factor if scale is None else float(scale), rotary_dim)


def _rotary_call(q, k, positions, freqs, interleaved, eps):
    """The parts that forward and backward share; q and k are the tensors
    whose heads are turned."""
    import torch
    dt = _dtype_id(_heads_view(q, "q"), "q")
    tokens, _, dim = q.shape
    if k is not None:
        _heads_view(k, "k", q.dtype, (tokens, None, dim), q)
    if positions.dtype not in (torch.int32, torch.int64):
        raise TypeError(f"positions must be int32 or int64, got "
                        f"{positions.dtype}")
    c = MtRotaryCall()
    c.positions = _dense(positions, "positions", positions.dtype, (tokens,),
                         q)
    c.turns = _dense(freqs.turns, "freqs", torch.int64,
                     (freqs.rotary_dim // 2,), q)
    c.tokens, c.dim, c.rotary_dim = tokens, dim, freqs.rotary_dim
    c.position_bytes = 8 if positions.dtype == torch.int64 else 4
    c.interleaved, c.scale = bool(interleaved), freqs.scale
    c.norm, c.eps = eps is not None, 0.0 if eps is None else eps
    return dt, c


def _out_pair(out, q, k):
    if out is None:
        return None, None
    if k is None and not isinstance(out, (tuple, list)):
        return out, None
    yq, yk = out
    return yq, yk


def _weight(w, name, q, eps):
    if w is None:
        return None
    if eps is None:
        raise ValueError(f"{name} belongs to the norm: give eps")
    return _dense(w, name, q.dtype, (q.shape[2],), q)


def rotary(q, k, positions, freqs, interleaved=False, q_weight=None,
           k_weight=None, eps=None, out=None, stream=None):
    """Rotary positions of the heads of q [tokens, q_heads, dim] and k
    [tokens, k_heads, dim] (None: q alone), each token at its entry of
    positions (int32 or int64).  q and k may be strided views (the last
    dimension dense).  With eps, each head is first RMS-normalised and
    multiplied by q_weight or k_weight (None: ones).  out: (q, k) to write to;
    the inputs themselves turn them in place.  Returns (q, k), or q alone
    where k is None."""
    import torch
    dt, c = _rotary_call(q, k, positions, freqs, interleaved, eps)
    if k is None and k_weight is not None:
        raise ValueError("k_weight without k")
    yq, yk = _out_pair(out, q, k)
    with _On(q.device, stream) as handle:
        for t, y, w, h, name in ((q, yq, q_weight, c.q, "q"),
                                 (k, yk, k_weight, c.k, "k")):
            if t is None:
                continue
            if y is None:
                y = torch.empty(t.shape, dtype=t.dtype, device=t.device)
                if name == "q":
                    yq = y
                else:
                    yk = y
            else:
                _heads_view(y, f"out ({name})", t.dtype, t.shape, q)
            h.x, h.y = t.data_ptr(), y.data_ptr()
            h.weight = _weight(w, f"{name}_weight", q, eps)
            h.x_token, h.x_head = t.stride(0), t.stride(1)
            h.y_token, h.y_head = y.stride(0), y.stride(1)
            h.heads = t.shape[1]
        mt_rotary(dt, c, handle)
    return yq if k is None else (yq, yk)


def rotary_backward(dq, dk, positions, freqs, interleaved=False, q=None,
                    k=None, q_weight=None, k_weight=None, eps=None, out=None,
                    stream=None):
    """Gradients of :func:`rotary`: dq and dk are those of its outputs, q and
    k its inputs (needed with the norm only), the rest as it was given.
    Returns (dq, dk) of the inputs, with eps (dq, dk, dq_weight, dk_weight),
    the weights' in FP32 (None where there is no weight).  out: (dq, dk) to
    write to; they may be dq and dk themselves."""
    import torch
    dt, c = _rotary_call(dq, dk, positions, freqs, interleaved, eps)
    norm = eps is not None
    if not norm and (q is not None or k is not None):
        raise ValueError("q and k belong to the norm: give eps")
    if dk is None and (k is not None or k_weight is not None):
        raise ValueError("k without dk")
    gq, gk = _out_pair(out, dq, dk)
    dws = [None, None]
    with _On(dq.device, stream) as handle:
        for i, (g, x, y, w, h, name) in enumerate(
                ((dq, q, gq, q_weight, c.q, "q"),
                 (dk, k, gk, k_weight, c.k, "k"))):
            if g is None:
                continue
            if y is None:
                y = torch.empty(g.shape, dtype=g.dtype, device=g.device)
                if i == 0:
                    gq = y
                else:
                    gk = y
            else:
                _heads_view(y, f"out ({name})", g.dtype, g.shape, dq)
            if norm:
                if x is None:
                    raise ValueError(f"the norm's backward pass needs {name}")
                _heads_view(x, name, g.dtype, g.shape, dq)
                h.x, h.x_token, h.x_head = (x.data_ptr(), x.stride(0),
                                            x.stride(1))
            h.weight = _weight(w, f"{name}_weight", dq, eps)
            if w is not None:
                dws[i] = torch.empty(g.shape[2], dtype=torch.float32,
                                     device=g.device)
                h.dweight = dws[i].data_ptr()
            h.dy, h.y = g.data_ptr(), y.data_ptr()
            h.dy_token, h.dy_head = g.stride(0), g.stride(1)
            h.y_token, h.y_head = y.stride(0), y.stride(1)
            h.heads = g.shape[1]
        n = mt_rotary_backward_workspace(c)
        ws = torch.empty(n, dtype=torch.uint8, device=dq.device) if n else None
        mt_rotary_backward(dt, c, ws.data_ptr() if n else None, n, handle)
    if norm:
        return gq, gk, dws[0], dws[1]
    return gq, gk


# ---- quantised cache --------------------------------------------------------
def cache_alloc(slots, heads, dim, group=None, format="e4m3", device="cuda"):
    """One cache tensor, zeroed: (codes [slots, heads, dim] of
    torch.float8_e4m3fn or torch.int8, scales [slots, heads, dim/group] of
    torch.float32).  group: values that share a scale (None: a whole head)."""
    import torch
    group = dim if group is None else group
    if format not in ("e4m3", "int8"):
        raise ValueError(f"format must be 'e4m3' or 'int8', got {format!r}")
    if group < 1 or dim % group:
        raise ValueError(f"group {group} must divide dim {dim}")
    codes = torch.zeros(slots, heads, dim, dtype=torch.int8, device=device)
    if format == "e4m3":
        codes = codes.view(torch.float8_e4m3fn)
    return codes, torch.zeros(slots, heads, dim // group,
                              dtype=torch.float32, device=device)


def _cache_call(k_cache, v_cache, slots, dt_like):
    import torch
    codes, scales = k_cache
    _tensor(codes, "k_cache codes", like=dt_like)
    formats = {torch.float8_e4m3fn: MT_CACHE_E4M3, torch.int8: MT_CACHE_INT8}
    if codes.dtype not in formats:
        raise TypeError(f"cache codes must be float8_e4m3fn or int8, got "
                        f"{codes.dtype}")
    if codes.dim() != 3 or scales.dim() != 3:
        raise ValueError("a cache is (codes [slots, heads, dim], scales "
                         "[slots, heads, dim/group])")
    n, heads, dim = codes.shape
    groups = scales.shape[2]
    if groups < 1 or dim % groups:
        raise ValueError(f"{groups} scales per head do not divide dim {dim}")
    c = MtCacheCall()
    c.format = formats[codes.dtype]
    c.slots, c.heads, c.dim, c.group = n, heads, dim, dim // groups
    c.tokens = slots.shape[0] if slots.dim() == 1 else 0
    c.slot = _dense(slots, "slots", torch.int64, (c.tokens,), codes)
    for name, cache, rows in (("k_cache", k_cache, c.k),
                              ("v_cache", v_cache, c.v)):
        if cache is None:
            continue
        rows.codes = _dense(cache[0], f"{name} codes", codes.dtype,
                            (n, heads, dim), codes)
        rows.scales = _dense(cache[1], f"{name} scales", torch.float32,
                             (n, heads, groups), codes)
    return c


def cache_write(k, v, k_cache, v_cache, slots, stream=None):
    """Stores the rows k and v [tokens, heads, dim] (strided views are fine;
    v and v_cache may be None) as 8-bit codes and scales in the slots
    slots[token] (int64) of k_cache and v_cache, each (codes, scales) as from
    :func:`cache_alloc`.  A token whose slot is outside the cache (-1: padding)
    stores nothing; the slots inside must differ from one another."""
    dt = _dtype_id(_heads_view(k, "k"), "k")
    if (v is None) != (v_cache is None):
        raise ValueError("v and v_cache come together")
    c = _cache_call(k_cache, v_cache, slots, k)
    shape = (c.tokens, c.heads, c.dim)
    for name, t, rows in (("k", k, c.k), ("v", v, c.v)):
        if t is None:
            continue
        _heads_view(t, name, k.dtype, shape, k)
        rows.rows = t.data_ptr()
        rows.token_stride, rows.head_stride = t.stride(0), t.stride(1)
    with _On(k.device, stream) as handle:
        mt_cache_write(dt, c, handle)


def cache_read(k_cache, v_cache, slots, dtype=None, out=None, stream=None):
    """The rows of the slots slots[token] (int64), as (k, v) of `dtype` (None:
    torch.bfloat16), or k alone where v_cache is None.  out: (k, v) to write
    to, strided views included; the row of a token whose slot is outside the
    cache is left as it was (in a new output: zero)."""
    import torch
    c = _cache_call(k_cache, v_cache, slots, k_cache[0])
    k, v = _out_pair(out, k_cache, v_cache)
    dtype = dtype or (torch.bfloat16 if k is None else k.dtype)
    shape, device = (c.tokens, c.heads, c.dim), k_cache[0].device
    with _On(device, stream) as handle:
        if k is None:
            k = torch.zeros(shape, dtype=dtype, device=device)
        if v_cache is not None and v is None:
            v = torch.zeros(shape, dtype=dtype, device=device)
        dt = _dtype_id(k, "out")
        for name, t, rows in (("out (k)", k, c.k), ("out (v)", v, c.v)):
            if t is None:
                continue
            _heads_view(t, name, dtype, shape, k_cache[0])
            rows.rows = t.data_ptr()
            rows.token_stride, rows.head_stride = t.stride(0), t.stride(1)
        mt_cache_read(dt, c, handle)
    return k if v_cache is None else (k, v)


def cache_slots(table, offsets, starts, page_size, rows, out=None,
                stream=None):
    """Slots (int64 [rows]) of a packed batch: rows offsets[s] ..
    offsets[s+1]-1 stand at positions starts[s], starts[s]+1, ... of sequence
    s, whose page p/page_size is table[s, p/page_size].  Rows outside the
    batch, and positions without a page (a negative entry, past the table),
    get -1.  table [sequences, pages], offsets [sequences+1] and starts
    [sequences] are int32."""
    import torch
    _tensor(table, "table", torch.int32)
    if table.dim() != 2 or (table.shape[1] > 1 and table.stride(1) != 1):
        raise ValueError("table must be [sequences, pages] with dense rows")
    n, pages = table.shape
    with _On(table.device, stream) as handle:
        if out is None:
            out = torch.empty(rows, dtype=torch.int64, device=table.device)
        mt_cache_slots(
            table.data_ptr(), table.stride(0), pages,
            _dense(offsets, "offsets", torch.int32, (n + 1,), table),
            _dense(starts, "starts", torch.int32, (n,), table), n, page_size,
            rows, _dense(out, "out", torch.int64, (rows,), table), handle)
    return out


# ---- logits -----------------------------------------------------------------
_MODES = {"logits": MT_LOGITS, "softmax": MT_LOGITS_SOFTMAX,
          "log_softmax": MT_LOGITS_LOG_SOFTMAX}


def process_logits(logits, tokens=None, lengths=None, prompt_lengths=None,
                   repetition=None, frequency=None, presence=None,
                   bias_ids=None, bias=None, mask=None, temperature=None,
                   mode="logits", out=None, stream=None):
    """Penalties, biases, temperature and mask on logits [rows, vocab] (rows
    may be strided), then softmax or log-softmax of the row, in one pass.

    tokens [rows, history] int32: ids of each row's history, of which the
    first lengths[row] count (int32; None: all) and the first
    prompt_lengths[row] are the prompt (int32; None: none); ids outside the
    vocabulary are passed over.  repetition (ids of the whole history),
    frequency and presence (ids after the prompt): float32 [rows].  bias_ids
    [rows, n] int32 and bias [rows, n] float32, n <= 1024: values added to
    single logits.  temperature: float32 [rows].  mask int32 [rows, words] or
    [words], words >= (vocab+31)//32: bit v%32 of word v//32 allows token v.
    The order is: repetition, frequency and presence, bias, temperature, mask.
    mode: "logits", "softmax" or "log_softmax"; a row of which the mask leaves
    nothing has probabilities 0 and log-probabilities -inf.  out may be
    logits."""
    import torch
    _tensor(logits, "logits", shape=(None, None))
    dt = _dtype_id(logits, "logits")
    rows, vocab = logits.shape
    if vocab > 1 and logits.stride(1) != 1:
        raise ValueError("logits: rows must be dense")
    if mode not in _MODES:
        raise ValueError(f"mode must be one of {sorted(_MODES)}, got {mode!r}")
    f32, i32 = torch.float32, torch.int32
    c = MtLogitsCall()
    c.rows, c.vocab, c.mode = rows, vocab, _MODES[mode]
    c.x, c.x_stride = logits.data_ptr(), logits.stride(0)
    if tokens is not None:
        _tensor(tokens, "tokens", i32, (rows, None), logits)
        if tokens.shape[1] > 1 and tokens.stride(1) != 1:
            raise ValueError("tokens: rows must be dense")
        if tokens.shape[1] > 0:
            c.tokens, c.history = tokens.data_ptr(), tokens.shape[1]
            c.tokens_stride = tokens.stride(0)
            if lengths is not None:
                c.lengths = _dense(lengths, "lengths", i32, (rows,), logits)
            if prompt_lengths is not None:
                c.prompt_lengths = _dense(prompt_lengths, "prompt_lengths",
                                          i32, (rows,), logits)
            if repetition is not None:
                c.repetition = _dense(repetition, "repetition", f32, (rows,),
                                      logits)
            if frequency is not None:
                c.frequency = _dense(frequency, "frequency", f32, (rows,),
                                     logits)
            if presence is not None:
                c.presence = _dense(presence, "presence", f32, (rows,),
                                    logits)
    elif not (lengths is prompt_lengths is repetition is frequency is
              presence is None):
        raise ValueError("lengths and penalties need tokens")
    if (bias is None) != (bias_ids is None):
        raise ValueError("bias and bias_ids come together")
    if bias is not None:
        c.bias_ids = _dense(bias_ids, "bias_ids", i32, (rows, None), logits)
        c.biases = bias_ids.shape[1]
        c.bias = _dense(bias, "bias", f32, (rows, c.biases), logits)
    if mask is not None:
        _tensor(mask, "mask", i32, None, logits)
        if mask.dim() not in (1, 2) or (mask.dim() == 2 and
                                        mask.shape[0] != rows):
            raise ValueError(f"mask must be [{rows}, words] or [words], got "
                             f"{tuple(mask.shape)}")
        if mask.shape[-1] < (vocab + 31) // 32:
            raise ValueError(f"mask needs {(vocab + 31) // 32} words per row, "
                             f"got {mask.shape[-1]}")
        if mask.shape[-1] > 1 and mask.stride(-1) != 1:
            raise ValueError("mask: rows must be dense")
        c.mask = mask.data_ptr()
        c.mask_stride = mask.stride(0) if mask.dim() == 2 and rows > 1 else 0
    if temperature is not None:
        c.temperature = _dense(temperature, "temperature", f32, (rows,),
                               logits)
    with _On(logits.device, stream) as handle:
        if out is None:
            out = torch.empty(logits.shape, dtype=logits.dtype,
                              device=logits.device)
        else:
            _tensor(out, "out", logits.dtype, logits.shape, logits)
            if vocab > 1 and out.stride(1) != 1:
                raise ValueError("out: rows must be dense")
        c.y, c.y_stride = out.data_ptr(), out.stride(0)
        mt_process_logits(dt, c, handle)
    return out

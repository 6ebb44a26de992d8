"""Binding of the decoder's row operators (``include/mt_decoder.h``): rotary
positions, the quantised cache and the logits.

The ``mt_*`` functions call the C functions of the same name; the functions
under them check tensors, allocate outputs and fill the calls.  Tensors of one
call are on one device and the work runs there, on ``stream`` (a
``torch.cuda.Stream``, a raw handle, or ``None`` for that device's current
stream); what a call allocates belongs to the stream it runs on.  These calls
do not synchronise and can be captured into a CUDA graph; what is made once
ahead of them is not part of that (:func:`rotary_frequencies` copies its table
from the host, :func:`cache_alloc` fills its tensors with zeros).

As in the rest of the package, autograd records nothing of a call: what comes
back requires no gradient, whatever the inputs did.  :func:`rotary_backward`
is the gradient of :func:`rotary`.
"""
from __future__ import annotations

import ctypes
import struct
from collections import namedtuple

from ._binding import (DTYPE_IDS, LIB_PATH, MT_OK, MTError,
                       lib as _base_lib, _check)

MT_ROTARY_PLAIN, MT_ROTARY_LINEAR, MT_ROTARY_NTK = 0, 1, 2
MT_ROTARY_YARN, MT_ROTARY_BANDS = 3, 4
MT_CACHE_E4M3, MT_CACHE_INT8 = 0, 1
MT_LOGITS, MT_LOGITS_SOFTMAX, MT_LOGITS_LOG_SOFTMAX = 0, 1, 2

# Symbols declared in include/mt_decoder.h.
DECODER_EXPORTS = (
    "mt_rotary_frequencies", "mt_rotary_turns", "mt_rotary",
    "mt_rotary_backward", "mt_rotary_backward_workspace", "mt_cache_write",
    "mt_cache_read", "mt_cache_slots", "mt_process_logits",
    "mt_cache_extend", "mt_cache_attention", "mt_cache_attention_workspace",
    "mt_block_norm", "mt_block_norm_backward",
    "mt_block_norm_backward_workspace",
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
# A call's time on the host is most of a small call's, so the functions below
# look at a tensor once (type, device, shape, strides, address), and pack the
# C structure in one step; only where something is wrong do they go through
# the checks one by one for what to say.
_torch = None
_DTYPES = {}
_calls = {}
# The C structures in one go (mt_rotary_call_t, mt_cache_call_t,
# mt_logits_call_t), native alignment.
_ROTARY = struct.Struct("@" + 2 * "5P6q2i" + "2Pq5i2fi")
_CACHE = struct.Struct("@" + 2 * "3P2q" + "Pqq4i")
_LOGITS = struct.Struct("@2P3q2iPq2i8PqP")


def _setup():
    """Torch and the library, once."""
    global _torch
    import torch
    _decoder_lib()
    _DTYPES.update({torch.float32: DTYPE_IDS["f32"],
                    torch.float16: DTYPE_IDS["f16"],
                    torch.bfloat16: DTYPE_IDS["bf16"]})
    L = ctypes.CDLL(LIB_PATH)  # the same library; packed structures as bytes
    text = ctypes.c_char_p
    for name, args in {
            "mt_rotary": [_I32, text, _P],
            "mt_rotary_backward": [_I32, text, _P, ctypes.c_size_t, _P],
            "mt_cache_write": [_I32, text, _P],
            "mt_cache_read": [_I32, text, _P],
            "mt_process_logits": [_I32, text, _P]}.items():
        fn = getattr(L, name)
        fn.argtypes, fn.restype = args, ctypes.c_int
        _calls[name] = fn
    _torch = torch


def _call(name, *args):
    st = _calls[name](*args)
    if st != MT_OK:
        raise MTError(st, name)


def _first(t, name):
    """(mt_dtype, device index) of a call's first tensor."""
    if _torch is None:
        _setup()
    try:
        dt, index = _DTYPES.get(t.dtype), t.get_device()
    except AttributeError:
        dt, index = None, -1
    if dt is None or index < 0:
        _tensor(t, name)
        raise TypeError(f"{name} must be float32, float16 or bfloat16, got "
                        f"{t.dtype}")
    return dt, index


def _tensor(t, name, dtype=None, shape=None, index=None):
    """Checks one tensor: CUDA, its type, its device, its shape (None entries
    are free)."""
    if not isinstance(t, _torch.Tensor):
        raise TypeError(f"{name}: expected a CUDA tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if index is not None and t.get_device() != index:
        raise ValueError(f"{name} is on {t.device}, not on cuda:{index}")
    if shape is not None:
        if t.dim() != len(shape) or any(
                w is not None and g != w for g, w in zip(t.shape, shape)):
            raise ValueError(f"{name} must have shape "
                             f"{tuple(shape)}, got {tuple(t.shape)}")
    return t


def _dense(t, name, dtype, shape, index):
    """Address of a contiguous tensor of this type, shape and device."""
    try:
        if (t.dtype is dtype and t.get_device() == index and
                t.shape == shape and t.is_contiguous()):
            return t.data_ptr()
    except AttributeError:
        pass
    _tensor(t, name, dtype, shape, index)
    raise ValueError(f"{name} must be contiguous")


def _opt(t, name, dtype, shape, index):
    return 0 if t is None else _dense(t, name, dtype, shape, index)


def _heads(t, name, dtype, shape, index):
    """(address, token stride, head stride) of a [tokens, heads, dim] tensor
    whose last dimension is dense."""
    try:
        st = t.stride()
        if (t.dtype is dtype and t.get_device() == index and
                t.shape == shape and (st[2] == 1 or shape[2] <= 1)):
            return t.data_ptr(), st[0], st[1]
    except (AttributeError, IndexError):
        pass
    _tensor(t, name, dtype, None, index)
    if t.dim() != 3:
        raise ValueError(f"{name} must be [tokens, heads, dim]")
    _tensor(t, name, dtype, shape, index)
    raise ValueError(f"{name}: the last dimension must be dense")


def _rows(t, name, dtype, rows, index):
    """(address, row stride, width) of a [rows, width] tensor with dense
    rows."""
    try:
        st, sh = t.stride(), t.shape
        if (t.dtype is dtype and t.get_device() == index and len(sh) == 2 and
                sh[0] == rows and (st[1] == 1 or sh[1] <= 1)):
            return t.data_ptr(), st[0], sh[1]
    except (AttributeError, IndexError):
        pass
    _tensor(t, name, dtype, (rows, None), index)
    raise ValueError(f"{name}: rows must be dense")


class _On:
    """A call's device and stream as a context: allocations inside belong to
    that stream, `handle` is its raw handle."""

    def __init__(self, index, stream):
        if stream is None:
            self.context = _torch.cuda.device(index)
            self.handle = _torch.cuda.current_stream(index).cuda_stream
            return
        if stream == 0:
            stream = _torch.cuda.default_stream(index)
        elif isinstance(stream, int):
            stream = _torch.cuda.ExternalStream(stream, device=index)
        if stream.device.index != index:
            raise ValueError(f"stream is on {stream.device}, the tensors are "
                             f"on cuda:{index}")
        self.context = _torch.cuda.stream(stream)
        self.handle = stream.cuda_stream

    def __enter__(self):
        self.context.__enter__()
        return self.handle

    def __exit__(self, *exc):
        return self.context.__exit__(*exc)


def _here(index, stream):
    """The raw handle of the current stream where the call needs no other
    device or stream than the current ones, else None."""
    if stream is None and _torch._C._cuda_getDevice() == index:
        return _torch._C._cuda_getCurrentRawStream(index)
    return None


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
    (rotary_dim/2 radians per position, below 1e6 in magnitude) in place of
    base and scaling.
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
            needs = {"factor"} | ({"original_length"} if kind in
                                  ("yarn", "bands") else set())
            if needs - set(scaling):
                raise ValueError(f"scaling {kind!r} needs "
                                 f"{sorted(needs - set(scaling))}")
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


def _new_like(t, shape, st0, st1):
    """A new dense tensor of t's shape: empty_like, the quicker call, unless
    rows repeat (its strides may then be in any order)."""
    if st0 and st1:
        return _torch.empty_like(t)
    return _torch.empty(shape, dtype=t.dtype, device=t.device)


_ABSENT = (0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0)


def _tail(positions, freqs, tokens, dim, interleaved, eps, index):
    """The fields of mt_rotary_call_t behind the heads."""
    pt = getattr(positions, "dtype", None)
    if pt is _torch.int64:
        size = 8
    elif pt is _torch.int32:
        size = 4
    else:
        raise TypeError(f"positions must be int32 or int64, got {pt}")
    turns, scale, rotary_dim = freqs
    return (_dense(positions, "positions", pt, (tokens,), index),
            _dense(turns, "freqs", _torch.int64, (rotary_dim >> 1,), index),
            tokens, size, dim, rotary_dim, 1 if interleaved else 0,
            0 if eps is None else 1, 0.0 if eps is None else eps, scale, 0)


def _three(t, name):
    sh = t.shape
    if len(sh) != 3:
        raise ValueError(f"{name} must be [tokens, heads, dim]")
    return sh


def _out_pair(out, alone):
    if out is None:
        return None, None
    if alone and not isinstance(out, (tuple, list)):
        return out, None
    return out


def _weight(w, name, dtype, dim, eps, index):
    if w is None:
        return 0
    if eps is None:
        raise ValueError(f"{name} belongs to the norm: give eps")
    return _dense(w, name, dtype, (dim,), index)


def rotary(q, k, positions, freqs, interleaved=False, q_weight=None,
           k_weight=None, eps=None, out=None, stream=None):
    """Rotary positions of the heads of q [tokens, q_heads, dim] and k
    [tokens, k_heads, dim] (None: q alone), each token at its entry of
    positions (int32 or int64).  q and k may be strided views (the last
    dimension dense).  With eps, each head is first RMS-normalised and
    multiplied by q_weight or k_weight (None: ones).  out: (q, k) to write to;
    the inputs themselves turn them in place.  Returns (q, k), or q alone
    where k is None; autograd does not record the call, its gradients are
    :func:`rotary_backward`'s."""
    dt, index = _first(q, "q")
    handle = _here(index, stream)
    if handle is None:
        with _On(index, stream) as handle:
            return _rotary(dt, index, handle, q, k, positions, freqs,
                           interleaved, q_weight, k_weight, eps, out)
    return _rotary(dt, index, handle, q, k, positions, freqs, interleaved,
                   q_weight, k_weight, eps, out)


def _rotary(dt, index, handle, q, k, positions, freqs, interleaved, q_weight,
            k_weight, eps, out):
    dtype, shape = q.dtype, _three(q, "q")
    tokens, q_heads, dim = shape
    tail = _tail(positions, freqs, tokens, dim, interleaved, eps, index)
    x, xt, xh = _heads(q, "q", dtype, shape, index)
    w = _weight(q_weight, "q_weight", dtype, dim, eps, index)
    yq, yk = _out_pair(out, k is None)
    if k is not None:
        k_shape = (tokens, _three(k, "k")[1], dim)
        kx, kxt, kxh = _heads(k, "k", dtype, k_shape, index)
        kw = _weight(k_weight, "k_weight", dtype, dim, eps, index)
    elif k_weight is not None:
        raise ValueError("k_weight without k")
    if yq is None:
        yq = _new_like(q, shape, xt, xh)
    y, yt, yh = _heads(yq, "out (q)", dtype, shape, index)
    if k is None:
        keys = _ABSENT
    else:
        if yk is None:
            yk = _new_like(k, k_shape, kxt, kxh)
        ky, kyt, kyh = _heads(yk, "out (k)", dtype, k_shape, index)
        keys = (kx, 0, ky, kw, 0, kxt, kxh, 0, 0, kyt, kyh, k_shape[1], 0)
    _call("mt_rotary", dt,
          _ROTARY.pack(x, 0, y, w, 0, xt, xh, 0, 0, yt, yh, q_heads, 0,
                       *keys, *tail), handle)
    return yq if k is None else (yq, yk)


def rotary_backward(dq, dk, positions, freqs, interleaved=False, q=None,
                    k=None, q_weight=None, k_weight=None, eps=None, out=None,
                    stream=None):
    """Gradients of :func:`rotary`: dq and dk are those of its outputs, q and
    k its inputs (needed with the norm only), the rest as it was given.
    Returns (dq, dk) of the inputs, with eps (dq, dk, dq_weight, dk_weight),
    the weights' in FP32 (None where there is no weight).  out: (dq, dk) to
    write to; they may be dq and dk themselves."""
    dt, index = _first(dq, "dq")
    if eps is None and (q is not None or k is not None):
        raise ValueError("q and k belong to the norm: give eps")
    if dk is None and (k is not None or k_weight is not None):
        raise ValueError("k without dk")
    handle = _here(index, stream)
    if handle is None:
        with _On(index, stream) as handle:
            return _rotary_backward(dt, index, handle, dq, dk, positions,
                                    freqs, interleaved, q, k, q_weight,
                                    k_weight, eps, out)
    return _rotary_backward(dt, index, handle, dq, dk, positions, freqs,
                            interleaved, q, k, q_weight, k_weight, eps, out)


def _gradients(name, g, x, y, w, dw, tokens, dim, dtype, eps, index):
    """One tensor of a backward call: its fields and its gradient."""
    shape = (tokens, _three(g, "d" + name)[1], dim)
    d, dt_, dh = _heads(g, "d" + name, dtype, shape, index)
    px = xt = xh = 0
    if eps is not None:
        if x is None:
            raise ValueError(f"the norm's backward pass needs {name}")
        px, xt, xh = _heads(x, name, dtype, shape, index)
    pw = _weight(w, name + "_weight", dtype, dim, eps, index)
    if y is None:
        y = _new_like(g, shape, dt_, dh)
    py, yt, yh = _heads(y, f"out ({name})", dtype, shape, index)
    pdw = 0 if dw is None else dw.data_ptr()
    return (px, d, py, pw, pdw, xt, xh, dt_, dh, yt, yh, shape[1], 0), y


def _rotary_backward(dt, index, handle, dq, dk, positions, freqs, interleaved,
                     q, k, q_weight, k_weight, eps, out):
    dtype = dq.dtype
    tokens, _, dim = _three(dq, "dq")
    tail = _tail(positions, freqs, tokens, dim, interleaved, eps, index)
    gq, gk = _out_pair(out, dk is None)
    wq = wk = None
    if eps is not None:
        f32 = _torch.float32
        if q_weight is not None:
            wq = _torch.empty_like(q_weight, dtype=f32)
        if k_weight is not None:
            wk = _torch.empty_like(k_weight, dtype=f32)
    queries, gq = _gradients("q", dq, q, gq, q_weight, wq, tokens, dim, dtype,
                             eps, index)
    keys = _ABSENT
    if dk is not None:
        keys, gk = _gradients("k", dk, k, gk, k_weight, wk, tokens, dim,
                              dtype, eps, index)
    call = _ROTARY.pack(*queries, *keys, *tail)
    n, address = 0, None
    if wq is not None or wk is not None:
        n = mt_rotary_backward_workspace(MtRotaryCall.from_buffer_copy(call))
        workspace = _torch.empty(n, dtype=_torch.uint8, device=dq.device)
        address = workspace.data_ptr()
    _call("mt_rotary_backward", dt, call, address, n, handle)
    return (gq, gk) if eps is None else (gq, gk, wq, wk)


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


_FORMATS = {}


def _cache(cache, name, like, index):
    """(codes' address, scales' address, their shapes) of one cache tensor;
    `like`: the shapes that it has to have, or None."""
    if not _FORMATS:
        _FORMATS.update({_torch.float8_e4m3fn: MT_CACHE_E4M3,
                         _torch.int8: MT_CACHE_INT8})
    codes, scales = cache
    if like is not None:
        return (_dense(codes, name + " codes", like[0], like[1], index),
                _dense(scales, name + " scales", _torch.float32, like[2],
                       index), like)
    _tensor(codes, name + " codes")
    if codes.dtype not in _FORMATS:
        raise TypeError(f"cache codes must be float8_e4m3fn or int8, got "
                        f"{codes.dtype}")
    cs, ss = codes.shape, getattr(scales, "shape", ())
    if len(cs) != 3 or len(ss) != 3:
        raise ValueError("a cache is (codes [slots, heads, dim], scales "
                         "[slots, heads, dim/group])")
    if ss[2] < 1 or cs[2] % ss[2]:
        raise ValueError(f"{ss[2]} scales per head do not divide dim {cs[2]}")
    return _cache(cache, name, (codes.dtype, cs, (cs[0], cs[1], ss[2])),
                  codes.get_device() if index is None else index)


def _cache_pack(kc, ks, kr, vc, vs, vr, slots, like, tokens, index):
    (n, heads, dim), groups = like[1], like[2][2]
    return _CACHE.pack(
        kc, ks, *kr, vc, vs, *vr,
        _dense(slots, "slots", _torch.int64, (tokens,), index), tokens, n,
        heads, dim, dim // groups, _FORMATS[like[0]])


def cache_write(k, v, k_cache, v_cache, slots, stream=None):
    """Stores the rows k and v [tokens, heads, dim] (strided views are fine;
    v and v_cache may be None) as 8-bit codes and scales in the slots
    slots[token] (int64) of k_cache and v_cache, each (codes, scales) as from
    :func:`cache_alloc`.  A token whose slot is outside the cache (-1: padding)
    stores nothing; the slots inside must differ from one another."""
    dt, index = _first(k, "k")
    if (v is None) != (v_cache is None):
        raise ValueError("v and v_cache come together")
    kc, ks, like = _cache(k_cache, "k_cache", None, index)
    tokens = _three(k, "k")[0]
    shape = (tokens, like[1][1], like[1][2])
    kr = _heads(k, "k", k.dtype, shape, index)
    vc = vs = 0
    vr = (0, 0, 0)
    if v is not None:
        vc, vs, _ = _cache(v_cache, "v_cache", like, index)
        vr = _heads(v, "v", k.dtype, shape, index)
    call = _cache_pack(kc, ks, kr, vc, vs, vr, slots, like, tokens, index)
    handle = _here(index, stream)
    if handle is None:
        with _On(index, stream) as handle:
            return _call("mt_cache_write", dt, call, handle)
    _call("mt_cache_write", dt, call, handle)


def cache_read(k_cache, v_cache, slots, dtype=None, out=None, stream=None):
    """The rows of the slots slots[token] (int64), as (k, v) of `dtype` (None:
    torch.bfloat16), or k alone where v_cache is None.  out: (k, v) to write
    to, strided views included; the row of a token whose slot is outside the
    cache is left as it was (in a new output: zero)."""
    if _torch is None:
        _setup()
    kc, ks, like = _cache(k_cache, "k_cache", None, None)
    index = k_cache[0].get_device()
    handle = _here(index, stream)
    if handle is None:
        with _On(index, stream) as handle:
            return _cache_read(kc, ks, like, index, handle, k_cache, v_cache,
                               slots, dtype, out)
    return _cache_read(kc, ks, like, index, handle, k_cache, v_cache, slots,
                       dtype, out)


def _cache_read(kc, ks, like, index, handle, k_cache, v_cache, slots, dtype,
                out):
    k, v = _out_pair(out, v_cache is None)
    if k is not None:
        dt, _ = _first(k, "out (k)")
        dtype = k.dtype if dtype is None else dtype
    else:
        dtype = _torch.bfloat16 if dtype is None else dtype
        dt = _DTYPES.get(dtype)
        if dt is None:
            raise TypeError(f"dtype must be float32, float16 or bfloat16, got "
                            f"{dtype}")
    _tensor(slots, "slots", _torch.int64, (None,), index)
    tokens = slots.shape[0]
    shape = (tokens, like[1][1], like[1][2])
    if k is None:
        k = _torch.zeros(shape, dtype=dtype, device=k_cache[0].device)
    kr = _heads(k, "out (k)", dtype, shape, index)
    vc = vs = 0
    vr = (0, 0, 0)
    if v_cache is not None:
        vc, vs, _ = _cache(v_cache, "v_cache", like, index)
        if v is None:
            v = _torch.zeros(shape, dtype=dtype, device=k_cache[0].device)
        vr = _heads(v, "out (v)", dtype, shape, index)
    _call("mt_cache_read", dt,
          _cache_pack(kc, ks, kr, vc, vs, vr, slots, like, tokens, index),
          handle)
    return k if v_cache is None else (k, v)


def cache_slots(table, offsets, starts, page_size, rows, out=None,
                stream=None):
    """Slots (int64 [rows]) of a packed batch: rows offsets[s] ..
    offsets[s+1]-1 stand at positions starts[s], starts[s]+1, ... of sequence
    s, whose page p/page_size is table[s, p/page_size].  Rows outside the
    batch, and positions without a page (a negative entry, past the table),
    get -1.  table [sequences, pages], offsets [sequences+1] and starts
    [sequences] are int32."""
    if _torch is None:
        _setup()
    i32, i64 = _torch.int32, _torch.int64
    _tensor(table, "table", i32)
    if table.dim() != 2 or (table.shape[1] > 1 and table.stride(1) != 1):
        raise ValueError("table must be [sequences, pages] with dense rows")
    (n, pages), index = table.shape, table.get_device()
    starts_at = _dense(starts, "starts", i32, (n,), index)
    offsets_at = _dense(offsets, "offsets", i32, (n + 1,), index)

    def run(handle, out):
        if out is None:
            out = _torch.empty(rows, dtype=i64, device=table.device)
        mt_cache_slots(table.data_ptr(), table.stride(0), pages, offsets_at,
                       starts_at, n, page_size, rows,
                       _dense(out, "out", i64, (rows,), index), handle)
        return out
    handle = _here(index, stream)
    if handle is None:
        with _On(index, stream) as handle:
            return run(handle, out)
    return run(handle, out)


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
    prompt_lengths[row] are the prompt (int32; None: none), both clamped to
    0..history; ids outside the vocabulary are passed over.  repetition (ids
    of the whole history), frequency and presence (ids after the prompt):
    float32 [rows].  bias_ids [rows, n] int32 and bias [rows, n] float32,
    n <= 1024: values added to single logits.  temperature: float32 [rows].
    mask int32 [rows, words] or [words], words >= (vocab+31)//32: bit v%32 of
    word v//32 allows token v.  The order is: repetition, frequency and
    presence, bias, temperature, mask.
    mode: "logits", "softmax" or "log_softmax"; a row of which the mask leaves
    nothing has probabilities 0 and log-probabilities -inf.  out may be
    logits."""
    dt, index = _first(logits, "logits")
    dtype = logits.dtype
    _tensor(logits, "logits", shape=(None, None))
    x, x_stride, vocab = _rows(logits, "logits", dtype, logits.shape[0], index)
    rows = logits.shape[0]
    kind = _MODES.get(mode)
    if kind is None:
        raise ValueError(f"mode must be one of {sorted(_MODES)}, got {mode!r}")
    f32, i32 = _torch.float32, _torch.int32
    each = (rows,)
    ids = ids_stride = history = count = 0
    lens = prompts = rep = freq = pres = 0
    if tokens is not None:
        ids, ids_stride, history = _rows(tokens, "tokens", i32, rows, index)
        lens = _opt(lengths, "lengths", i32, each, index)
        prompts = _opt(prompt_lengths, "prompt_lengths", i32, each, index)
        rep = _opt(repetition, "repetition", f32, each, index)
        freq = _opt(frequency, "frequency", f32, each, index)
        pres = _opt(presence, "presence", f32, each, index)
        if history == 0:
            ids = lens = prompts = rep = freq = pres = 0
    elif not (lengths is prompt_lengths is repetition is frequency is
              presence is None):
        raise ValueError("lengths and penalties need tokens")
    b_ids = b = 0
    if bias is not None or bias_ids is not None:
        if bias is None or bias_ids is None:
            raise ValueError("bias and bias_ids come together")
        _tensor(bias_ids, "bias_ids", i32, (rows, None), index)
        count = bias_ids.shape[1]
        b_ids = _dense(bias_ids, "bias_ids", i32, (rows, count), index)
        b = _dense(bias, "bias", f32, (rows, count), index)
    m = m_stride = 0
    if mask is not None:
        if mask.dim() == 1:
            mask = mask[None].expand(rows, -1)
        m, m_stride, words = _rows(mask, "mask", i32, rows, index)
        if words < (vocab + 31) >> 5:
            raise ValueError(f"mask needs {(vocab + 31) >> 5} words per row, "
                             f"got {words}")
        if rows == 1:
            m_stride = 0
    temp = _opt(temperature, "temperature", f32, each, index)

    def run(handle, out):
        if out is None:
            out = _new_like(logits, logits.shape, x_stride, 1)
        y, y_stride, width = _rows(out, "out", dtype, rows, index)
        if width != vocab:
            raise ValueError(f"out must have shape {tuple(logits.shape)}, got "
                             f"{tuple(out.shape)}")
        _call("mt_process_logits", dt,
              _LOGITS.pack(x, y, rows, x_stride, y_stride, vocab, kind, ids,
                           ids_stride, history, count, lens, prompts, rep,
                           freq, pres, b_ids, b, m, m_stride, temp), handle)
        return out
    handle = _here(index, stream)
    if handle is None:
        with _On(index, stream) as handle:
            return run(handle, out)
    return run(handle, out)

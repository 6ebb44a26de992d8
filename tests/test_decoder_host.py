"""The decoder's row operators without a GPU: the header and the library's
exports, frequencies and turns, and every refusal (arguments are checked
before any CUDA call)."""
import ctypes
import math
import os
import re
import subprocess

import pytest
import torch

import row_reduction_gb300 as mt
from decoder_util import norm64, rotary_backward_ref, rotate
from row_reduction_gb300 import _decoder as dec
from row_reduction_gb300 import build as mt_build

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
INV, UNS, OOR = (mt.MT_ERR_INVALID_ARGUMENT, mt.MT_ERR_UNSUPPORTED,
                 mt.MT_ERR_OUT_OF_RESOURCES)
A = 0x10000000  # addresses that are never used: every call is refused first


@pytest.fixture(scope="module", autouse=True)
def built():
    mt_build.build()


def test_library_exports_every_declared_symbol():
    src = open(os.path.join(ROOT, "include", "mt_decoder.h")).read()
    declared = sorted(set(re.findall(r"^MT_API[^(]*?\b(mt_\w+)\s*\(", src,
                                     flags=re.M)))
    assert sorted(mt.DECODER_EXPORTS) == declared
    for name in declared:
        assert hasattr(mt.lib(), name), name


@pytest.mark.parametrize("std,lang", [("c99", "c"), ("c++11", "c++")])
def test_header_is_plain_c_and_matches_the_structures(tmp_path, std, lang):
    sizes = {"mt_rotary_scaling_t": dec.MtRotaryScaling,
             "mt_rotary_heads_t": dec.MtRotaryHeads,
             "mt_rotary_call_t": dec.MtRotaryCall,
             "mt_cache_rows_t": dec.MtCacheRows,
             "mt_cache_call_t": dec.MtCacheCall,
             "mt_logits_call_t": dec.MtLogitsCall}
    lines = []
    for name, cls in sizes.items():
        lines.append(f'printf("{name} %d\\n", (int)sizeof({name}));')
        for f, _ in cls._fields_:
            lines.append(f'printf("{name}.{f} %d\\n", '
                         f'(int)offsetof({name}, {f}));')
    src = tmp_path / "inc.c"
    src.write_text('#include <stdio.h>\n#include <stddef.h>\n'
                   '#include "mt_decoder.h"\nint main(void) {\n' +
                   "\n".join(lines) + "\nreturn 0;\n}\n")
    exe = tmp_path / "inc"
    subprocess.run(["gcc" if lang == "c" else "g++", f"-std={std}", "-Wall",
                    "-Wextra", "-pedantic", "-Werror", "-x", lang, "-I",
                    os.path.join(ROOT, "include"), str(src), "-o", str(exe)],
                   check=True)
    out = subprocess.run([str(exe)], capture_output=True, text=True,
                         check=True).stdout
    got = dict(line.split() for line in out.splitlines())
    for name, cls in sizes.items():
        assert int(got[name]) == ctypes.sizeof(cls), name
        for f, _ in cls._fields_:
            assert int(got[f"{name}.{f}"]) == getattr(cls, f).offset, (name, f)


# ---- frequencies -------------------------------------------------------------
def scaling(kind, **kw):
    return dec.MtRotaryScaling(type=kind, **kw)


def test_plain_linear_and_ntk_frequencies():
    f, s = mt.mt_rotary_frequencies(8, 10000.0)
    assert s == 1.0
    assert f == pytest.approx([1.0, 0.1, 0.01, 0.001], rel=1e-15)
    f, s = mt.mt_rotary_frequencies(8, 10000.0,
                                    scaling(mt.MT_ROTARY_LINEAR, factor=4.0))
    assert f == pytest.approx([0.25, 0.025, 0.0025, 0.00025], rel=1e-15)
    # the fastest pair stays, the slowest is divided by the factor
    f, s = mt.mt_rotary_frequencies(8, 10000.0,
                                    scaling(mt.MT_ROTARY_NTK, factor=4.0))
    assert f[0] == 1.0 and f[-1] == pytest.approx(0.001 / 4, rel=1e-14)


def test_yarn_and_bands_keep_fast_pairs_and_stretch_slow_ones():
    n, base, s, length = 128, 10000.0, 8.0, 4096.0
    plain, _ = mt.mt_rotary_frequencies(n, base)
    for kind, low, high in ((mt.MT_ROTARY_YARN, 1.0, 32.0),
                            (mt.MT_ROTARY_BANDS, 1.0, 4.0)):
        f, factor = mt.mt_rotary_frequencies(
            n, base, scaling(kind, factor=s, original_length=length, low=low,
                             high=high))
        assert factor == (pytest.approx(0.1 * math.log(s) + 1, rel=1e-15)
                          if kind == mt.MT_ROTARY_YARN else 1.0)
        for i, (p, q) in enumerate(zip(plain, f)):
            turns = length * p / (2 * math.pi)
            keep = (p / s - q) / (p / s - p)
            if kind == mt.MT_ROTARY_BANDS:
                want = min(max((turns - low) / (high - low), 0.0), 1.0)
                assert keep == pytest.approx(want, abs=1e-12)
            else:
                pair = lambda r: n * math.log(length / (r * 2 * math.pi)) / (2 * math.log(base))  # noqa: E731
                lo = max(math.floor(pair(high)), 0)
                hi = min(math.ceil(pair(low)), n - 1)
                want = 1 - min(max((i - lo) / (hi - lo), 0.0), 1.0)
                assert keep == pytest.approx(want, abs=1e-12)
        assert f[0] == 1.0 and f[-1] == pytest.approx(plain[-1] / s, rel=1e-14)


def test_turns_are_the_frequencies_to_64_bits():
    from decimal import Decimal, getcontext
    getcontext().prec = 60
    two_pi = 2 * Decimal("3.14159265358979323846264338327950288419716939937510"
                         "58209749445923")
    freqs = [1.0, 0.1, 1e-9, 6.283185307179586, 7.0, 1000.5, -1.0, -1e-9, 0.0]
    for f, t in zip(freqs, mt.mt_rotary_turns(freqs)):
        want = Decimal(f) / two_pi * 2 ** 64
        off = (Decimal(t) - want) % 2 ** 64
        off = min(off, 2 ** 64 - off)
        # floor and two conversions: one unit, and the product's low part
        # rounds at 2^-106 of the frequency in turns
        assert off <= 2 + abs(want) * Decimal(2) ** -104, (f, off)


def test_frequencies_refuse():
    ok = dict(factor=2.0, original_length=100.0, low=1.0, high=4.0)
    for n, base, sc in (
            (7, 10000.0, None), (0, 10000.0, None), (514, 10000.0, None),
            (8, 1.0, None), (8, math.nan, None), (8, math.inf, None),
            (8, 10.0, scaling(9, **ok)), (8, 10.0, scaling(-1, **ok)),
            (2, 10.0, scaling(mt.MT_ROTARY_NTK, **ok)),
            (8, 10.0, scaling(mt.MT_ROTARY_LINEAR, factor=0.5)),
            (8, 10.0, scaling(mt.MT_ROTARY_LINEAR, factor=math.inf)),
            (8, 10.0, scaling(mt.MT_ROTARY_YARN, factor=2.0)),
            (8, 10.0, scaling(mt.MT_ROTARY_BANDS, **dict(ok, low=4.0))),
            (8, 10.0, scaling(mt.MT_ROTARY_BANDS, **dict(ok, low=0.0)))):
        with pytest.raises(mt.MTError) as e:
            mt.mt_rotary_frequencies(n, base, sc)
        assert e.value.status == INV
    for f in (math.nan, math.inf, 1e7):
        with pytest.raises(mt.MTError):
            mt.mt_rotary_turns([1.0, f])
    with pytest.raises(ValueError, match="unknown scaling keys"):
        mt.rotary_frequencies(8, scaling={"type": "linear", "facter": 2.0},
                              device="cpu")
    with pytest.raises(ValueError, match="scaling type"):
        mt.rotary_frequencies(8, scaling={"type": "cubic", "factor": 2.0},
                              device="cpu")
    with pytest.raises(ValueError, match="needs 4 frequencies"):
        mt.rotary_frequencies(8, freqs=[1.0], device="cpu")


# ---- the plain formulas ---------------------------------------------------------
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("eps", [None, 1e-6])
def test_plain_gradients_match_differences(interleaved, eps):
    """The 64-bit gradients that the GPU tests compare with, against central
    differences of the 64-bit forward (error of order h^2 = 1e-10, and
    rounding 1e-16/h)."""
    gen = torch.Generator().manual_seed(1)
    x = torch.randn(3, 2, 10, generator=gen, dtype=torch.float64)
    dy = torch.randn(3, 2, 10, generator=gen, dtype=torch.float64)
    w = None if eps is None else \
        1 + 0.1 * torch.randn(10, generator=gen, dtype=torch.float64)
    pos = torch.tensor([0, 5, 1000])
    freqs = [1.0, 0.3, 0.01]

    def loss(x, w):
        z = x if eps is None else norm64(x, w, eps)[0]
        return float((rotate(z, pos, freqs, 1.25, 6, interleaved) * dy).sum())
    dx, _, dw, _ = rotary_backward_ref(dy, x, pos, freqs, 1.25, 6,
                                       interleaved, w, eps)
    h = 1e-5
    for i in range(x.numel()):
        step = torch.zeros(x.numel(), dtype=torch.float64)
        step[i] = h
        step = step.view_as(x)
        want = (loss(x + step, w) - loss(x - step, w)) / (2 * h)
        assert float(dx.flatten()[i]) == pytest.approx(want, abs=1e-7)
    if eps is not None:
        for i in range(10):
            step = torch.zeros(10, dtype=torch.float64)
            step[i] = h
            want = (loss(x, w + step) - loss(x, w - step)) / (2 * h)
            assert float(dw[i]) == pytest.approx(want, abs=1e-7)


# ---- refusals: rotary --------------------------------------------------------
def heads(x=A, y=2 * A, dy=None, n=2, weight=None, dweight=None, dim=16,
          **kw):
    h = dec.MtRotaryHeads(x=x, dy=dy, y=y, weight=weight, dweight=dweight,
                          heads=n, x_token=n * dim, x_head=dim,
                          dy_token=n * dim, dy_head=dim, y_token=n * dim,
                          y_head=dim)
    for k, v in kw.items():
        setattr(h, k, v)
    return h


def call(q=None, k=None, **kw):
    c = dec.MtRotaryCall(
        q=heads() if q is None else q,
        k=heads(n=0) if k is None else k, positions=A, turns=A, tokens=4,
        position_bytes=8, dim=16, rotary_dim=16, scale=1.0)
    for name, v in kw.items():
        setattr(c, name, v)
    return c


@pytest.mark.parametrize("c,want", [
    (call(dim=0), INV), (call(rotary_dim=15), INV), (call(rotary_dim=18), INV),
    (call(rotary_dim=0), INV), (call(tokens=-1), INV),
    (call(interleaved=2), INV), (call(norm=2), INV), (call(reserved=1), INV),
    (call(position_bytes=2), INV), (call(positions=None), INV),
    (call(positions=A + 4), INV), (call(turns=None), INV),
    (call(turns=A + 4), INV), (call(dim=514), UNS),
    (call(norm=1, eps=-1.0), INV), (call(norm=1, eps=math.nan), INV),
    (call(q=heads(x=None)), INV), (call(q=heads(y=None)), INV),
    (call(q=heads(x=A + 1)), INV), (call(q=heads(n=-1)), INV),
    (call(q=heads(n=65537, x_token=0, y_token=65537 * 16)), UNS),
    (call(q=heads(dy=A)), INV), (call(q=heads(dweight=A)), INV),
    (call(q=heads(weight=A)), INV),           # weight without norm
    (call(k=heads(y=None)), INV),
    (call(q=heads(y_head=8)), INV),           # rows of the output overlap
    (call(q=heads(y_token=16)), INV), (call(q=heads(y_token=0)), INV),
    (call(q=heads(x_token=2 ** 62)), INV),    # offsets past an int64
    (call(tokens=2 ** 33 + 1, q=heads(n=1)), UNS),
])
@pytest.mark.parametrize("dtype", [1, 2])
def test_rotary_refuses(c, want, dtype):
    with pytest.raises(mt.MTError) as e:
        mt.mt_rotary(dtype, c, None)
    assert e.value.status == want


def test_rotary_refuses_types_and_accepts_nothing_to_do():
    for dtype in (-1, 3):
        with pytest.raises(mt.MTError):
            mt.mt_rotary(dtype, call(), None)
    with pytest.raises(mt.MTError):
        mt.mt_rotary(0, call(q=heads(x=A + 2)), None)  # 4-byte elements
    mt.mt_rotary(0, call(tokens=0), None)
    mt.mt_rotary(0, call(q=heads(n=0), positions=None), None)
    mt.mt_rotary(0, call(q=heads(x=None, y=None), tokens=0), None)


@pytest.mark.parametrize("c,ws,n,want", [
    (call(q=heads(x=None, dy=None)), None, 0, INV),
    (call(q=heads(dy=A)), None, 0, INV),          # x without norm
    (call(q=heads(x=None, dy=A, dweight=A)), None, 0, INV),
    (call(q=heads(dy=A, x=None), norm=1), None, 0, INV),
    (call(q=heads(dy=A, dweight=A), norm=1), A, 16, OOR),
    (call(q=heads(dy=A, dweight=A), norm=1), None, 1 << 20, INV),
    (call(q=heads(dy=A, dweight=A), norm=1), A + 8, 1 << 20, INV),
    (call(q=heads(dy=A, dweight=A + 2), norm=1), A, 1 << 20, INV),
    (call(q=heads(dy=A, dy_token=2 ** 62), norm=1), None, 0, INV),
])
def test_rotary_backward_refuses(c, ws, n, want):
    with pytest.raises(mt.MTError) as e:
        mt.mt_rotary_backward(2, c, ws, n, None)
    assert e.value.status == want


def test_rotary_backward_workspace():
    assert mt.mt_rotary_backward_workspace(call()) == 0
    assert mt.mt_rotary_backward_workspace(
        call(norm=1, q=heads(dy=A))) == 0
    n = mt.mt_rotary_backward_workspace(
        call(norm=1, q=heads(dy=A, dweight=A)))
    assert n == 304 * 16 * 4
    with pytest.raises(mt.MTError):
        mt.mt_rotary_backward_workspace(call(dim=513))


# ---- refusals: cache -----------------------------------------------------------
def rows(**kw):
    r = dec.MtCacheRows(codes=A, scales=A, rows=A, token_stride=32,
                        head_stride=16)
    for k, v in kw.items():
        setattr(r, k, v)
    return r


def cache(k=None, v=None, **kw):
    c = dec.MtCacheCall(k=rows() if k is None else k,
                        v=dec.MtCacheRows() if v is None else v, slot=A,
                        tokens=4, slots=64, heads=2, dim=16, group=16,
                        format=0)
    for name, val in kw.items():
        setattr(c, name, val)
    return c


@pytest.mark.parametrize("write", [True, False])
@pytest.mark.parametrize("c,want", [
    (cache(tokens=-1), INV), (cache(slots=-1), INV), (cache(heads=0), INV),
    (cache(dim=0), INV), (cache(group=0), INV), (cache(group=5), INV),
    (cache(group=32), INV), (cache(format=2), INV), (cache(format=-1), INV),
    (cache(slot=None), INV), (cache(slot=A + 4), INV),
    (cache(k=rows(codes=None)), INV), (cache(k=rows(scales=None)), INV),
    (cache(k=rows(rows=None)), INV), (cache(k=rows(rows=A + 1)), INV),
    (cache(k=rows(scales=A + 2)), INV),
    (cache(v=dec.MtCacheRows(codes=A)), INV),   # half a value tensor
    (cache(heads=1 << 20, dim=16), UNS),
    (cache(slots=2 ** 60), INV),
    (cache(k=rows(token_stride=2 ** 62)), INV),
    (cache(tokens=2 ** 36), UNS), (cache(tokens=2 ** 28, group=4), UNS),
])
def test_cache_refuses(c, want, write):
    with pytest.raises(mt.MTError) as e:
        (mt.mt_cache_write if write else mt.mt_cache_read)(2, c, None)
    assert e.value.status == want


def test_cache_read_refuses_overlapping_outputs_and_accepts_nothing_to_do():
    with pytest.raises(mt.MTError):
        mt.mt_cache_read(2, cache(k=rows(token_stride=0)), None)
    for f in (mt.mt_cache_read, mt.mt_cache_write):
        f(2, cache(tokens=0), None)
        f(2, cache(tokens=0, slot=None, k=dec.MtCacheRows()), None)
        f(2, cache(slots=0), None)
        with pytest.raises(mt.MTError):
            f(3, cache(), None)


@pytest.mark.parametrize("kw", [
    dict(pages_per_sequence=-1), dict(sequences=-1), dict(page_size=0),
    dict(rows=-1), dict(table_stride=-1), dict(slot=None),
    dict(offsets=None), dict(starts=None), dict(table=None),
    dict(table=A + 2), dict(slot=A + 4), dict(table_stride=2 ** 62)])
def test_cache_slots_refuses(kw):
    a = dict(table=A, table_stride=8, pages_per_sequence=8, offsets=A,
             starts=A, sequences=3, page_size=16, rows=5, slot=A, stream=None)
    with pytest.raises(mt.MTError) as e:
        mt.mt_cache_slots(**{**a, **kw})
    assert e.value.status == INV
    mt.mt_cache_slots(**{**a, "rows": 0, "slot": None})


# ---- refusals: logits ----------------------------------------------------------
def logits(**kw):
    c = dec.MtLogitsCall(x=A, y=A, rows=2, x_stride=100, y_stride=100,
                         vocab=100)
    for k, v in kw.items():
        setattr(c, k, v)
    return c


@pytest.mark.parametrize("c,want", [
    (logits(rows=-1), INV), (logits(vocab=0), INV), (logits(mode=3), INV),
    (logits(mode=-1), INV), (logits(history=-1), INV),
    (logits(biases=-1), INV), (logits(vocab=524281, y_stride=524281), UNS),
    (logits(history=1 << 20, tokens=A), UNS), (logits(biases=1025), UNS),
    (logits(x=None), INV), (logits(y=None), INV), (logits(x=A + 1), INV),
    (logits(y=A + 1), INV), (logits(history=4), INV),
    (logits(tokens=A + 2, history=4), INV), (logits(lengths=A), INV),
    (logits(repetition=A), INV), (logits(frequency=A), INV),
    (logits(presence=A), INV), (logits(prompt_lengths=A), INV),
    (logits(biases=2), INV), (logits(biases=2, bias=A), INV),
    (logits(biases=2, bias_ids=A), INV),
    (logits(mask=A, mask_stride=3), INV), (logits(y_stride=99), INV),
    (logits(x_stride=-100), INV),
    (logits(tokens=A, history=4, tokens_stride=-4), INV),
    (logits(x_stride=2 ** 62), INV), (logits(temperature=A + 2), INV),
    (logits(rows=2 ** 24 + 1), UNS),
])
def test_process_logits_refuses(c, want):
    with pytest.raises(mt.MTError) as e:
        mt.mt_process_logits(2, c, None)
    assert e.value.status == want


def test_process_logits_accepts_nothing_to_do():
    mt.mt_process_logits(2, logits(rows=0), None)
    mt.mt_process_logits(0, logits(rows=0, x=None, y=None), None)
    with pytest.raises(mt.MTError):
        mt.mt_process_logits(3, logits(), None)


def test_tensor_functions_refuse_cpu_tensors():
    x = torch.zeros(2, 3, 16)
    f = mt.rotary_frequencies(16, device="cpu")
    with pytest.raises(ValueError, match="CUDA"):
        mt.rotary(x, x, torch.zeros(2, dtype=torch.int64), f)
    with pytest.raises(ValueError, match="CUDA"):
        mt.rotary_backward(x, x, torch.zeros(2, dtype=torch.int64), f)
    with pytest.raises(ValueError, match="CUDA"):
        mt.process_logits(x[0])
    c = mt.cache_alloc(4, 3, 16, device="cpu")
    with pytest.raises(ValueError, match="CUDA"):
        mt.cache_write(x, x, c, c, torch.zeros(2, dtype=torch.int64))
    with pytest.raises(ValueError, match="CUDA"):
        mt.cache_read(c, None, torch.zeros(2, dtype=torch.int64))
    with pytest.raises(ValueError, match="CUDA"):
        mt.cache_slots(torch.zeros(2, 2, dtype=torch.int32), x, x, 16, 4)
    with pytest.raises(ValueError, match="divide"):
        mt.cache_alloc(4, 3, 16, group=5, device="cpu")
    with pytest.raises(ValueError, match="format"):
        mt.cache_alloc(4, 3, 16, format="int4", device="cpu")


def test_packed_structures_match_the_header():
    for packed, cls in ((dec._ROTARY, dec.MtRotaryCall),
                        (dec._CACHE, dec.MtCacheCall),
                        (dec._LOGITS, dec.MtLogitsCall)):
        assert packed.size == ctypes.sizeof(cls)

        def leaves(c):
            out = []
            for name, kind in c._fields_:
                if issubclass(kind, ctypes.Structure):
                    out += leaves(kind)
                else:
                    out.append(kind)
            return out
        kinds = leaves(cls)
        values = [float(i) if k is ctypes.c_float else i + 1
                  for i, k in enumerate(kinds)]
        got = cls.from_buffer_copy(packed.pack(*values))

        def read(c):
            out = []
            for name, kind in c._fields_:
                v = getattr(c, name)
                out += read(v) if isinstance(v, ctypes.Structure) else [v]
            return out
        assert read(got) == values

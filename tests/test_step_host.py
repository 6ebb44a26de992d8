"""The operators around a decoder's cache without a GPU: structures, every
refusal of the C entry points (before any CUDA call), and the plain gradients
against differences."""
import ctypes
import math
import os
import subprocess

import pytest
import torch

import row_reduction_gb300 as mt
from row_reduction_gb300 import _step as st
from row_reduction_gb300 import build as mt_build
from step_util import block_norm_back_ref, block_norm_ref

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
INV, UNS, OOR = (mt.MT_ERR_INVALID_ARGUMENT, mt.MT_ERR_UNSUPPORTED,
                 mt.MT_ERR_OUT_OF_RESOURCES)
F32, F16, BF16 = 0, 1, 2
A = 0x10000000  # addresses that are never used: every call is refused first
MAX32 = 2 ** 31 - 1


@pytest.fixture(scope="module", autouse=True)
def built():
    mt_build.build()


@pytest.mark.parametrize("std,lang", [("c99", "c"), ("c++11", "c++")])
def test_structures_match_the_header(tmp_path, std, lang):
    sizes = {"mt_cache_extend_call_t": st.MtCacheExtendCall,
             "mt_attention_call_t": st.MtAttentionCall,
             "mt_block_norm_call_t": st.MtBlockNormCall,
             "mt_block_norm_back_t": st.MtBlockNormBack}
    lines = ['printf("after %d\\nbefore %d\\n", MT_NORM_AFTER, '
             'MT_NORM_BEFORE);']
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
    assert (int(got["after"]), int(got["before"])) == (
        mt.MT_NORM_AFTER, mt.MT_NORM_BEFORE)
    for name, cls in sizes.items():
        assert int(got[name]) == ctypes.sizeof(cls), name
        for f, _ in cls._fields_:
            assert int(got[f"{name}.{f}"]) == getattr(cls, f).offset, (name, f)
    for packed, cls in ((st._EXTEND, st.MtCacheExtendCall),
                        (st._ATTENTION, st.MtAttentionCall),
                        (st._NORM, st.MtBlockNormCall),
                        (st._NORM_BACK, st.MtBlockNormBack)):
        assert packed.size == ctypes.sizeof(cls)


def refused(status, fn, *args):
    with pytest.raises(mt.MTError) as e:
        fn(*args)
    assert e.value.status == status, args[-3:]


def changed(call, **kw):
    c = type(call).from_buffer_copy(call)
    for k, v in kw.items():
        assert hasattr(c, k)
        setattr(c, k, v)
    return c


# ---- pages of a step ---------------------------------------------------------
EXTEND = st.MtCacheExtendCall(
    table=A, table_stride=8, lengths=2 * A, counts=3 * A, free_pages=4 * A,
    free_count=5 * A, offsets=6 * A, slots=7 * A, positions=8 * A,
    new_lengths=9 * A, new_free_count=10 * A, rows=4, pages=8, sequences=3,
    free_size=5, page_size=16)


@pytest.mark.parametrize("status,change", [
    (INV, dict(rows=-1)), (INV, dict(pages=-1)), (INV, dict(sequences=-1)),
    (INV, dict(free_size=-1)), (INV, dict(page_size=0)),
    (INV, dict(table_stride=-1)), (INV, dict(table_stride=7)),
    (INV, dict(table_stride=2 ** 62)),
    (INV, dict(table=None)), (INV, dict(lengths=None)),
    (INV, dict(counts=None)), (INV, dict(free_pages=None)),
    (INV, dict(free_count=None)), (INV, dict(offsets=None)),
    (INV, dict(slots=None)), (INV, dict(positions=None)),
    (INV, dict(new_lengths=None)), (INV, dict(new_free_count=None)),
    (INV, dict(new_lengths=2 * A)), (INV, dict(new_lengths=3 * A)),
    (INV, dict(new_free_count=5 * A)), (INV, dict(table=A + 2)),
    (INV, dict(slots=7 * A + 4)), (INV, dict(positions=8 * A + 1)),
    (INV, dict(free_pages=A + 1)), (INV, dict(offsets=A + 1)),
    (UNS, dict(rows=2 ** 31)), (UNS, dict(sequences=MAX32)),
    (UNS, dict(free_size=MAX32))])
def test_extend_refuses(status, change):
    refused(status, mt.mt_cache_extend, changed(EXTEND, **change), None)


def test_extend_refuses_nothing():
    assert mt.lib().mt_cache_extend(None, None) == INV


# ---- attention ---------------------------------------------------------------
ATTENTION = st.MtAttentionCall(
    q=A, out=2 * A, lse=3 * A, q_row=512, q_head=128, out_row=512,
    out_head=128, k_codes=4 * A, v_codes=5 * A, k_scales=6 * A,
    v_scales=7 * A, table=8 * A, table_stride=10, offsets=9 * A,
    starts=10 * A, first=11 * A, last=12 * A, slopes=13 * A, rows=6,
    slots=1000, sequences=2, pages=10, page_size=16, q_heads=4, k_heads=2,
    dim=128, group=64, format=mt.MT_CACHE_E4M3, window=0, scale=0.1, cap=0.0,
    reserved=0)


@pytest.mark.parametrize("status,change", [
    (INV, dict(rows=-1)), (INV, dict(slots=-1)), (INV, dict(sequences=-1)),
    (INV, dict(pages=-1)), (INV, dict(page_size=0)), (INV, dict(k_heads=0)),
    (INV, dict(q_heads=0)), (INV, dict(q_heads=5)), (INV, dict(dim=0)),
    (INV, dict(group=0)), (INV, dict(group=48)), (INV, dict(window=-1)),
    (INV, dict(reserved=1)), (INV, dict(format=2)), (INV, dict(format=-1)),
    (INV, dict(scale=math.nan)), (INV, dict(scale=math.inf)),
    (INV, dict(cap=-1.0)), (INV, dict(cap=math.nan)),
    (INV, dict(cap=math.inf)), (INV, dict(table_stride=-1)),
    (INV, dict(table_stride=2 ** 62)), (INV, dict(slots=2 ** 60)),
    (INV, dict(q_row=2 ** 62)), (INV, dict(out_row=100)),
    (INV, dict(out_head=64)), (INV, dict(out_row=0)),
    (INV, dict(q=None)), (INV, dict(out=None)), (INV, dict(k_codes=None)),
    (INV, dict(v_codes=None)), (INV, dict(k_scales=None)),
    (INV, dict(v_scales=None)), (INV, dict(table=None)),
    (INV, dict(offsets=None)), (INV, dict(starts=None)),
    (INV, dict(q=A + 1)), (INV, dict(out=A + 1)), (INV, dict(lse=A + 2)),
    (INV, dict(k_scales=A + 2)), (INV, dict(first=A + 2)),
    (INV, dict(slopes=A + 1)), (INV, dict(offsets=A + 3)),
    (UNS, dict(dim=1024, group=1024, out_row=4096, out_head=1024)),
    (UNS, dict(q_heads=65538, out_row=65538 * 128)),
    (UNS, dict(rows=2 ** 31))])
def test_attention_refuses(status, change):
    c = changed(ATTENTION, **change)
    refused(status, mt.mt_cache_attention, BF16, c, A, 1 << 30, None)
    refused(status, mt.mt_cache_attention_workspace, BF16, c)


def test_attention_refuses_types_and_takes_empty_calls():
    for dt in (-1, 3):
        refused(INV, mt.mt_cache_attention, dt, ATTENTION, A, 1 << 30, None)
    assert mt.lib().mt_cache_attention(BF16, None, A, 1 << 30, None) == INV
    for kw in (dict(rows=0), dict(sequences=0)):
        c = changed(ATTENTION, **kw)
        mt.mt_cache_attention(BF16, c, None, 0, None)
        assert mt.mt_cache_attention_workspace(BF16, c) == 0


# ---- norms around a block ----------------------------------------------------
NORM = st.MtBlockNormCall(
    x=A, residual=2 * A, gate=3 * A, weight=4 * A, next_weight=5 * A,
    h=6 * A, y=7 * A, x_stride=64, residual_stride=64, gate_stride=0,
    h_stride=64, y_stride=64, rows=4, cols=64, norms=3, eps=1e-6,
    residual_scale=1.0)
BACK = st.MtBlockNormBack(
    dy=A, dh=2 * A, x=3 * A, h=4 * A, gate=5 * A, weight=6 * A,
    next_weight=7 * A, dx=8 * A, dresidual=9 * A, dgate=None,
    dgate_sum=10 * A, dweight=11 * A, dnext_weight=12 * A, dy_stride=64,
    dh_stride=64, x_stride=64, h_stride=64, gate_stride=0, dx_stride=64,
    dresidual_stride=64, dgate_stride=64, rows=4, cols=64, norms=3, eps=1e-6,
    residual_scale=1.0)
SIZES = [(INV, dict(rows=-1)), (INV, dict(cols=0)), (INV, dict(norms=0)),
         (INV, dict(norms=4)), (INV, dict(eps=-1.0)),
         (INV, dict(eps=math.nan)), (INV, dict(residual_scale=math.inf)),
         (INV, dict(residual_scale=math.nan)), (INV, dict(x_stride=2 ** 62)),
         (INV, dict(gate_stride=2 ** 62)), (INV, dict(x=A + 1)),
         (INV, dict(weight=A + 1)), (INV, dict(next_weight=A + 1)),
         (UNS, dict(cols=(1 << 20) + 1)), (UNS, dict(rows=2 ** 31))]


@pytest.mark.parametrize("status,change", SIZES + [
    (INV, dict(x=None)), (INV, dict(residual=None)), (INV, dict(h=None)),
    (INV, dict(y=None)), (INV, dict(h=7 * A)), (INV, dict(h_stride=63)),
    (INV, dict(y_stride=0)), (INV, dict(y_stride=-64)),
    (INV, dict(norms=2)),               # weight without its norm
    (INV, dict(norms=1)),               # next_weight and y without theirs
    (INV, dict(norms=1, next_weight=None)), (INV, dict(residual=A + 1))])
def test_block_norm_refuses(status, change):
    refused(status, mt.mt_block_norm, BF16, changed(NORM, **change), None)


@pytest.mark.parametrize("status,change", SIZES + [
    (INV, dict(dy=None)), (INV, dict(h=None)), (INV, dict(x=None)),
    (INV, dict(dx=None)), (INV, dict(dresidual=None)),
    (INV, dict(dx=9 * A)), (INV, dict(dgate=13 * A)),
    (INV, dict(dgate=8 * A, dgate_sum=None)),
    (INV, dict(dgate=13 * A, dgate_sum=None, dgate_stride=8)),
    (INV, dict(gate=None)), (INV, dict(gate=None, dgate_sum=None,
                                       dgate=A)),
    (INV, dict(dx_stride=63)), (INV, dict(dresidual_stride=0)),
    (INV, dict(norms=2)), (INV, dict(norms=2, weight=None)),
    (INV, dict(norms=1)), (INV, dict(norms=1, dy=None, h=None)),
    (INV, dict(norms=1, dy=None, h=None, next_weight=None,
               dnext_weight=None, dh=None)),
    (INV, dict(norms=2, weight=None, dweight=None, x=None)),
    (INV, dict(dweight=A + 2)), (INV, dict(dgate_sum=A + 1))])
def test_block_norm_backward_refuses(status, change):
    refused(status, mt.mt_block_norm_backward, BF16, changed(BACK, **change),
            A, 1 << 30, None)


def test_block_norm_backward_workspace():
    need = mt.mt_block_norm_backward_workspace(BF16, BACK)
    assert need > 0
    refused(OOR, mt.mt_block_norm_backward, BF16, BACK, A, need - 1, None)
    refused(INV, mt.mt_block_norm_backward, BF16, BACK, None, need, None)
    refused(INV, mt.mt_block_norm_backward, BF16, BACK, A + 8, need, None)
    none = changed(BACK, dgate_sum=None, dweight=None, dnext_weight=None)
    assert mt.mt_block_norm_backward_workspace(BF16, none) == 0
    refused(UNS, mt.mt_block_norm_backward_workspace, BF16,
            changed(BACK, cols=(1 << 20) + 1))


def test_block_norm_types_and_empty_calls():
    for dt in (-1, 3):
        refused(INV, mt.mt_block_norm, dt, NORM, None)
        refused(INV, mt.mt_block_norm_backward, dt, BACK, A, 1 << 30, None)
    mt.mt_block_norm(BF16, changed(NORM, rows=0, x=None, h=None), None)
    mt.mt_block_norm_backward(
        BF16, changed(BACK, rows=0, dgate_sum=None, dweight=None,
                      dnext_weight=None), None, 0, None)


# ---- the plain formulas ------------------------------------------------------
@pytest.mark.parametrize("norms", ["both", "before", "after"])
@pytest.mark.parametrize("gate", ["none", "vector", "matrix"])
def test_plain_gradients_match_differences(norms, gate):
    """The 64-bit gradients that the GPU tests compare with, against central
    differences of the 64-bit forward (h^2 = 1e-10, rounding 1e-16 / h)."""
    g = torch.Generator().manual_seed(1)

    def rand(*shape):
        return torch.randn(*shape, generator=g, dtype=torch.float64)
    rows, cols, scale, eps = 3, 7, 0.7, 1e-2
    t = dict(x=rand(rows, cols), residual=rand(rows, cols),
             gate={"none": None, "vector": rand(cols),
                   "matrix": rand(rows, cols)}[gate],
             weight=rand(cols) if norms != "before" else None,
             next_weight=rand(cols) if norms != "after" else None)
    dy, dh = rand(rows, cols), rand(rows, cols)

    def forward(t):
        return block_norm_ref(t["x"], t["residual"], t["weight"], t["gate"],
                              t["next_weight"], norms, scale, eps)

    def loss(t):
        y, _, h, _ = forward(t)
        return float((h * dh).sum() + (0 if y is None else (y * dy).sum()))
    h = forward(t)[2]
    got = block_norm_back_ref(dy if norms != "after" else None, dh, t["x"], h,
                              t["weight"], t["gate"], t["next_weight"], norms,
                              scale, eps)
    names = [n for n in ("x", "residual", "gate", "weight", "next_weight")
             if t[n] is not None]
    assert len(got) == len(names)
    step = 1e-5
    for name, (d, _) in zip(names, got):
        for i in range(d.numel()):
            e = torch.zeros(d.numel(), dtype=torch.float64)
            e[i] = step
            up, down = (dict(t, **{name: t[name] + s * e.view_as(t[name])})
                        for s in (1, -1))
            want = (loss(up) - loss(down)) / (2 * step)
            assert float(d.flatten()[i]) == pytest.approx(want, abs=1e-7)


@pytest.mark.parametrize("change", [
    dict(offsets=2 * A), dict(offsets=10 * A), dict(slots=3 * A),
    dict(positions=4 * A), dict(positions=7 * A), dict(new_lengths=5 * A),
    dict(new_free_count=A), dict(table=4 * A), dict(table=6 * A)], ids=str)
def test_extend_refuses_outputs_that_are_inputs(change):
    refused(INV, mt.mt_cache_extend, changed(EXTEND, **change), None)


@pytest.mark.parametrize("change", [
    dict(out=ATTENTION.q), dict(cap=1e-40), dict(cap=1e-3, scale=1e38)],
    ids=str)
def test_attention_refuses_more(change):
    c = changed(ATTENTION, **change)
    refused(INV, mt.mt_cache_attention, BF16, c, A, 1 << 30, None)

"""Edges of the operators around a decoder's cache without a GPU: what their C
calls allow and few callers use."""
import ctypes
import os
import re
import subprocess

import pytest

import row_reduction_gb300 as mt
from test_step_choices_host import fake  # noqa: F401
from test_step_host import A, ATTENTION, BACK, built, changed  # noqa: F401

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

RULES = r"""
#include "mt_decoder_internal.h"
extern "C" int plain(const mt_block_norm_back_t *c) {
    return mt::gate_plain(*c);
}
"""


@pytest.fixture(scope="module")
def rules(tmp_path_factory):
    """The rules that the host goes by, built with the host compiler."""
    d = tmp_path_factory.mktemp("rules")
    (d / "rules.cpp").write_text(RULES)
    cuda = next(p for p in (os.environ.get("CUDA_HOME"), "/usr/local/cuda")
                if p and os.path.exists(os.path.join(p, "include")))
    subprocess.run(["g++", "-std=c++17", "-O1", "-shared", "-fPIC", "-I",
                    os.path.join(ROOT, "row_reduction_gb300", "csrc"), "-I",
                    os.path.join(cuda, "include"), str(d / "rules.cpp"), "-o",
                    str(d / "rules.so")], check=True)
    return ctypes.CDLL(str(d / "rules.so"))


# ---- norms around a block ----------------------------------------------------
@pytest.mark.parametrize("change,plain", [
    # x is there, or no gate is
    (dict(), True), (dict(dgate_sum=None), True),
    (dict(gate=None, dgate_sum=None), True),
    (dict(gate=None, dgate_sum=None, x=None), True),
    (dict(gate_stride=64, dgate=13 * A, dgate_sum=None), True),
    (dict(gate_stride=64, dgate_sum=None, rows=1), True),
    # a gate matrix without its gradient
    (dict(gate_stride=64, dgate_sum=None), False),
    # a gate, of which nothing is asked that would need x, and no x: the
    # kernels that bring rows ahead would read it
    (dict(dgate_sum=None, x=None), False),
    (dict(dgate_sum=None, x=None, rows=1), False),
    (dict(dgate_sum=None, x=None, gate_stride=64), False),
    (dict(dgate_sum=None, x=None, gate_stride=64, rows=1), False)], ids=str)
def test_a_gate_without_x_goes_the_general_way(rules, change, plain):
    c = changed(BACK, norms=2, weight=None, dweight=None, **change)
    assert bool(rules.plain(ctypes.byref(c))) == plain


def test_backward_workspace_goes_by_the_rows():
    """A row of partial sums for each CTA at most, and for each row at most: a
    call of few wide rows asks for little."""
    def need(**kw):
        return mt.mt_block_norm_backward_workspace(
            0, changed(BACK, **{**dict(dy_stride=1 << 20, dh_stride=1 << 20,
                                       x_stride=1 << 20, h_stride=1 << 20,
                                       dx_stride=1 << 20,
                                       dresidual_stride=1 << 20), **kw}))
    for cols, most in ((64, 608), (2048, 608), (2049, 304), (16384, 304),
                       (1 << 20, 304)):
        row = 3 * cols * 4
        for rows in (0, 1, 2, 8, 303, 304, 305, 607, 608, 609, 10 ** 6):
            assert need(rows=rows, cols=cols) == min(rows, most) * row


# ---- attention over the cache ------------------------------------------------
def test_more_rows_than_a_launch_takes(fake):  # noqa: F811
    """A warp per row and query head, four to a CTA, 2^31 - 1 CTAs at most."""
    most = 4 * (2 ** 31 - 1)

    def call(dim, rows, heads):
        return changed(ATTENTION, dim=dim, group=dim, q_heads=heads, k_heads=1,
                       rows=rows, q_row=heads * dim, q_head=dim,
                       out_row=heads * dim, out_head=dim)

    def status(c):
        n = ctypes.c_size_t()
        got = fake.mt_cache_attention_workspace(2, ctypes.byref(c),
                                                ctypes.byref(n))
        assert got == fake.mt_cache_attention(
            2, ctypes.byref(c), ctypes.c_void_p(A), ctypes.c_size_t(1 << 50),
            None)
        return got
    assert status(call(8, most // 4, 4)) == 0
    assert status(call(8, most // 1024, 1024)) == 0
    assert status(call(8, most // 1024 + 1, 1024)) == mt.MT_ERR_UNSUPPORTED
    assert status(call(8, 2 ** 31 - 1, 65536)) == mt.MT_ERR_UNSUPPORTED
    assert status(call(64, 2 ** 31 - 1, 65536)) == 0    # matrix kernels


def test_a_warp_comes_together_before_tensor_memory():
    """Loads from tensor memory and stores to it are the whole warp's, and come
    behind code in which its lanes go different ways: each stands right behind
    a __syncwarp().  (Whether lanes were apart cannot be seen from outside.)"""
    csrc = os.path.join(ROOT, "row_reduction_gb300", "csrc")
    found = 0
    for name in sorted(os.listdir(csrc)):
        if not name.endswith((".cu", ".cuh")):
            continue
        with open(os.path.join(csrc, name)) as f:
            text = f.read()
        for m in re.finditer(r"tcgen05\.(ld|st)\.sync", text):
            before = text[:text.rindex("asm volatile", 0, m.start())]
            assert before.rstrip().endswith("__syncwarp();"), (name, m.group())
            found += 1
    assert found == 2

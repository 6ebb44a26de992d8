"""The choices of variants of the operators around a decoder's cache without a
GPU: csrc/step.cpp built with the host compiler against launches that only note
what they were given."""
import ctypes
import os
import subprocess

import pytest

import row_reduction_gb300 as mt
from row_reduction_gb300 import _step as st
from test_step_host import ATTENTION, BACK, NORM, changed

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
INV, OOR = mt.MT_ERR_INVALID_ARGUMENT, mt.MT_ERR_OUT_OF_RESOURCES
F32, F16, BF16 = 0, 1, 2
A = 0x10000000

FAKES = r"""
#include "step.cpp"
static int g_sms = 152, g_which, g_V;
static mt::AttentionPlan g_plan;
extern "C" {
void fake_sms(int n) { g_sms = n; }
void fake_last(int *o) {
    const int v[] = {g_which, g_V, g_plan.nt, g_plan.times, g_plan.per,
                     g_plan.parts, g_plan.heads, g_plan.whole, g_plan.ctas};
    for (int i = 0; i < 9; ++i) o[i] = v[i];
}
cudaError_t cudaMemsetAsync(void *, int, size_t, cudaStream_t) {
    return cudaSuccess;
}
}
namespace mt {
mt_status status_from_cuda(cudaError_t e) {
    return e == cudaSuccess ? MT_OK : MT_ERR_CUDA;
}
cudaError_t current_sm_count(int *n) { *n = g_sms; return cudaSuccess; }
cudaError_t launch_cache_extend(const mt_cache_extend_call_t &, cudaStream_t) {
    g_which = 1;
    return cudaSuccess;
}
cudaError_t launch_attention_any(int, const mt_attention_call_t &,
                                 cudaStream_t) {
    g_which = 2;
    return cudaSuccess;
}
#define FAKE(name, n)                                                         \
    cudaError_t name(const AttentionPlan &p, const mt_attention_call_t &,     \
                     int, void *, cudaStream_t) {                             \
        g_which = n; g_plan = p;                                              \
        return cudaSuccess;                                                   \
    }
FAKE(launch_attention_e4m3_p1n1, 111) FAKE(launch_attention_e4m3_p1n2, 112)
FAKE(launch_attention_e4m3_p2n1, 121) FAKE(launch_attention_e4m3_p2n2, 122)
FAKE(launch_attention_int8_p1n1, 211) FAKE(launch_attention_int8_p1n2, 212)
FAKE(launch_attention_int8_p2n1, 221) FAKE(launch_attention_int8_p2n2, 222)
FAKE(launch_attention_rows_e4m3_p1, 110) FAKE(launch_attention_rows_e4m3_p2, 120)
FAKE(launch_attention_rows_int8_p1, 210) FAKE(launch_attention_rows_int8_p2, 220)
FAKE(launch_attention_tiles_e4m3, 109) FAKE(launch_attention_tiles_int8, 209)
#define FAKE_NORM(dt)                                                         \
    cudaError_t launch_block_norm_##dt(const mt_block_norm_call_t &, int V,   \
                                       cudaStream_t) {                        \
        g_which = 3; g_V = V;                                                 \
        return cudaSuccess;                                                   \
    }                                                                         \
    cudaError_t launch_block_norm_back_##dt(const mt_block_norm_back_t &,     \
                                            int V, float *, int *blocks,      \
                                            cudaStream_t) {                   \
        g_which = 4; g_V = V; *blocks = 1;                                    \
        return cudaSuccess;                                                   \
    }
FAKE_NORM(f32)
FAKE_NORM(f16)
FAKE_NORM(bf16)
cudaError_t launch_norm_sums(const float *, int, int, float *, float *,
                             float *, cudaStream_t) {
    return cudaSuccess;
}
}  // namespace mt
"""
NAMES = ("which", "V", "nt", "times", "per", "parts", "heads", "whole",
         "ctas")


@pytest.fixture(scope="module")
def fake(tmp_path_factory):
    d = tmp_path_factory.mktemp("fake")
    (d / "fake.cpp").write_text(FAKES)
    cuda = next(p for p in (os.environ.get("CUDA_HOME"), "/usr/local/cuda")
                if p and os.path.exists(os.path.join(p, "include")))
    subprocess.run(["g++", "-std=c++17", "-O1", "-shared", "-fPIC", "-I",
                    os.path.join(ROOT, "row_reduction_gb300", "csrc"), "-I",
                    os.path.join(cuda, "include"), str(d / "fake.cpp"), "-o",
                    str(d / "fake.so")], check=True)
    return ctypes.CDLL(str(d / "fake.so"))


def last(fake):
    out = (ctypes.c_int * 9)()
    fake.fake_last(out)
    return dict(zip(NAMES, out))


def attend(fake, dtype, call, room=1 << 40):
    size, P = ctypes.c_size_t, ctypes.c_void_p
    n = size()
    assert fake.mt_cache_attention_workspace(
        ctypes.c_int(dtype), ctypes.byref(call), ctypes.byref(n)) == 0
    status = fake.mt_cache_attention(
        ctypes.c_int(dtype), ctypes.byref(call), P(A),
        size(min(room, n.value)), None)
    return status, n.value, last(fake)


@pytest.mark.parametrize("dim,groups,takes", [
    (64, 1, True), (64, 2, True), (64, 4, False), (80, 1, True),
    (80, 5, False), (96, 1, True), (96, 3, False), (128, 1, True),
    (128, 2, True), (128, 4, True), (128, 8, False), (256, 1, True),
    (256, 2, True), (256, 4, False), (256, 8, True), (32, 1, False),
    (512, 1, False), (7, 1, False)])
@pytest.mark.parametrize("dtype", [F32, F16, BF16])
@pytest.mark.parametrize("fmt", [0, 1])
def test_attention_heads(fake, dim, groups, takes, dtype, fmt):
    c = changed(ATTENTION, dim=dim, group=dim // groups, format=fmt, rows=2,
                q_row=4 * dim, q_head=dim, out_row=4 * dim, out_head=dim)
    status, size, got = attend(fake, dtype, c)
    assert status == 0
    if not takes:
        assert got["which"] == 2 and size == 0
        return
    parts = 1 if dtype == BF16 else 2
    assert got["which"] == 100 * (fmt + 1) + 10 * parts + 1
    assert got["heads"] == 2 and got["times"] == 2 and got["per"] == 4
    assert got["ctas"] in (2 * 152, 3 * 152)
    assert size == got["ctas"] * (2 * 32 * (dim + 2) * 4 + 24)
    assert attend(fake, dtype, c, size - 1)[0] == OOR


@pytest.mark.parametrize("q_heads,k_heads,rows,sequences,nt,per,parts,heads", [
    (8, 8, 10, 10, 1, 8, 1, 4),        # one column per sequence
    (32, 8, 64, 64, 1, 2, 1, 4), (32, 4, 64, 64, 1, 1, 1, 4),
    (32, 8, 192, 64, 2, 4, 1, 4), (9, 1, 5, 5, 2, 1, 1, 1),
    (24, 1, 5, 5, 2, 1, 2, 1), (10, 5, 5, 5, 1, 4, 1, 1),
    (12, 6, 6, 6, 1, 4, 1, 2), (32, 8, 11, 1, 2, 4, 1, 4),
    (32, 8, 12, 1, 0, 16, 1, 1), (80, 1, 1, 1, 0, 1, 2, 1),
    (15, 3, 500, 50, 0, 12, 1, 1)])
def test_attention_tiles(fake, q_heads, k_heads, rows, sequences, nt, per,
                         parts, heads):
    c = changed(ATTENTION, q_heads=q_heads, k_heads=k_heads, rows=rows,
                sequences=sequences, q_row=q_heads * 128,
                out_row=q_heads * 128, group=128)
    status, size, got = attend(fake, BF16, c)
    assert status == 0
    assert {k: got[k] for k in ("nt", "per", "parts", "heads")} == dict(
        nt=nt, per=per, parts=parts, heads=heads)
    assert got["which"] == 110 + nt
    columns = 32 * nt if nt else 64
    assert size == got["ctas"] * (2 * columns * 130 * 4 + 24)
    # every query head and row has a column, none has two
    width = 8 * nt if nt else 64
    times = q_heads // k_heads
    assert per * min(times, width) <= width and parts * width >= times
    assert k_heads % heads == 0


def test_attention_any_addresses_and_sizes(fake):
    """What the matrix kernels do not take goes the general way."""
    for kw in (dict(k_codes=4 * A + 16), dict(v_codes=5 * A + 4),
               dict(k_scales=6 * A + 4), dict(v_scales=7 * A + 8),
               dict(slots=2 ** 31), dict(slots=0), dict(pages=0)):
        status, size, got = attend(fake, BF16, changed(ATTENTION, **kw))
        assert (status, size, got["which"]) == (0, 0, 2), kw
    # four values at a time where addresses and strides allow it
    for kw, whole in ((dict(), 3), (dict(q=A + 4), 2), (dict(out=2 * A + 2), 1),
                      (dict(q_row=514), 2), (dict(out_head=131, out_row=1000),
                                             1)):
        assert attend(fake, BF16, changed(ATTENTION, **kw))[2]["whole"] == \
            whole, kw


@pytest.mark.parametrize("sms", [1, 20, 132, 152, 160])
def test_attention_ctas_go_by_the_device(fake, sms):
    fake.fake_sms(sms)
    _, size, got = attend(fake, BF16, ATTENTION)
    fake.fake_sms(152)
    assert got["ctas"] == 2 * sms
    assert size == 2 * sms * (2 * 32 * 130 * 4 + 24)


@pytest.mark.parametrize("es,dtype", [(4, F32), (2, F16), (2, BF16)])
def test_norms_take_the_widest_packs(fake, es, dtype):
    full = 16 // es

    def forward(**kw):
        c = changed(NORM, **kw)
        assert fake.mt_block_norm(ctypes.c_int(dtype), ctypes.byref(c),
                                  None) == 0
        return last(fake)["V"]

    def back(**kw):
        c = changed(BACK, **kw)
        assert fake.mt_block_norm_backward(
            ctypes.c_int(dtype), ctypes.byref(c), ctypes.c_void_p(A),
            ctypes.c_size_t(1 << 40), None) == 0
        return last(fake)["V"]
    assert forward() == full and back() == full
    for name in ("x", "residual", "gate", "weight", "next_weight", "h", "y"):
        base = getattr(NORM, name)
        for off in (1, 2, 4):
            assert forward(**{name: base + off * es}) == min(off, full)
    for name in ("dy", "dh", "x", "h", "gate", "weight", "next_weight", "dx",
                 "dresidual"):
        base = getattr(BACK, name)
        assert back(**{name: base + es}) == 1
    assert forward(cols=62) == 2 and forward(cols=61) == 1
    assert back(cols=60) == 4 and back(cols=61) == 1
    assert forward(x_stride=66) == 2 and back(dx_stride=65) == 1
    assert forward(rows=1, x_stride=65) == full


@pytest.mark.parametrize("q_heads,k_heads,rows,sequences,dim,group,dtype,takes", [
    (32, 8, 64, 1, 128, 128, BF16, True), (32, 8, 63, 1, 128, 128, BF16, False),
    (32, 8, 128, 2, 64, 64, BF16, True), (32, 8, 127, 2, 64, 64, BF16, False),
    (32, 8, 1000, 1, 128, 64, BF16, False), (32, 8, 1000, 1, 96, 96, BF16, False),
    (32, 8, 1000, 1, 256, 256, BF16, False), (32, 8, 1000, 1, 128, 128, F16, False),
    (32, 8, 1000, 1, 128, 128, F32, False), (390, 2, 7, 1, 128, 128, BF16, True),
    (8, 8, 256, 1, 128, 128, BF16, True)])
@pytest.mark.parametrize("fmt", [0, 1])
def test_attention_on_tensor_memory(fake, q_heads, k_heads, rows, sequences, dim,
                                    group, dtype, takes, fmt):
    c = changed(ATTENTION, q_heads=q_heads, k_heads=k_heads, rows=rows,
                sequences=sequences, q_row=q_heads * dim, q_head=dim,
                out_row=q_heads * dim, out_head=dim, dim=dim, group=group,
                format=fmt)
    status, size, got = attend(fake, dtype, c)
    assert status == 0
    assert (got["which"] == 100 * (fmt + 1) + 9) == takes
    if not takes:
        assert got["nt"] >= 0
        return
    times = q_heads // k_heads
    assert got["nt"] == -1 and got["heads"] == 1 and got["ctas"] == 2 * 152
    assert size == got["ctas"] * (2 * 128 * (dim + 2) * 4 + 24)
    assert got["per"] * min(times, 128) <= 128
    assert got["parts"] * 128 >= times
    assert attend(fake, dtype, c, size - 1)[0] == OOR

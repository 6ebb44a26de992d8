"""The limits and the choices of variants of the decoder's row operators
without a GPU: csrc/decoder.cpp built with the host compiler against CUDA and
kernel launches that only note what they were given."""
import ctypes
import os
import subprocess

import pytest

import row_reduction_gb300 as mt
from row_reduction_gb300 import _decoder as dec

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
INV, UNS = mt.MT_ERR_INVALID_ARGUMENT, mt.MT_ERR_UNSUPPORTED
F32, F16, BF16 = 0, 1, 2
A = 0x10000000  # an address that nothing looks at

FAKES = r"""
#include "decoder.cpp"

static int g_dev, g_dev_sms[64], g_vec, g_V, g_K, g_launches;
static mt::RotArgs g_rot;
extern "C" {
cudaError_t cudaGetDevice(int *d) { *d = g_dev; return cudaSuccess; }
cudaError_t cudaDeviceGetAttribute(int *v, enum cudaDeviceAttr, int d) {
    *v = g_dev_sms[d];
    return cudaSuccess;
}
cudaError_t cudaFuncSetAttribute(const void *, enum cudaFuncAttribute, int) {
    return cudaSuccess;
}
cudaError_t cudaMemsetAsync(void *, int, size_t, cudaStream_t) {
    return cudaSuccess;
}
void fake_device(int sms) {  // a device of its own for each size
    g_dev = sms / 4;
    g_dev_sms[g_dev] = sms;
}
int fake_launches() { return g_launches; }
void fake_last(int *o) {
    const int v[] = {g_vec, g_V, g_K, g_rot.log2S, g_rot.blocks[0],
                     g_rot.blocks[1], g_rot.threads, g_rot.t[0].groups,
                     g_rot.t[1].groups};
    for (int i = 0; i < 9; ++i) o[i] = v[i];
}
}
namespace mt {
mt_status status_from_cuda(cudaError_t e) {
    return e == cudaSuccess ? MT_OK : MT_ERR_CUDA;
}
#define FAKE_TYPE(dt)                                                         \
    cudaError_t launch_rotary_##dt(const RotArgs &a, int V, int K, bool,      \
                                   bool, cudaStream_t) {                      \
        g_rot = a; g_V = V; g_K = K; ++g_launches;                            \
        return cudaSuccess;                                                   \
    }                                                                         \
    cudaError_t launch_rotary_backward_##dt(const RotArgs &a, int V, int K,   \
                                            bool, cudaStream_t) {             \
        g_rot = a; g_V = V; g_K = K; ++g_launches;                            \
        return cudaSuccess;                                                   \
    }                                                                         \
    cudaError_t launch_logits_##dt(const mt_logits_call_t &, cudaStream_t) {  \
        ++g_launches;                                                         \
        return cudaSuccess;                                                   \
    }
FAKE_TYPE(f32)
FAKE_TYPE(f16)
FAKE_TYPE(bf16)
cudaError_t launch_rotary_dweight(const float *, int, const int32_t[2],
                                  float *, float *, cudaStream_t) {
    return cudaSuccess;
}
cudaError_t launch_cache_write(int, const CacheArgs &, int vec, cudaStream_t) {
    g_vec = vec; ++g_launches;
    return cudaSuccess;
}
cudaError_t launch_cache_read(int, const CacheArgs &, int vec, cudaStream_t) {
    g_vec = vec; ++g_launches;
    return cudaSuccess;
}
cudaError_t launch_cache_slots(const int32_t *, int64_t, int32_t,
                               const int32_t *, const int32_t *, int32_t,
                               int32_t, int64_t, int64_t *, cudaStream_t) {
    ++g_launches;
    return cudaSuccess;
}
}  // namespace mt
"""


class Fake:
    """The entry points, and what their last launch was given."""

    def __init__(self, path):
        self.lib = ctypes.CDLL(str(path))
        P, I, L = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64
        for name, args in {
                "mt_rotary": [I, P, P],
                "mt_rotary_backward": [I, P, P, ctypes.c_size_t, P],
                "mt_cache_write": [I, P, P], "mt_cache_read": [I, P, P],
                "mt_process_logits": [I, P, P],
                "mt_cache_slots": [P, L, I, P, P, I, I, L, P, P],
                "mt_rotary_turns": [P, I, P]}.items():
            getattr(self.lib, name).argtypes = args
        self.lib.fake_device(152)

    def __getattr__(self, name):
        def run(dtype, call, *rest):
            return getattr(self.lib, "mt_" + name)(
                dtype, ctypes.byref(call), *rest, None)
        return run

    def last(self):
        out = (ctypes.c_int32 * 9)()
        self.lib.fake_last(out)
        return dict(zip(("vec", "V", "K", "log2S", "q_blocks", "k_blocks",
                         "threads", "q_groups", "k_groups"), out))


@pytest.fixture(scope="module")
def fake(tmp_path_factory):
    d = tmp_path_factory.mktemp("choices")
    (d / "fakes.cpp").write_text(FAKES)
    cuda = os.environ.get("CUDA_HOME", "/usr/local/cuda")
    subprocess.run(
        ["g++", "-std=c++17", "-O1", "-shared", "-fPIC",
         "-Wl,-Bsymbolic", "-I",  # the fakes, not a loaded CUDA runtime
         os.path.join(cuda, "include"), "-I",
         os.path.join(ROOT, "row_reduction_gb300", "csrc"),
         str(d / "fakes.cpp"), "-o", str(d / "fakes.so")], check=True)
    return Fake(d / "fakes.so")


def heads(n, dim, x=A, **kw):
    return dec.MtRotaryHeads(x=x, y=A, heads=n, x_token=n * dim, x_head=dim,
                             dy_token=n * dim, dy_head=dim, y_token=n * dim,
                             y_head=dim, **kw)


def rotary(tokens, hq, hk, dim=128, norm=0, back=False):
    kw = dict(dy=A) if back else {}
    x = A if norm or not back else None
    return dec.MtRotaryCall(q=heads(hq, dim, x, **kw),
                            k=heads(hk, dim, x, **kw), positions=A, turns=A,
                            tokens=tokens, position_bytes=8, dim=dim,
                            rotary_dim=dim, norm=norm, scale=1.0)


def cache(tokens, heads_, dim, group, rows=A, codes=A):
    r = dec.MtCacheRows(codes=codes, scales=A, rows=rows,
                        token_stride=heads_ * dim, head_stride=dim)
    return dec.MtCacheCall(k=r, slot=A, tokens=tokens, slots=64,
                           heads=heads_, dim=dim, group=group, format=0)


# ---- limits, as the header states them -------------------------------------------
def test_rotary_limits(fake):
    for f, back in ((fake.rotary, False),
                    (lambda t, c: fake.rotary_backward(t, c, None, 0), True)):
        assert f(BF16, rotary(2, 65536, 1, back=back)) == 0
        assert f(BF16, rotary(2, 65537, 1, back=back)) == UNS
        assert f(BF16, rotary(2 ** 33, 1, 1, back=back)) == 0
        assert f(BF16, rotary(2 ** 33 + 1, 1, 1, back=back)) == UNS


def test_turns_limit(fake):
    for f, want in ((999999.0, 0), (-999999.0, 0), (1e6, INV), (-1e6, INV),
                    (float("nan"), INV)):
        turns = ctypes.c_uint64()
        assert fake.lib.mt_rotary_turns(ctypes.byref(ctypes.c_double(f)), 1,
                                        ctypes.byref(turns)) == want


def test_logits_and_slots_limits(fake):
    def call(rows):
        return dec.MtLogitsCall(x=A, y=A, rows=rows, x_stride=8, y_stride=8,
                                vocab=8)
    assert fake.process_logits(BF16, call(2 ** 24)) == 0
    assert fake.process_logits(BF16, call(2 ** 24 + 1)) == UNS

    def slots(rows):
        return fake.lib.mt_cache_slots(A, 8, 8, A, A, 3, 16, rows, A, None)
    assert slots(2 ** 38) == 0
    assert slots(2 ** 38 + 1) == UNS


@pytest.mark.parametrize("write", [True, False])
@pytest.mark.parametrize("rows,codes", [(A, A), (A + 2, A), (A, A + 1),
                                        (A + 16, A), (A, A + 8)])
@pytest.mark.parametrize("heads_,dim,group", [
    (8, 128, 128), (8, 128, 8), (1, 1024, 1024), (8, 80, 5), (3, 100, 4)])
def test_cache_limits_do_not_depend_on_addresses(fake, write, rows, codes,
                                                 heads_, dim, group):
    f = fake.cache_write if write else fake.cache_read
    most = 2 ** (40 if group % 8 == 0 else 32) // (heads_ * dim)
    assert f(BF16, cache(most, heads_, dim, group, rows, codes)) == 0
    assert f(BF16, cache(most + 1, heads_, dim, group, rows, codes)) == UNS


@pytest.mark.parametrize("scaling,missing", [
    (dict(type="linear"), "factor"), (dict(type="ntk"), "factor"),
    (dict(type="yarn", original_length=100), "factor"),
    (dict(type="bands", factor=2.0), "original_length"),
    (dict(type="yarn", factor=2.0), "original_length")])
def test_scalings_say_what_they_need(scaling, missing):
    with pytest.raises(ValueError, match=missing):
        mt.rotary_frequencies(8, scaling=scaling, device="cpu")


# ---- choices by the device's size --------------------------------------------------
@pytest.mark.parametrize("sms", [20, 76, 132, 148, 152, 160])
@pytest.mark.parametrize("dtype", [F32, F16, BF16])
@pytest.mark.parametrize("hq,hk", [(32, 8), (8, 1), (1, 0), (20, 5), (64, 1)])
def test_backward_takes_the_blocks_that_are_resident(fake, sms, dtype, hq, hk):
    """Equal shares of the work for two blocks per SM: one more would run
    alone after the rest.  304 rows of partial sums at most."""
    fake.lib.fake_device(sms)
    most = min(304, 2 * sms)
    for tokens in (1, 7, 300, 4096, 100003):
        c = rotary(tokens, hq, hk, norm=1, back=True)
        assert fake.rotary_backward(dtype, c, None, 0) == 0
        got = fake.last()
        warps = got["threads"] // 32
        q, k = got["q_blocks"], got["k_blocks"]
        assert 1 <= q and (k >= 1) == (hk > 0) and q + k <= most
        for blocks, groups in ((q, got["q_groups"]), (k, got["k_groups"])):
            assert blocks <= -(-tokens * groups // warps)
        if tokens >= 4096:
            assert q + k >= most - 1
    fake.lib.fake_device(152)


def test_backward_shares_never_exceed_the_blocks(fake):
    """Any numbers of groups: the two tensors' parts, rounded down but at least
    one each, fit the rows of partial sums."""
    for sms in (8, 28, 148, 152):
        fake.lib.fake_device(sms)
        most = min(304, 2 * sms)
        for hq in [*range(1, 70), 400, 9001, 65536]:
            for hk in [*range(0, 70, 3), 1000, 65536]:
                c = rotary(10 ** 6, hq, hk, dim=256, norm=1, back=True)
                assert fake.rotary_backward(F32, c, None, 0) == 0
                got = fake.last()
                assert got["q_blocks"] + got["k_blocks"] <= most
    fake.lib.fake_device(152)


@pytest.mark.parametrize("sms", [76, 148, 152])
def test_forward_splits_a_token_until_the_device_is_full(fake, sms):
    """Warps per token: one more doubling while 16 per SM are not reached (a
    last one, to ask for all heads at once, may follow)."""
    fake.lib.fake_device(sms)
    for tokens in (1, 8, 100, 1000, sms * 16 - 1, sms * 16, 100000):
        for norm in (0, 1):
            assert fake.rotary(F32, rotary(tokens, 32, 8, norm=norm)) == 0
            got = fake.last()
            split, groups = 1 << got["log2S"], got["q_groups"] + got["k_groups"]
            assert split >= groups or tokens * split >= sms * 16
            assert split == 1 or tokens * split // 4 < sms * 16 or not norm
            if tokens >= sms * 24:
                assert split == 1 or not norm
    fake.lib.fake_device(152)

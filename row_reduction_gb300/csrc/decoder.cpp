// decoder.cpp -- C entry points of the decoder's row operators: argument
// checks, choice of kernel variants, frequencies of rotary positions.
#include <math.h>
#include <stdint.h>

#include <atomic>
#include <mutex>
#include <unordered_set>

#include "mt_decoder_internal.h"

namespace mt {

namespace {
constexpr int kMaxDevices = 64;
std::atomic<int> g_sms[kMaxDevices];
std::mutex g_smem_mu;
std::unordered_set<uint64_t> g_smem;
}  // namespace

cudaError_t current_sm_count(int *out) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const bool known = dev >= 0 && dev < kMaxDevices;
    int v = known ? g_sms[dev].load(std::memory_order_relaxed) : 0;
    if (v == 0) {
        e = cudaDeviceGetAttribute(&v, cudaDevAttrMultiProcessorCount, dev);
        if (e != cudaSuccess) return e;
        if (known) g_sms[dev].store(v, std::memory_order_relaxed);
    }
    *out = v;
    return cudaSuccess;
}

cudaError_t allow_max_smem(const void *kernel) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const uint64_t key = (reinterpret_cast<uintptr_t>(kernel) << 8) ^
                         (uint64_t)(dev & 0xff);
    try {
        std::lock_guard<std::mutex> lk(g_smem_mu);
        if (g_smem.count(key)) return cudaSuccess;
        e = cudaFuncSetAttribute(kernel,
                                 cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 kDecoderSmemBytes);
        if (e == cudaSuccess) g_smem.insert(key);
    } catch (...) {
        return cudaErrorMemoryAllocation;
    }
    return e;
}

namespace {

bool misaligned(const void *p, int bytes) {
    return (reinterpret_cast<uintptr_t>(p) & (uintptr_t)(bytes - 1)) != 0;
}
bool known_dtype(int dt) { return dt >= 0 && dt < DT_COUNT; }

// Element offsets stay below this: twice the byte size of the widest type
// still fits an int64.
constexpr int64_t kMaxOffset = INT64_MAX / 16;

// |a| * b <= kMaxOffset for b >= 0 (adds to *sum, which must stay so too).
bool add_extent(int64_t stride, int64_t n, int64_t *sum) {
    if (n <= 1 || stride == 0) return true;
    if (stride == INT64_MIN) return false;
    const int64_t a = stride < 0 ? -stride : stride;
    if (a > (kMaxOffset - *sum) / (n - 1)) return false;
    *sum += a * (n - 1);
    return true;
}
bool reachable(int64_t ts, int64_t hs, int64_t tokens, int64_t heads) {
    int64_t sum = 1024;
    return add_extent(ts, tokens, &sum) && add_extent(hs, heads, &sum);
}
// Rows of an output (tokens x heads rows of dim values) do not overlap: the
// smaller stride steps over a row, the larger one over all rows of the
// other.
bool disjoint(int64_t ts, int64_t hs, int64_t tokens, int64_t heads,
              int64_t dim) {
    const int64_t t = ts < 0 ? -ts : ts, h = hs < 0 ? -hs : hs;
    if (tokens > 1 && t < dim) return false;
    if (heads > 1 && h < dim) return false;
    if (tokens > 1 && heads > 1)
        return t <= h ? h >= t * (tokens - 1) + dim
                      : t >= h * (heads - 1) + dim;
    return true;
}

// Largest V in {full, ..., 2, 1} whose packs of V*es bytes fit every listed
// address, stride and offset (all in `bits`, OR-ed together, in elements for
// strides and offsets and in bytes/es for addresses).
int widest(uint64_t bits, int full) {
    int v = full;
    while (v > 1 && (bits & (uint64_t)(v - 1))) v >>= 1;
    return v;
}

// ---- rotary ----------------------------------------------------------------
enum RotKind { ROT_FORWARD, ROT_BACKWARD };

// Slots and groups of heads at V values per pack; K is returned: one slot per
// lane, or (heads wider than a warp's slots) as many as the widest head needs
// at this V.
int rotary_layout(RotArgs *a, int V) {
    const int rest = a->dim - 2 * a->pairs;
    a->rot_slots = a->pairs / V;
    a->slots = a->rot_slots + (rest + 2 * V - 1) / (2 * V);
    a->log2L = 0;
    while (a->log2L < 5 && (1 << a->log2L) < a->slots) ++a->log2L;
    for (int i = 0; i < 2; ++i)
        a->t[i].groups =
            (int32_t)(((int64_t)a->t[i].heads + (32 >> a->log2L) - 1) >>
                      (5 - a->log2L));
    return a->slots <= 32 ? 1 : kRotMaxDim / (64 * V);
}

// Common checks; fills `a`, V and K.  With nothing to do, *empty.
mt_status rotary_setup(int dtype, const mt_rotary_call_t *c, RotKind kind,
                       RotArgs *a, int *V, int *K, bool *empty) {
    if (c == nullptr || !known_dtype(dtype)) return MT_ERR_INVALID_ARGUMENT;
    const int es = dtype_size(dtype);
    if (c->tokens < 0 || c->dim < 1 || c->rotary_dim < 2 ||
        c->rotary_dim > c->dim || (c->rotary_dim & 1) ||
        (c->interleaved & ~1) || (c->norm & ~1) || c->reserved != 0 ||
        (c->position_bytes != 4 && c->position_bytes != 8))
        return MT_ERR_INVALID_ARGUMENT;
    if (c->dim > kRotMaxDim) return MT_ERR_UNSUPPORTED;
    if (c->norm && !(c->eps >= 0.f)) return MT_ERR_INVALID_ARGUMENT;
    const bool back = kind == ROT_BACKWARD;
    *empty = c->tokens == 0 || (c->q.heads == 0 && c->k.heads == 0);
    // Both layouts hold V whole pairs in two packs of V values; the values
    // that pass come in such double packs too (an odd head: one by one).
    const int rest = c->dim - c->rotary_dim;
    uint64_t bits = (uint64_t)(c->rotary_dim / 2) |
                    (uint64_t)(rest & 1 ? 1 : rest / 2);
    const mt_rotary_heads_t *hs[2] = {&c->q, &c->k};
    for (int i = 0; i < 2; ++i) {
        const mt_rotary_heads_t &h = *hs[i];
        if (h.heads < 0 || h.reserved != 0) return MT_ERR_INVALID_ARGUMENT;
        // pointers that the call does not take
        if ((!back && (h.dy || h.dweight)) || (!c->norm && h.weight) ||
            (back && !c->norm && (h.x || h.dweight)))
            return MT_ERR_INVALID_ARGUMENT;
        if (misaligned(h.x, es) || misaligned(h.dy, es) ||
            misaligned(h.y, es) || misaligned(h.weight, es) ||
            misaligned(h.dweight, 4))
            return MT_ERR_INVALID_ARGUMENT;
        if (h.heads == 0 || c->tokens == 0) continue;
        const bool x = !back || c->norm;
        if ((x && !h.x) || (back && !h.dy) || !h.y)
            return MT_ERR_INVALID_ARGUMENT;
        if (h.heads > 65536) return MT_ERR_UNSUPPORTED;
        if ((x && !reachable(h.x_token, h.x_head, c->tokens, h.heads)) ||
            (back && !reachable(h.dy_token, h.dy_head, c->tokens, h.heads)) ||
            !reachable(h.y_token, h.y_head, c->tokens, h.heads) ||
            !disjoint(h.y_token, h.y_head, c->tokens, h.heads, c->dim))
            return MT_ERR_INVALID_ARGUMENT;
        auto add = [&](const void *p, int64_t ts, int64_t hs_) {
            bits |= (uint64_t)(reinterpret_cast<uintptr_t>(p) / es);
            if (c->tokens > 1) bits |= (uint64_t)ts;
            if (h.heads > 1) bits |= (uint64_t)hs_;
        };
        if (x) add(h.x, h.x_token, h.x_head);
        if (back) add(h.dy, h.dy_token, h.dy_head);
        add(h.y, h.y_token, h.y_head);
        add(h.weight, 0, 0);
    }
    if (*empty) return MT_OK;
    if (c->positions == nullptr || c->turns == nullptr ||
        misaligned(c->positions, c->position_bytes) || misaligned(c->turns, 8))
        return MT_ERR_INVALID_ARGUMENT;

    *V = widest(bits, 16 / es);
    for (int i = 0; i < 2; ++i) {
        const mt_rotary_heads_t &h = *hs[i];
        RotHeads &r = a->t[i];
        r.x = h.x;
        r.dy = h.dy;
        r.y = h.y;
        r.w = h.weight;
        r.xt = h.x_token;
        r.xh = h.x_head;
        r.dt = h.dy_token;
        r.dh = h.dy_head;
        r.yt = h.y_token;
        r.yh = h.y_head;
        r.heads = h.heads;
    }
    a->pos = c->positions;
    a->pos64 = c->position_bytes == 8;
    a->turns = c->turns;
    a->tokens = c->tokens;
    a->dim = c->dim;
    a->pairs = c->rotary_dim / 2;
    *K = rotary_layout(a, *V);
    a->eps = c->eps;
    a->inv_dim = 1.f / (float)c->dim;
    a->scale = c->scale;
    a->sign = back ? -1.f : 1.f;
    return MT_OK;
}

// Warps per token (a power of two): one while the tokens fill the device,
// more where there are few, up to one group of heads each.
int split_log2(int64_t tokens, int groups, int sms) {
    int l = 0;
    while ((1 << l) < groups && (tokens << l) < (int64_t)sms * 16) ++l;
    return l;
}

// Whether a warp of the forward rotation, with one slot per lane, asks for all
// its groups at once.
bool rotary_at_once(const RotArgs &a) {
    return rotary_fits(a, 2, 2) || rotary_fits(a, 3, 1);
}

// Twice the warps where each then asks for all its groups at once: without
// norm they only turn the angles twice (BF16, 57359 tokens of 15 + 3 heads of
// 64: 47 us for 52; FP32, 16049 of 10 + 2 of 96: 26 for 32, 700 of 32 + 8 of
// 128: 4.2 for 5.1); with it, where they still fit the device at once
// (1237 of 15 + 5 of 80: 4.5 for 5.9; many tokens 69 for 62).  Not with eight
// angles to a lane (30000 of 5 + 5 of 160, interleaved: 51 for 46).
void rotary_split(RotArgs *a, int V, int K, bool norm, int sms) {
    a->log2S = split_log2(a->tokens, a->t[0].groups + a->t[1].groups, sms);
    if (K != 1 || V == 8 || rotary_at_once(*a) ||
        a->tokens << a->log2S >= (norm ? sms * 24 : 1 << 30))
        return;
    RotArgs b = *a;
    ++b.log2S;
    if (rotary_at_once(b)) *a = b;
}

cudaError_t rotary_launch(int dtype, const RotArgs &a, int V, int K, bool ilv,
                          bool norm, cudaStream_t s) {
    switch (dtype) {
        case DT_F32: return launch_rotary_f32(a, V, K, ilv, norm, s);
        case DT_F16: return launch_rotary_f16(a, V, K, ilv, norm, s);
        default: return launch_rotary_bf16(a, V, K, ilv, norm, s);
    }
}

// 16-bit values go in packs of 16 bytes, of which each lane's eight angles
// and coefficients serve many heads, or of 8 bytes: twice the groups, but
// half the angles and 80 registers for 122.  The latter where a warp then
// still asks for all its groups at once (BF16 with norm: 57359 tokens of 4 + 1
// heads of 64 32 us for 54, 40000 of 3 + 1 of 128 27 for 42, 8 of 32 + 8 of
// 128 1.6 for 2.0), or where there is no norm's sum to add over twice the
// lanes (40000 of 16 + 4 of 128: 95 us for 86 with it, 64 for 69 without, and
// 16384 of 32 + 8 of 128 51 us either way).
cudaError_t rotary_forward(int dtype, RotArgs a, int V, int K, bool ilv,
                           bool norm, cudaStream_t s) {
    int sms = 0;
    cudaError_t e = current_sm_count(&sms);
    if (e != cudaSuccess) return e;
    rotary_split(&a, V, K, norm, sms);
    if (V == 8) {
        RotArgs b = a;
        if (rotary_layout(&b, 4) == 1) {
            rotary_split(&b, 4, 1, norm, sms);
            if (rotary_at_once(b) || !norm)
                return rotary_launch(dtype, b, 4, 1, ilv, norm, s);
        }
    }
    return rotary_launch(dtype, a, V, K, ilv, norm, s);
}

// A launch's grid (warps of kRotThreads/32 per CTA) must fit 2^31 - 1.
bool too_many_tokens(int64_t tokens) { return tokens > (1LL << 33); }

size_t backward_workspace(const mt_rotary_call_t *c) {
    return (size_t)kRotBackBlocks * (size_t)c->dim * sizeof(float);
}

// ---- cache -----------------------------------------------------------------
mt_status cache_setup(int dtype, const mt_cache_call_t *c, bool write,
                      CacheArgs *a, int *vec, bool *empty) {
    if (c == nullptr || !known_dtype(dtype)) return MT_ERR_INVALID_ARGUMENT;
    if (c->tokens < 0 || c->slots < 0 || c->heads < 1 || c->dim < 1 ||
        c->group < 1 || c->group > c->dim || c->dim % c->group != 0 ||
        (c->format != MT_CACHE_E4M3 && c->format != MT_CACHE_INT8))
        return MT_ERR_INVALID_ARGUMENT;
    const int64_t width = (int64_t)c->heads * c->dim;
    if (width > (1 << 20)) return MT_ERR_UNSUPPORTED;
    if (c->slots > kMaxOffset / width) return MT_ERR_INVALID_ARGUMENT;
    const int es = dtype_size(dtype);
    const bool both = c->v.codes || c->v.scales || c->v.rows;
    *empty = c->tokens == 0 || c->slots == 0;
    uint64_t bits = 0, code_bits = 0;
    const mt_cache_rows_t *rs[2] = {&c->k, &c->v};
    for (int i = 0; i < (both ? 2 : 1); ++i) {
        const mt_cache_rows_t &r = *rs[i];
        if (misaligned(r.scales, 4) || misaligned(r.rows, es))
            return MT_ERR_INVALID_ARGUMENT;
        if (!*empty && (!r.codes || !r.scales || !r.rows))
            return MT_ERR_INVALID_ARGUMENT;
        if (!reachable(r.token_stride, r.head_stride, c->tokens, c->heads) ||
            (!write && !*empty &&
             !disjoint(r.token_stride, r.head_stride, c->tokens, c->heads,
                       c->dim)))
            return MT_ERR_INVALID_ARGUMENT;
        bits |= (uint64_t)(reinterpret_cast<uintptr_t>(r.rows) / es);
        if (c->tokens > 1) bits |= (uint64_t)r.token_stride;
        if (c->heads > 1) bits |= (uint64_t)r.head_stride;
        code_bits |= (uint64_t)reinterpret_cast<uintptr_t>(r.codes);
        a->codes[i] = static_cast<uint8_t *>(r.codes);
        a->scales[i] = r.scales;
        a->rows[i] = r.rows;
        a->ts[i] = r.token_stride;
        a->hs[i] = r.head_stride;
    }
    if (*empty) return MT_OK;
    if (c->slot == nullptr || misaligned(c->slot, 8))
        return MT_ERR_INVALID_ARGUMENT;
    // Values per lane: 16 where groups hold whole sixteens and the rows'
    // addresses and strides allow 32-byte accesses (64 bytes are two of them
    // for FP32) and the codes 16-byte ones; else 8 with accesses half as
    // wide; else one value at a time.  A warp holds a group when writing.
    *vec = 0;
    for (int v = 16; v >= 8 && *vec == 0; v /= 2)
        if (c->group % v == 0 && (code_bits & (uint64_t)(v - 1)) == 0 &&
            (bits & (uint64_t)(2 * v / es - 1)) == 0 &&
            (!write || c->group <= 32 * v))
            *vec = v;
    a->slot = c->slot;
    a->tokens = c->tokens;
    a->slots = c->slots;
    a->tensors = both ? 2 : 1;
    a->heads = c->heads;
    a->dim = c->dim;
    a->group = c->group;
    a->int8 = c->format == MT_CACHE_INT8;
    // The same at every address, whichever kernel that leads to.
    if (c->tokens > (1LL << (c->group % 8 == 0 ? 40 : 32)) / width)
        return MT_ERR_UNSUPPORTED;
    return MT_OK;
}

}  // namespace
}  // namespace mt

using namespace mt;

extern "C" {

mt_status mt_rotary_frequencies(int32_t rotary_dim, double base,
                                const mt_rotary_scaling_t *scaling,
                                double *freqs, double *factor) {
    const int type = scaling ? scaling->type : (int)MT_ROTARY_PLAIN;
    if (rotary_dim < 2 || rotary_dim > kRotMaxDim || (rotary_dim & 1) ||
        !(base > 1.0) || !isfinite(base) || freqs == nullptr ||
        factor == nullptr || type < MT_ROTARY_PLAIN || type > MT_ROTARY_BANDS)
        return MT_ERR_INVALID_ARGUMENT;
    const double two_pi = 6.283185307179586476925;
    double s = 1.0, length = 0.0, low = 0.0, high = 0.0;
    if (type != MT_ROTARY_PLAIN) {
        s = scaling->factor;
        if (scaling->reserved != 0 || !(s >= 1.0) || !isfinite(s))
            return MT_ERR_INVALID_ARGUMENT;
    }
    if (type == MT_ROTARY_NTK && rotary_dim < 4) return MT_ERR_INVALID_ARGUMENT;
    if (type == MT_ROTARY_YARN || type == MT_ROTARY_BANDS) {
        length = scaling->original_length;
        low = scaling->low;
        high = scaling->high;
        if (!(length > 0.0) || !isfinite(length) || !(low > 0.0) ||
            !(high > low) || !isfinite(high))
            return MT_ERR_INVALID_ARGUMENT;
    }
    const double n = (double)rotary_dim;
    if (type == MT_ROTARY_NTK) base *= pow(s, n / (n - 2.0));
    // YARN: pair index (real) that makes r turns over the original length.
    auto pair_of = [&](double r) {
        return n * log(length / (r * two_pi)) / (2.0 * log(base));
    };
    const double first =
        type == MT_ROTARY_YARN ? fmax(floor(pair_of(high)), 0.0) : 0.0;
    const double last =
        type == MT_ROTARY_YARN ? fmin(ceil(pair_of(low)), n - 1.0) : 0.0;
    for (int i = 0; i < rotary_dim / 2; ++i) {
        double f = pow(base, -2.0 * i / n);
        double keep = 1.0;  // part of the pair that keeps its frequency
        if (type == MT_ROTARY_LINEAR) keep = 0.0;
        if (type == MT_ROTARY_YARN)
            keep = 1.0 - fmin(fmax((i - first) / fmax(last - first, 0.001),
                                   0.0), 1.0);
        if (type == MT_ROTARY_BANDS)
            keep = fmin(fmax((length * f / two_pi - low) / (high - low), 0.0),
                        1.0);
        freqs[i] = type == MT_ROTARY_NTK ? f : f * (keep + (1.0 - keep) / s);
    }
    *factor = type == MT_ROTARY_YARN ? 0.1 * log(s) + 1.0 : 1.0;
    return MT_OK;
}

mt_status mt_rotary_turns(const double *freqs, int32_t n, uint64_t *turns) {
    if (n < 0 || (n > 0 && (freqs == nullptr || turns == nullptr)))
        return MT_ERR_INVALID_ARGUMENT;
    for (int i = 0; i < n; ++i)
        if (!(fabs(freqs[i]) < 1e6)) return MT_ERR_INVALID_ARGUMENT;
    // 1 / 2 pi as the sum of two doubles: hi carries 53 bits, lo the next.
    const double inv_hi = 0.15915494309189535, inv_lo = -9.839338337591243e-18;
    for (int i = 0; i < n; ++i) {
        const double f = fabs(freqs[i]);
        const double hi = f * inv_hi;
        const double lo = fma(f, inv_hi, -hi) + f * inv_lo;
        const double frac = hi - floor(hi);  // exact; in [0, 1)
        // In units of 2^-64: frac as two 32-bit halves, so that no step
        // leaves the range of the conversions.
        const double up = floor(frac * 4294967296.0);
        const double down = (frac * 4294967296.0 - up) * 4294967296.0;
        const int64_t small = llrint(lo * 18446744073709551616.0);
        const uint64_t t = ((uint64_t)up << 32) + (uint64_t)llrint(down) +
                           (uint64_t)small;
        turns[i] = freqs[i] < 0.0 ? 0 - t : t;
    }
    return MT_OK;
}

mt_status mt_rotary(int dtype, const mt_rotary_call_t *call,
                    mt_stream_t stream) {
    RotArgs a = {};
    int V = 1, K = 1;
    bool empty = false;
    if (mt_status st = rotary_setup(dtype, call, ROT_FORWARD, &a, &V, &K,
                                    &empty))
        return st;
    if (empty) return MT_OK;
    if (too_many_tokens(a.tokens)) return MT_ERR_UNSUPPORTED;
    return status_from_cuda(rotary_forward(dtype, a, V, K,
                                           call->interleaved != 0,
                                           call->norm != 0,
                                           (cudaStream_t)stream));
}

mt_status mt_rotary_backward_workspace(const mt_rotary_call_t *call,
                                       size_t *bytes) {
    if (call == nullptr || bytes == nullptr || call->dim < 1)
        return MT_ERR_INVALID_ARGUMENT;
    if (call->dim > kRotMaxDim) return MT_ERR_UNSUPPORTED;
    *bytes = call->norm && (call->q.dweight || call->k.dweight)
                 ? backward_workspace(call) : 0;
    return MT_OK;
}

mt_status mt_rotary_backward(int dtype, const mt_rotary_call_t *call,
                             void *workspace, size_t workspace_bytes,
                             mt_stream_t stream) {
    RotArgs a = {};
    int V = 1, K = 1;
    bool empty = false;
    if (mt_status st = rotary_setup(dtype, call, ROT_BACKWARD, &a, &V, &K,
                                    &empty))
        return st;
    cudaStream_t s = (cudaStream_t)stream;
    const bool dw = call->q.dweight || call->k.dweight;
    // Gradients of tensors without rows are zero.
    const mt_rotary_heads_t *hs[2] = {&call->q, &call->k};
    if (dw) {
        if (!empty && workspace_bytes < backward_workspace(call))
            return MT_ERR_OUT_OF_RESOURCES;
        if (!empty && (workspace == nullptr || misaligned(workspace, 16)))
            return MT_ERR_INVALID_ARGUMENT;
    }
    if (!empty && too_many_tokens(a.tokens)) return MT_ERR_UNSUPPORTED;
    for (int i = 0; i < 2; ++i)
        if (hs[i]->dweight && (empty || hs[i]->heads == 0)) {
            cudaError_t e = cudaMemsetAsync(hs[i]->dweight, 0,
                                            call->dim * sizeof(float), s);
            if (e != cudaSuccess) return status_from_cuda(e);
        }
    if (empty) return MT_OK;
    if (!call->norm) {
        for (int i = 0; i < 2; ++i) {
            a.t[i].x = a.t[i].dy;
            a.t[i].xt = a.t[i].dt;
            a.t[i].xh = a.t[i].dh;
        }
        return status_from_cuda(rotary_forward(dtype, a, V, K,
                                               call->interleaved != 0, false,
                                               s));
    }
    // As many CTAs as are resident at once (each takes an equal share of the
    // work), shared out between queries and keys by their heads' groups.
    // FP32 takes the larger CTAs where every warp has work: few items are
    // done sooner by warps with all their registers (333 tokens of 12 + 4
    // heads of 64: 5.8 us for 6.9).
    int sms = 0;
    cudaError_t e = current_sm_count(&sms);
    if (e != cudaSuccess) return status_from_cuda(e);
    const int blocks = 2 * sms < kRotBackBlocks ? 2 * sms : kRotBackBlocks;
    const int g0 = a.t[0].groups, g1 = a.t[1].groups;
    a.threads = dtype == DT_F32 && K == 1 &&
                        a.tokens * (g0 + g1) >
                            (int64_t)blocks * (kRotBackThreads / 32)
                    ? kRotBackThreads : kRotThreads;
    const int warps = a.threads / 32;
    for (int i = 0; i < 2; ++i) {
        const int64_t items = a.tokens * a.t[i].groups;
        const int64_t need = (items + warps - 1) / warps;
        // Rounded down, so that the two (one at least each) stay within
        // blocks: where one is raised to 1, the other is below blocks.
        int64_t share = (int64_t)blocks * a.t[i].groups / (g0 + g1);
        if (share < 1) share = 1;
        if (share > need) share = need;
        a.blocks[i] = a.t[i].heads ? (int32_t)share : 0;
    }
    a.partial = dw ? static_cast<float *>(workspace) : nullptr;
    switch (dtype) {
        case DT_F32:
            e = launch_rotary_backward_f32(a, V, K, call->interleaved != 0, s);
            break;
        case DT_F16:
            e = launch_rotary_backward_f16(a, V, K, call->interleaved != 0, s);
            break;
        default:
            e = launch_rotary_backward_bf16(a, V, K, call->interleaved != 0,
                                            s);
    }
    if (e == cudaSuccess && dw)
        e = launch_rotary_dweight(
            a.partial, a.dim, a.blocks,
            a.blocks[0] ? call->q.dweight : nullptr,
            a.blocks[1] ? call->k.dweight : nullptr, s);
    return status_from_cuda(e);
}

mt_status mt_cache_write(int dtype, const mt_cache_call_t *call,
                         mt_stream_t stream) {
    CacheArgs a = {};
    int vec = 0;
    bool empty = false;
    if (mt_status st = cache_setup(dtype, call, true, &a, &vec, &empty))
        return st;
    if (empty) return MT_OK;
    return status_from_cuda(
        launch_cache_write(dtype, a, vec, (cudaStream_t)stream));
}

mt_status mt_cache_read(int dtype, const mt_cache_call_t *call,
                        mt_stream_t stream) {
    CacheArgs a = {};
    int vec = 0;
    bool empty = false;
    if (mt_status st = cache_setup(dtype, call, false, &a, &vec, &empty))
        return st;
    if (empty) return MT_OK;
    return status_from_cuda(
        launch_cache_read(dtype, a, vec, (cudaStream_t)stream));
}

mt_status mt_cache_slots(const int32_t *table, int64_t table_stride,
                         int32_t pages_per_sequence, const int32_t *offsets,
                         const int32_t *starts, int32_t sequences,
                         int32_t page_size, int64_t rows, int64_t *slot,
                         mt_stream_t stream) {
    if (pages_per_sequence < 0 || sequences < 0 || page_size < 1 || rows < 0 ||
        table_stride < 0 || misaligned(table, 4) || misaligned(offsets, 4) ||
        misaligned(starts, 4) || misaligned(slot, 8))
        return MT_ERR_INVALID_ARGUMENT;
    if (rows == 0) return MT_OK;
    if (slot == nullptr ||
        (sequences > 0 && (offsets == nullptr || starts == nullptr)) ||
        (sequences > 0 && pages_per_sequence > 0 && table == nullptr))
        return MT_ERR_INVALID_ARGUMENT;
    if (sequences > 1 && table_stride > kMaxOffset / sequences)
        return MT_ERR_INVALID_ARGUMENT;
    if (rows > (1LL << 38)) return MT_ERR_UNSUPPORTED;
    return status_from_cuda(launch_cache_slots(
        table, table_stride, pages_per_sequence, offsets, starts, sequences,
        page_size, rows, slot, (cudaStream_t)stream));
}

mt_status mt_process_logits(int dtype, const mt_logits_call_t *call,
                            mt_stream_t stream) {
    if (call == nullptr || !known_dtype(dtype)) return MT_ERR_INVALID_ARGUMENT;
    const mt_logits_call_t &c = *call;
    const int es = dtype_size(dtype);
    if (c.rows < 0 || c.vocab < 1 || c.mode < MT_LOGITS ||
        c.mode > MT_LOGITS_LOG_SOFTMAX || c.history < 0 || c.biases < 0)
        return MT_ERR_INVALID_ARGUMENT;
    if (c.vocab > kLogitsMaxVocab || c.history > (1 << 20) - 1 ||
        c.biases > kLogitsMaxBias)
        return MT_ERR_UNSUPPORTED;
    if (misaligned(c.x, es) || misaligned(c.y, es) || misaligned(c.tokens, 4) ||
        misaligned(c.lengths, 4) || misaligned(c.prompt_lengths, 4) ||
        misaligned(c.repetition, 4) || misaligned(c.frequency, 4) ||
        misaligned(c.presence, 4) || misaligned(c.bias_ids, 4) ||
        misaligned(c.bias, 4) || misaligned(c.mask, 4) ||
        misaligned(c.temperature, 4))
        return MT_ERR_INVALID_ARGUMENT;
    // Parts that need one another.
    if (c.history > 0 && c.tokens == nullptr && c.rows > 0)
        return MT_ERR_INVALID_ARGUMENT;
    if (!c.tokens && (c.lengths || c.prompt_lengths || c.repetition ||
                      c.frequency || c.presence))
        return MT_ERR_INVALID_ARGUMENT;
    if (c.biases > 0 && c.rows > 0 && (!c.bias_ids || !c.bias))
        return MT_ERR_INVALID_ARGUMENT;
    if (c.mask && c.mask_stride != 0 && c.mask_stride < (c.vocab + 31) / 32)
        return MT_ERR_INVALID_ARGUMENT;
    if (c.rows > 1 && (c.y_stride < c.vocab || c.x_stride < 0))
        return MT_ERR_INVALID_ARGUMENT;
    if (c.rows > 1 && c.tokens && c.tokens_stride < 0)
        return MT_ERR_INVALID_ARGUMENT;
    if (c.rows == 0) return MT_OK;
    if (c.x == nullptr || c.y == nullptr) return MT_ERR_INVALID_ARGUMENT;
    int64_t extent = c.vocab;
    if (!add_extent(c.x_stride, c.rows, &extent))
        return MT_ERR_INVALID_ARGUMENT;
    extent = c.vocab;
    if (!add_extent(c.y_stride, c.rows, &extent))
        return MT_ERR_INVALID_ARGUMENT;
    extent = c.history;
    if (!add_extent(c.tokens_stride, c.rows, &extent))
        return MT_ERR_INVALID_ARGUMENT;
    extent = c.vocab;
    if (c.mask && !add_extent(c.mask_stride, c.rows, &extent))
        return MT_ERR_INVALID_ARGUMENT;
    if (c.rows > (1LL << 24)) return MT_ERR_UNSUPPORTED;
    cudaStream_t s = (cudaStream_t)stream;
    try {
        return status_from_cuda(dtype == DT_F32   ? launch_logits_f32(c, s)
                                : dtype == DT_F16 ? launch_logits_f16(c, s)
                                                  : launch_logits_bf16(c, s));
    } catch (...) {  // no memory for a table of what kernels were set up
        return MT_ERR_OUT_OF_RESOURCES;
    }
}

}  // extern "C"

// cache.cu -- the quantised cache: rows of heads stored as 8-bit codes with
// one FP32 scale per group of values, read back, and the slots of a packed
// batch's rows from its page tables.
//
//   scale = max(amax (1/q), 2^-126),  code = round(x (1/scale)),  q = 448, 127
//   value = code scale
//
// The floor 2^-126 keeps 1/scale finite, so a group of zeros has codes 0 and
// no case of its own.  A group that holds a NaN or an infinity gets scale NaN
// and codes 0.
#include <cuda_fp8.h>

#include "mt_decoder.cuh"

namespace mt {
namespace {

constexpr int kThreads = 256;     // of the narrow kernels
constexpr int kMaxThreads = 512;  // of the wide ones
constexpr float kTiny = 1.17549435e-38f;  // 2^-126

// Four values times `inv` as four codes.  int8: adding 1.5 * 2^23 leaves the
// product rounded to an integer (half to even) in the low bits of the sum,
// two's complement, exactly for |v| <= 2^22: one addition in place of a
// conversion at a quarter of its rate.  The product is rounded before that,
// as in the definition; the packed forms of the two are not used here, since
// they came out as one fused operation, which takes ties the other way.
template <bool INT8>
__device__ __forceinline__ unsigned encode4(float2 v, float2 w, float inv) {
    if (INT8) {
        const auto code = [inv](float x) {
            return __float_as_uint(__fadd_rn(__fmul_rn(x, inv), 12582912.f));
        };
        const unsigned lo = __byte_perm(code(v.x), code(v.y), 0x0040);
        const unsigned hi = __byte_perm(code(w.x), code(w.y), 0x0040);
        return __byte_perm(lo, hi, 0x5410);
    }
    v = mul2(v, both(inv));
    w = mul2(w, both(inv));
    const unsigned lo = __nv_cvt_float2_to_fp8x2(v, __NV_SATFINITE, __NV_E4M3);
    const unsigned hi = __nv_cvt_float2_to_fp8x2(w, __NV_SATFINITE, __NV_E4M3);
    return lo | hi << 16;
}
template <bool INT8>
__device__ __forceinline__ unsigned encode(float v, float inv) {
    return encode4<INT8>(make_float2(v, 0.f), make_float2(0.f, 0.f), inv) &
           0xffu;
}
// The numbers of four codes.  int8: byte b + 128 under the exponent of 2^23
// is the float 2^23 + 128 + b.
template <bool INT8>
__device__ __forceinline__ void decode4(unsigned c, float2 &v, float2 &w) {
    if (INT8) {
        const unsigned u = c ^ 0x80808080u;
        const float2 off = both(-8388736.f);  // 2^23 + 128
        v = add2(make_float2(
                     __uint_as_float(__byte_perm(u, 0x4b000000u, 0x7540)),
                     __uint_as_float(__byte_perm(u, 0x4b000000u, 0x7541))),
                 off);
        w = add2(make_float2(
                     __uint_as_float(__byte_perm(u, 0x4b000000u, 0x7542)),
                     __uint_as_float(__byte_perm(u, 0x4b000000u, 0x7543))),
                 off);
    } else {
        v = __half22float2(__half2(__nv_cvt_fp8x2_to_halfraw2(
            (__nv_fp8x2_storage_t)(c & 0xffffu), __NV_E4M3)));
        w = __half22float2(__half2(__nv_cvt_fp8x2_to_halfraw2(
            (__nv_fp8x2_storage_t)(c >> 16), __NV_E4M3)));
    }
}
template <bool INT8>
__device__ __forceinline__ float decode(unsigned byte) {
    float2 v, w;
    decode4<INT8>(byte, v, w);
    return v.x;
}

// Scale of a group and the factor its values take: 1/scale, or 0 for a group
// that is not finite (then `bad` is set and its codes are 0).
template <bool INT8>
__device__ __forceinline__ float group_scale(float amax, float &inv,
                                             bool &bad) {
    bad = !(amax < INFINITY);
    const float s = fmaxf(amax * (INT8 ? (float)(1.0 / 127.0)
                                       : (float)(1.0 / 448.0)), kTiny);
    inv = __frcp_rn(s);
    return bad ? __int_as_float(0x7fffffff) : s;
}

// Thread map of the wide kernels.  A token's work is `per` units of one lane
// (over both tensors); a CTA of `rows` * per threads (rounded up to warps)
// serves `rows` tokens at a time, so a lane keeps its place in the row for
// every token it serves and computes its offsets once.  Rows longer than a
// CTA take several (grid.y).
struct Map {
    unsigned per;     // lanes of a token
    unsigned rows;    // tokens of a CTA at a time
    int32_t log2L;    // write: lanes of a group
};

// Writing: groups of up to 512 values, 8 values (one 16-byte access; two for
// FP32) P times per lane, L lanes per group: lane l owns the packs l and
// (P = 2) l + L, so that every access of a warp is contiguous.  N tokens of
// a lane are in flight.
constexpr int kV = 8;

template <typename T>
struct Values8 {
    static constexpr int kLoads = sizeof(T) == 4 ? 2 : 1;
    Raw<T, kV / kLoads> raw[kLoads];
    __device__ __forceinline__ void load(const T *p) {
#pragma unroll
        for (int i = 0; i < kLoads; ++i) raw[i].load(p + i * (kV / kLoads));
    }
    __device__ __forceinline__ void widen(float2 *z) const {
#pragma unroll
        for (int i = 0; i < kLoads; ++i)
            raw[i].widen(&z[0].x + i * (kV / kLoads));
    }
};
template <typename T>
__device__ __forceinline__ void store8(T *p, const float2 *z) {
    st_vec<T, 16 / sizeof(T)>(p, &z[0].x);
    if (sizeof(T) == 4) st_vec<T, 16 / sizeof(T)>(p + 4, &z[0].x + 4);
}

template <typename T, bool INT8, int P, int N>
__global__ void __launch_bounds__(kMaxThreads)
    write_wide_kernel(const CacheArgs a, const Map m) {
    grid_launch_dependents();
    grid_wait_prerequisites();
    const int L = 1 << m.log2L;
    const unsigned unit = blockIdx.y * blockDim.x + threadIdx.x;
    const unsigned row = unit / m.per;  // 0 where a token takes several CTAs
    const unsigned u = unit - row * m.per;
    const unsigned groups = (unsigned)(a.dim / a.group);
    const unsigned per_tensor = (unsigned)a.heads * groups;
    const unsigned gt = u >> m.log2L;  // group of the token
    const int i = gt >= per_tensor ? 1 : 0;
    const unsigned g = gt - (i ? per_tensor : 0);
    const unsigned head = g / groups;
    const int l = (int)(u & (unsigned)(L - 1));
    const bool mine = row < m.rows && gt < per_tensor * (unsigned)a.tensors;
    const int at0 = l * kV;
    const T *x = static_cast<const T *>(a.rows[i]) + (int64_t)head * a.hs[i] +
                 (int64_t)(g - head * groups) * a.group;
    const int64_t ts = a.ts[i];
    // Tokens of this lane: first, first + step, ...; the loop's length is
    // the same for all lanes of a CTA (the exchanges need whole warps).
    const int64_t step = (int64_t)gridDim.x * m.rows;
    for (int64_t base = (int64_t)blockIdx.x * m.rows; base < a.tokens;
         base += step * N) {
        Values8<T> raw[N][P];
        int64_t slot[N];
#pragma unroll
        for (int n = 0; n < N; ++n) {
            const int64_t t = base + n * step + row;
            slot[n] = -1;
            if (mine && t < a.tokens) {
                slot[n] = a.slot[t];
#pragma unroll
                for (int p = 0; p < P; ++p)
                    if (at0 + p * L * kV < a.group)
                        raw[n][p].load(x + t * ts + at0 + p * L * kV);
            }
        }
#pragma unroll
        for (int n = 0; n < N; ++n) {
            if (base + n * step >= a.tokens) break;  // whole CTAs
            const bool in = mine && base + n * step + row < a.tokens;
            float2 z[P][kV / 2];
            float amax = 0.f;
#pragma unroll
            for (int p = 0; p < P; ++p)
                if (in && at0 + p * L * kV < a.group) {
                    raw[n][p].widen(z[p]);
#pragma unroll
                    for (int e = 0; e < kV / 2; ++e)
                        amax = nanmax(amax, nanmax(fabsf(z[p][e].x),
                                                   fabsf(z[p][e].y)));
                }
            for (int off = L >> 1; off > 0; off >>= 1)
                amax = nanmax(amax, __shfl_xor_sync(kFull, amax, off));
            if (!in || slot[n] < 0 || slot[n] >= a.slots) continue;
            float inv;
            bool bad;
            const float s = group_scale<INT8>(amax, inv, bad);
            const int64_t group = slot[n] * per_tensor + g;
            uint8_t *c = a.codes[i] + group * a.group + at0;
#pragma unroll
            for (int p = 0; p < P; ++p)
                if (at0 + p * L * kV < a.group) {
                    unsigned w[2];
#pragma unroll
                    for (int h = 0; h < 2; ++h)
                        w[h] = bad ? 0u
                                   : encode4<INT8>(z[p][2 * h],
                                                   z[p][2 * h + 1], inv);
                    *reinterpret_cast<uint2 *>(c + p * L * kV) =
                        make_uint2(w[0], w[1]);
                }
            if (l == 0) a.scales[i][group] = s;
        }
    }
}

// Any group: a warp per group reads it twice (the second time from L1).
template <typename T, bool INT8>
__global__ void __launch_bounds__(kThreads)
    write_any_kernel(const CacheArgs a, unsigned per_row) {
    grid_launch_dependents();
    grid_wait_prerequisites();
    const int lane = threadIdx.x & 31;
    const int64_t n = (int64_t)blockIdx.x * (kThreads >> 5) +
                      (threadIdx.x >> 5);
    const int64_t row = n / per_row;
    const unsigned g = (unsigned)(n - row * per_row);
    const int64_t t = a.tensors == 2 ? row >> 1 : row;
    const int i = a.tensors == 2 ? (int)(row & 1) : 0;
    if (t >= a.tokens) return;
    const int64_t slot = a.slot[t];
    if (slot < 0 || slot >= a.slots) return;
    const unsigned groups = (unsigned)(a.dim / a.group);
    const unsigned head = g / groups, part = g - head * groups;
    const T *x = static_cast<const T *>(a.rows[i]) + t * a.ts[i] +
                 head * a.hs[i] + part * a.group;
    float amax = 0.f;
    for (int e = lane; e < a.group; e += 32)
        amax = nanmax(amax, fabsf(to_f(x[e])));
    amax = warp_nanmax(amax);
    float inv;
    bool bad;
    const float s = group_scale<INT8>(amax, inv, bad);
    const int64_t group = slot * per_row + g;
    uint8_t *c = a.codes[i] + group * a.group;
    for (int e = lane; e < a.group; e += 32)
        c[e] = bad ? 0 : (uint8_t)encode<INT8>(to_f(x[e]), inv);
    if (lane == 0) a.scales[i][group] = s;
}

// Reading back.  A row's codes are contiguous (heads x dim bytes): 8 of them
// per lane, the lane's place in the row the same for all its tokens, N tokens
// in flight.
template <typename T, bool INT8, int N>
__global__ void __launch_bounds__(kMaxThreads)
    read_wide_kernel(const CacheArgs a, const Map m) {
    grid_launch_dependents();
    grid_wait_prerequisites();
    const unsigned unit = blockIdx.y * blockDim.x + threadIdx.x;
    const unsigned row = unit / m.per;
    const unsigned u = unit - row * m.per;
    const unsigned width = (unsigned)(a.heads * a.dim);
    const unsigned packs = width / kV;
    const int i = u >= packs ? 1 : 0;
    if (row >= m.rows || u >= packs * (unsigned)a.tensors) return;
    const unsigned v = (u - (i ? packs : 0)) * kV;
    const unsigned head = v / (unsigned)a.dim;
    const uint8_t *codes = a.codes[i] + v;
    const float *scales = a.scales[i] + v / (unsigned)a.group;
    const unsigned groups = width / (unsigned)a.group;
    T *y = static_cast<T *>(a.rows[i]) + (int64_t)head * a.hs[i] +
           (v - head * (unsigned)a.dim);
    const int64_t ts = a.ts[i];
    const int64_t step = (int64_t)gridDim.x * m.rows;
    for (int64_t t0 = (int64_t)blockIdx.x * m.rows + row; t0 < a.tokens;
         t0 += step * N) {
        int64_t slot[N];
#pragma unroll
        for (int n = 0; n < N; ++n) {
            const int64_t t = t0 + n * step;
            slot[n] = t < a.tokens ? a.slot[t] : -1;
            if (slot[n] >= a.slots) slot[n] = -1;
        }
        uint2 c[N];
        float s[N];
#pragma unroll
        for (int n = 0; n < N; ++n)
            if (slot[n] >= 0) {
                c[n] = *reinterpret_cast<const uint2 *>(codes +
                                                        slot[n] * width);
                s[n] = scales[slot[n] * groups];
            }
#pragma unroll
        for (int n = 0; n < N; ++n)
            if (slot[n] >= 0) {
                float2 z[kV / 2];
                decode4<INT8>(c[n].x, z[0], z[1]);
                decode4<INT8>(c[n].y, z[2], z[3]);
#pragma unroll
                for (int e = 0; e < kV / 2; ++e) z[e] = mul2(z[e], both(s[n]));
                store8<T>(y + (t0 + n * step) * ts, z);
            }
    }
}

// One value per thread: any sizes, strides and addresses.
template <typename T, bool INT8>
__global__ void __launch_bounds__(kThreads)
    read_any_kernel(const CacheArgs a, unsigned width) {
    grid_launch_dependents();
    grid_wait_prerequisites();
    const int64_t n = (int64_t)blockIdx.x * kThreads + threadIdx.x;
    const int64_t row = n / width;
    const unsigned v = (unsigned)(n - row * width);
    const int64_t t = a.tensors == 2 ? row >> 1 : row;
    const int i = a.tensors == 2 ? (int)(row & 1) : 0;
    if (t >= a.tokens) return;
    const int64_t slot = a.slot[t];
    if (slot < 0 || slot >= a.slots) return;
    const unsigned head = v / (unsigned)a.dim, d = v - head * (unsigned)a.dim;
    const float s = a.scales[i][slot * (width / (unsigned)a.group) +
                                v / (unsigned)a.group];
    static_cast<T *>(a.rows[i])[t * a.ts[i] + (int64_t)head * a.hs[i] + d] =
        from_f<T>(decode<INT8>(a.codes[i][slot * width + v]) * s);
}

__global__ void __launch_bounds__(kThreads)
    slots_kernel(const int32_t *table, int64_t stride, int32_t width,
                 const int32_t *offsets, const int32_t *starts,
                 int32_t sequences, int32_t page, int64_t rows,
                 int64_t *slot) {
    grid_launch_dependents();
    grid_wait_prerequisites();
    const int64_t r = (int64_t)blockIdx.x * kThreads + threadIdx.x;
    if (r >= rows) return;
    // Last sequence that begins at or before r.
    int lo = 0, hi = sequences;  // offsets[lo] <= r < offsets[hi]
    int64_t got = -1;
    if (sequences > 0 && r >= offsets[0] && r < offsets[sequences]) {
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (offsets[mid] <= r) lo = mid; else hi = mid;
        }
        const int64_t p = (int64_t)starts[lo] + (r - offsets[lo]);
        if (p >= 0 && p / page < width) {
            const int32_t id = table[lo * stride + p / page];
            if (id >= 0) got = (int64_t)id * page + p % page;
        }
    }
    slot[r] = got;
}

// Threads, tokens per CTA and grid for `per` lanes per token: as many tokens
// as fit 256 threads, a CTA of at most 512; at most four waves of CTAs, which
// then loop over tokens.
struct Shape {
    Map map;
    dim3 grid;
    int threads;
};
cudaError_t shape_for(int64_t tokens, unsigned per, int log2L, int flight,
                      Shape *out) {
    int sms = 0;
    cudaError_t e = current_sm_count(&sms);
    if (e != cudaSuccess) return e;
    unsigned rows = per >= 256 ? 1 : 256 / per;
    if (rows > tokens) rows = (unsigned)tokens;
    const unsigned lanes = rows * per;
    const unsigned parts = (lanes + kMaxThreads - 1) / kMaxThreads;
    const unsigned threads = ((lanes + parts - 1) / parts + 31) / 32 * 32;
    const int64_t need = (tokens + rows - 1) / rows;
    const int64_t full = (int64_t)sms * (2048 / threads) / parts;
    // few tokens: one round of one token each; many: `flight` per round
    int64_t x = need;
    if (x > 4 * full) x = 4 * full;
    (void)flight;
    if (x < 1) x = 1;
    out->map = {per, rows, log2L};
    out->grid = dim3((unsigned)x, parts);
    out->threads = (int)threads;
    return cudaSuccess;
}

template <typename K>
cudaError_t launch_shape(K kernel, const Shape &s, const CacheArgs &a,
                         cudaStream_t stream) {
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = s.grid;
    cfg.blockDim = dim3((unsigned)s.threads);
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, a, s.map);
}

template <typename T, bool INT8>
cudaError_t write_as(const CacheArgs &a, bool vec, cudaStream_t s) {
    const unsigned per_row = (unsigned)(a.heads * (a.dim / a.group));
    const int64_t groups = a.tokens * a.tensors * (int64_t)per_row;
    if (vec) {
        // two packs per lane where the group has them
        const int P = a.group > kV ? 2 : 1;
        int log2L = 0;
        while ((kV * P << log2L) < a.group) ++log2L;
        Shape shape;
        cudaError_t e = shape_for(
            a.tokens, (unsigned)(a.tensors * per_row) << log2L, log2L, 2,
            &shape);
        if (e != cudaSuccess) return e;
        return P == 2
                   ? launch_shape(write_wide_kernel<T, INT8, 2, 2>, shape, a, s)
                   : launch_shape(write_wide_kernel<T, INT8, 1, 2>, shape, a, s);
    }
    const int64_t per = kThreads / 32;
    return launch_dependent(write_any_kernel<T, INT8>,
                            (groups + per - 1) / per, kThreads, 0, s, a,
                            per_row);
}

template <typename T, bool INT8>
cudaError_t read_as(const CacheArgs &a, bool vec, cudaStream_t s) {
    const unsigned width = (unsigned)(a.heads * a.dim);
    if (vec) {
        Shape shape;
        cudaError_t e = shape_for(a.tokens,
                                  (unsigned)a.tensors * (width / kV), 0, 4,
                                  &shape);
        if (e != cudaSuccess) return e;
        return launch_shape(read_wide_kernel<T, INT8, 4>, shape, a, s);
    }
    const int64_t n = a.tokens * a.tensors * (int64_t)width;
    return launch_dependent(read_any_kernel<T, INT8>,
                            (n + kThreads - 1) / kThreads, kThreads, 0, s, a,
                            width);
}

}  // namespace

#define MT_CACHE_TYPES(f)                                                    \
    switch (dtype) {                                                         \
        case DT_F32:                                                         \
            return a.int8 ? f<float, true>(a, vec, s)                        \
                          : f<float, false>(a, vec, s);                      \
        case DT_F16:                                                         \
            return a.int8 ? f<__half, true>(a, vec, s)                       \
                          : f<__half, false>(a, vec, s);                     \
        default:                                                             \
            return a.int8 ? f<__nv_bfloat16, true>(a, vec, s)                \
                          : f<__nv_bfloat16, false>(a, vec, s);              \
    }

cudaError_t launch_cache_write(int dtype, const CacheArgs &a, bool vec,
                               cudaStream_t s) {
    MT_CACHE_TYPES(write_as)
}
cudaError_t launch_cache_read(int dtype, const CacheArgs &a, bool vec,
                              cudaStream_t s) {
    MT_CACHE_TYPES(read_as)
}
#undef MT_CACHE_TYPES

cudaError_t launch_cache_slots(const int32_t *table, int64_t stride,
                               int32_t width, const int32_t *offsets,
                               const int32_t *starts, int32_t sequences,
                               int32_t page, int64_t rows, int64_t *slot,
                               cudaStream_t s) {
    return launch_dependent(slots_kernel, (rows + kThreads - 1) / kThreads,
                            kThreads, 0, s, table, stride, width, offsets,
                            starts, sequences, page, rows, slot);
}

}  // namespace mt

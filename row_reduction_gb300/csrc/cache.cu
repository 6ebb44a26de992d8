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

constexpr int kThreads = 256;
constexpr float kTiny = 1.17549435e-38f;  // 2^-126

template <bool INT8>
__device__ __forceinline__ unsigned encode(float v) {
    if (INT8) return (unsigned)__float2int_rn(v) & 0xffu;
    return __nv_cvt_float_to_fp8(v, __NV_SATFINITE, __NV_E4M3);
}
template <bool INT8>
__device__ __forceinline__ float decode(unsigned byte) {
    if (INT8) return (float)(int)(signed char)byte;
    return __half2float(__half(__nv_cvt_fp8_to_halfraw(
        (__nv_fp8_storage_t)byte, __NV_E4M3)));
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

// Groups of up to 256 values: V values (16 bytes of x for 16-bit types, 8
// values always) per lane, a power of two of lanes per group, one access in
// and one out per lane.  Group indices run over (token, tensor, head, group).
constexpr int kV = 8;

template <typename T, bool INT8>
__global__ void __launch_bounds__(kThreads)
    write_vec_kernel(const CacheArgs a, int log2L, unsigned per_row) {
    grid_launch_dependents();
    grid_wait_prerequisites();
    const int L = 1 << log2L;
    const int l = threadIdx.x & (L - 1);
    const int64_t n = (int64_t)blockIdx.x * (kThreads >> log2L) +
                      (threadIdx.x >> log2L);
    const int64_t row = n / per_row;  // (token, tensor)
    const unsigned g = (unsigned)(n - row * per_row);
    const int64_t t = a.tensors == 2 ? row >> 1 : row;
    const int i = a.tensors == 2 ? (int)(row & 1) : 0;
    const unsigned groups = (unsigned)(a.dim / a.group);
    const unsigned head = g / groups, part = g - head * groups;
    const int at = l * kV;
    const bool in = t < a.tokens && at < a.group;
    float z[kV];
    float amax = 0.f;
    if (in) {
        ld_vec<T, 16 / sizeof(T)>(
            static_cast<const T *>(a.rows[i]) + t * a.ts[i] +
                head * a.hs[i] + part * a.group + at, z);
        if (sizeof(T) == 4)
            ld_vec<T, 16 / sizeof(T)>(
                static_cast<const T *>(a.rows[i]) + t * a.ts[i] +
                    head * a.hs[i] + part * a.group + at + 4, z + 4);
#pragma unroll
        for (int e = 0; e < kV; ++e) amax = nanmax(amax, fabsf(z[e]));
    }
    for (int off = L >> 1; off > 0; off >>= 1)
        amax = nanmax(amax, __shfl_xor_sync(kFull, amax, off));
    if (!in) return;
    const int64_t slot = a.slot[t];
    if (slot < 0 || slot >= a.slots) return;
    float inv;
    bool bad;
    const float s = group_scale<INT8>(amax, inv, bad);
    unsigned w[2] = {0u, 0u};
    if (!bad) {
#pragma unroll
        for (int e = 0; e < kV; ++e)
            w[e >> 2] |= encode<INT8>(z[e] * inv) << (8 * (e & 3));
    }
    const int64_t group = slot * per_row + g;
    *reinterpret_cast<uint2 *>(a.codes[i] + group * a.group + at) =
        make_uint2(w[0], w[1]);
    if (l == 0) a.scales[i][group] = s;
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
        c[e] = bad ? 0 : (uint8_t)encode<INT8>(to_f(x[e]) * inv);
    if (lane == 0) a.scales[i][group] = s;
}

// Reading back.  A row's codes are contiguous (heads x dim bytes); a thread
// takes V of them and writes V values.
template <typename T, bool INT8, int V>
__global__ void __launch_bounds__(kThreads)
    read_kernel(const CacheArgs a, unsigned packs) {
    grid_launch_dependents();
    grid_wait_prerequisites();
    const int64_t n = (int64_t)blockIdx.x * kThreads + threadIdx.x;
    const int64_t row = n / packs;
    const unsigned p = (unsigned)(n - row * packs);
    const int64_t t = a.tensors == 2 ? row >> 1 : row;
    const int i = a.tensors == 2 ? (int)(row & 1) : 0;
    if (t >= a.tokens) return;
    const int64_t slot = a.slot[t];
    if (slot < 0 || slot >= a.slots) return;
    const unsigned v = p * V;
    const unsigned head = v / (unsigned)a.dim, d = v - head * a.dim;
    const int64_t width = (int64_t)a.heads * a.dim;
    const uint8_t *c = a.codes[i] + slot * width + v;
    const float s = a.scales[i][slot * (width / a.group) + v / a.group];
    T *y = static_cast<T *>(a.rows[i]) + t * a.ts[i] + head * a.hs[i] + d;
    if constexpr (V == 8) {
        const uint2 w = *reinterpret_cast<const uint2 *>(c);
        float z[8];
#pragma unroll
        for (int e = 0; e < 8; ++e)
            z[e] = decode<INT8>((e < 4 ? w.x >> (8 * e) : w.y >> (8 * (e - 4))) & 0xffu) * s;
        st_vec<T, 16 / sizeof(T)>(y, z);
        if (sizeof(T) == 4) st_vec<T, 16 / sizeof(T)>(y + 4, z + 4);
    } else {
        *y = from_f<T>(decode<INT8>(*c) * s);
    }
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

template <typename T, bool INT8>
cudaError_t write_as(const CacheArgs &a, bool vec, cudaStream_t s) {
    const unsigned per_row = (unsigned)(a.heads * (a.dim / a.group));
    const int64_t groups = a.tokens * a.tensors * (int64_t)per_row;
    if (vec) {
        int log2L = 0;
        while ((kV << log2L) < a.group) ++log2L;
        const int64_t per = kThreads >> log2L;
        return launch_dependent(write_vec_kernel<T, INT8>,
                                (groups + per - 1) / per, kThreads, 0, s, a,
                                log2L, per_row);
    }
    const int64_t per = kThreads / 32;
    return launch_dependent(write_any_kernel<T, INT8>,
                            (groups + per - 1) / per, kThreads, 0, s, a,
                            per_row);
}

template <typename T, bool INT8>
cudaError_t read_as(const CacheArgs &a, bool vec, cudaStream_t s) {
    const unsigned width = (unsigned)(a.heads * a.dim);
    const unsigned packs = vec ? width / 8 : width;
    const int64_t n = a.tokens * a.tensors * (int64_t)packs;
    const int64_t grid = (n + kThreads - 1) / kThreads;
    if (vec)
        return launch_dependent(read_kernel<T, INT8, 8>, grid, kThreads, 0, s,
                                a, packs);
    return launch_dependent(read_kernel<T, INT8, 1>, grid, kThreads, 0, s, a,
                            packs);
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

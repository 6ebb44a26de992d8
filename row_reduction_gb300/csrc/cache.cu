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
constexpr int64_t kNarrowGrid = 1 << 18;  // most CTAs of the narrow ones
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

// V values of a row as they lie in memory: 16 (32-byte accesses; one for
// 16-bit types, two for FP32) or 8 (16-byte ones).
template <typename T, int V>
struct Values {
    static constexpr int kWords = V * (int)sizeof(T) / 4;
    unsigned w[kWords];
    __device__ __forceinline__ void load(const T *p) {
        const unsigned *q = reinterpret_cast<const unsigned *>(p);
        if constexpr (V == 16) {
#pragma unroll
            for (int i = 0; i < kWords; i += 8)
                asm volatile("ld.global.v8.b32 {%0, %1, %2, %3, %4, %5, %6, "
                             "%7}, [%8];"
                             : "=r"(w[i]), "=r"(w[i + 1]), "=r"(w[i + 2]),
                               "=r"(w[i + 3]), "=r"(w[i + 4]), "=r"(w[i + 5]),
                               "=r"(w[i + 6]), "=r"(w[i + 7])
                             : "l"(q + i));
        } else {
#pragma unroll
            for (int i = 0; i < kWords; i += 4) {
                const uint4 u = *reinterpret_cast<const uint4 *>(q + i);
                w[i] = u.x; w[i + 1] = u.y; w[i + 2] = u.z; w[i + 3] = u.w;
            }
        }
    }
    // Four values from 4 i on.
    __device__ __forceinline__ void four(int i, float2 &a, float2 &b) const {
        float z[4];
        if constexpr (sizeof(T) == 2) {
            Pack<T>::unpack(w[2 * i], z);
            Pack<T>::unpack(w[2 * i + 1], z + 2);
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e) z[e] = __uint_as_float(w[4 * i + e]);
        }
        a = make_float2(z[0], z[1]);
        b = make_float2(z[2], z[3]);
    }
    // Largest magnitude, as the bits of its type: for floats of one sign the
    // order of the bits is the order of the values, NaN above infinity.
    __device__ __forceinline__ unsigned largest() const {
        unsigned m = 0;
#pragma unroll
        for (int i = 0; i < kWords; ++i)
            m = sizeof(T) == 2 ? __vmaxu2(m, w[i] & 0x7fff7fffu)
                               : max(m, w[i] & 0x7fffffffu);
        return sizeof(T) == 2 ? max(m & 0xffffu, m >> 16) : m;
    }
};
template <typename T>
__device__ __forceinline__ float magnitude(unsigned bits) {
    if constexpr (sizeof(T) == 4) return __uint_as_float(bits);
    const unsigned short h = (unsigned short)bits;
    return to_f(*reinterpret_cast<const T *>(&h));
}
template <typename T, int V>
__device__ __forceinline__ void store_values(T *p, const float2 *z) {
    constexpr int kWords = V * (int)sizeof(T) / 4;
    constexpr int kPer = Pack<T>::kPerWord;
    unsigned w[kWords];
#pragma unroll
    for (int i = 0; i < kWords; ++i) w[i] = Pack<T>::pack(&z[0].x + i * kPer);
    unsigned *q = reinterpret_cast<unsigned *>(p);
    if constexpr (V == 16) {
#pragma unroll
        for (int i = 0; i < kWords; i += 8)
            asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, "
                         "%8};" ::"l"(q + i),
                         "r"(w[i]), "r"(w[i + 1]), "r"(w[i + 2]),
                         "r"(w[i + 3]), "r"(w[i + 4]), "r"(w[i + 5]),
                         "r"(w[i + 6]), "r"(w[i + 7])
                         : "memory");
    } else {
#pragma unroll
        for (int i = 0; i < kWords; i += 4)
            *reinterpret_cast<uint4 *>(q + i) =
                make_uint4(w[i], w[i + 1], w[i + 2], w[i + 3]);
    }
}

// Writing: groups of up to 32 V values, V per lane and L lanes per group.
// The next token's values are on their way while a token's are reduced and
// stored.  Bound by the loads in flight: BF16, 16384 rows of 2 x 8 heads of
// 128 to int8 by 64 20 us, 5.2 TB/s (36 us before rows overlapped, with
// 16-byte accesses).
template <typename T, bool INT8, int V>
__global__ void __launch_bounds__(kMaxThreads, 2)
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
    const int at = (int)(u & (unsigned)(L - 1)) * V;
    const bool mine = row < m.rows && at < a.group &&
                      gt < per_tensor * (unsigned)a.tensors;
    const int64_t ts = a.ts[i];
    const int64_t step = (int64_t)gridDim.x * m.rows;
    int64_t base = (int64_t)blockIdx.x * m.rows;  // the CTA's, of each round
    const T *x = static_cast<const T *>(a.rows[i]) + (int64_t)head * a.hs[i] +
                 (int64_t)(g - head * groups) * a.group + at +
                 (base + row) * ts;
    uint8_t *codes = a.codes[i] + (int64_t)g * a.group + at;
    float *scales = a.scales[i] + g;
    Values<T, V> next;
    int64_t next_slot = -1;
    bool in = mine && base + row < a.tokens;
    if (in) {
        next.load(x);
        next_slot = a.slot[base + row];
    }
    // The loop's length is the same for all lanes of a CTA (the exchanges
    // need whole warps).
    for (; base < a.tokens; base += step) {
        const Values<T, V> v = next;
        const int64_t slot = in ? next_slot : -1;
        const bool there = in;
        x += step * ts;
        in = mine && base + step + row < a.tokens;
        if (in) {
            next.load(x);
            next_slot = a.slot[base + step + row];
        }
        unsigned bits = there ? v.largest() : 0u;
        for (int off = L >> 1; off > 0; off >>= 1)
            bits = max(bits, __shfl_xor_sync(kFull, bits, off));
        if (slot < 0 || slot >= a.slots) continue;
        float inv;
        bool bad;
        const float s = group_scale<INT8>(magnitude<T>(bits), inv, bad);
        unsigned w[V / 4];
#pragma unroll
        for (int h = 0; h < V / 4; ++h) {
            float2 p, q;
            v.four(h, p, q);
            w[h] = bad ? 0u : encode4<INT8>(p, q, inv);
        }
        uint8_t *c = codes + slot * per_tensor * a.group;
        if constexpr (V == 16)
            *reinterpret_cast<uint4 *>(c) =
                make_uint4(w[0], w[1], w[2], w[3]);
        else
            *reinterpret_cast<uint2 *>(c) = make_uint2(w[0], w[1]);
        if (at == 0) scales[slot * per_tensor] = s;
    }
}

// Any group: a warp at a time reads it twice (the second time from L1).  32
// registers keep 64 warps per SM (38 and 48 warps: 13.6 us for 12.8 at 64 rows
// of 2 x 8 heads of 128 by 4).  Bound by instructions per group, whatever its
// size: 16384 such rows 1.6 ms.
template <typename T, bool INT8>
__global__ void __launch_bounds__(kThreads, 8)
    write_any_kernel(const CacheArgs a, unsigned per_row) {
    grid_launch_dependents();
    grid_wait_prerequisites();
    const int lane = threadIdx.x & 31;
    const int64_t total = a.tokens * a.tensors * (int64_t)per_row;
#pragma unroll 1
    for (int64_t n = (int64_t)blockIdx.x * (kThreads >> 5) +
                     (threadIdx.x >> 5);
         n < total; n += (int64_t)gridDim.x * (kThreads >> 5)) {
        const int64_t row = n / per_row;
        const unsigned g = (unsigned)(n - row * per_row);
        const int64_t t = a.tensors == 2 ? row >> 1 : row;
        const int i = a.tensors == 2 ? (int)(row & 1) : 0;
        const int64_t slot = a.slot[t];
        if (slot < 0 || slot >= a.slots) continue;
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
}

// Reading back.  A row's codes are contiguous (heads x dim bytes): V of them
// per lane, the lane's place in the row the same for all its tokens.  N
// tokens' codes are on their way while N tokens are stored, and the slots of
// the N after them.  Bound by the loads in flight: 100003 rows of 2 x 8 heads
// of 128 from e4m3 to BF16 106 us, 5.9 TB/s, 87% of the measured copy
// bandwidth (117 us with 8 values per lane and no overlap of rows).
template <typename T, bool INT8, int V, int N>
__global__ void __launch_bounds__(kMaxThreads, 2)
    read_wide_kernel(const CacheArgs a, const Map m) {
    grid_launch_dependents();
    grid_wait_prerequisites();
    const unsigned unit = blockIdx.y * blockDim.x + threadIdx.x;
    const unsigned row = unit / m.per;
    const unsigned u = unit - row * m.per;
    const unsigned width = (unsigned)(a.heads * a.dim);
    const unsigned packs = width / V;
    const int i = u >= packs ? 1 : 0;
    if (row >= m.rows || u >= packs * (unsigned)a.tensors) return;
    const unsigned v = (u - (i ? packs : 0)) * V;
    const unsigned head = v / (unsigned)a.dim;
    const uint8_t *codes = a.codes[i] + v;
    const float *scales = a.scales[i] + v / (unsigned)a.group;
    const unsigned groups = width / (unsigned)a.group;
    const int64_t ts = a.ts[i];
    T *y = static_cast<T *>(a.rows[i]) + (int64_t)head * a.hs[i] +
           (v - head * (unsigned)a.dim);
    const int64_t step = (int64_t)gridDim.x * m.rows;
    int64_t t = (int64_t)blockIdx.x * m.rows + row;
    struct Stage {
        int64_t slot[N];
        unsigned c[N][V / 4];
        float s[N];
    };
    const auto look = [&](int64_t from, int64_t *slot) {
#pragma unroll
        for (int n = 0; n < N; ++n) {
            const int64_t at = from + n * step;
            slot[n] = at < a.tokens ? a.slot[at] : -1;
        }
    };
    const auto load = [&](const int64_t *slot, Stage &st) {
#pragma unroll
        for (int n = 0; n < N; ++n) {
            st.slot[n] = slot[n] < a.slots ? slot[n] : -1;
            if (st.slot[n] < 0) continue;
            const uint8_t *c = codes + st.slot[n] * width;
            if constexpr (V == 16) {
                const uint4 q = *reinterpret_cast<const uint4 *>(c);
                st.c[n][0] = q.x; st.c[n][1] = q.y;
                st.c[n][2] = q.z; st.c[n][3] = q.w;
            } else {
                const uint2 q = *reinterpret_cast<const uint2 *>(c);
                st.c[n][0] = q.x; st.c[n][1] = q.y;
            }
            st.s[n] = scales[st.slot[n] * groups];
        }
    };
    Stage next;
    int64_t slot[N];
    look(t, slot);
    load(slot, next);
    look(t + N * step, slot);
    for (; t < a.tokens; t += N * step) {
        const Stage now = next;
        load(slot, next);
        look(t + 2 * N * step, slot);
#pragma unroll
        for (int n = 0; n < N; ++n)
            if (now.slot[n] >= 0) {
                float2 z[V / 2];
#pragma unroll
                for (int h = 0; h < V / 4; ++h)
                    decode4<INT8>(now.c[n][h], z[2 * h], z[2 * h + 1]);
#pragma unroll
                for (int e = 0; e < V / 2; ++e)
                    z[e] = mul2(z[e], both(now.s[n]));
                store_values<T, V>(y + (t + n * step) * ts, z);
            }
    }
}

// One value per thread at a time: any sizes, strides and addresses.
template <typename T, bool INT8>
__global__ void __launch_bounds__(kThreads)
    read_any_kernel(const CacheArgs a, unsigned width) {
    grid_launch_dependents();
    grid_wait_prerequisites();
    const int64_t total = a.tokens * a.tensors * (int64_t)width;
#pragma unroll 1
    for (int64_t n = (int64_t)blockIdx.x * kThreads + threadIdx.x; n < total;
         n += (int64_t)gridDim.x * kThreads) {
        const int64_t row = n / width;
        const unsigned v = (unsigned)(n - row * width);
        const int64_t t = a.tensors == 2 ? row >> 1 : row;
        const int i = a.tensors == 2 ? (int)(row & 1) : 0;
        const int64_t slot = a.slot[t];
        if (slot < 0 || slot >= a.slots) continue;
        const unsigned head = v / (unsigned)a.dim;
        const unsigned d = v - head * (unsigned)a.dim;
        const float s = a.scales[i][slot * (width / (unsigned)a.group) +
                                    v / (unsigned)a.group];
        static_cast<T *>(a.rows[i])[t * a.ts[i] + (int64_t)head * a.hs[i] +
                                    d] =
            from_f<T>(decode<INT8>(a.codes[i][slot * width + v]) * s);
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

// Threads, tokens per CTA and grid for `per` lanes per token: as many tokens
// as fit 256 threads, a CTA of at most 512; CTAs enough to fill the device
// once (two of 512 threads per SM), each of which loops over its tokens.
struct Shape {
    Map map;
    dim3 grid;
    int threads;
};
cudaError_t shape_for(int64_t tokens, unsigned per, int log2L, Shape *out) {
    int sms = 0;
    cudaError_t e = current_sm_count(&sms);
    if (e != cudaSuccess) return e;
    unsigned rows = per >= 256 ? 1 : 256 / per;
    if (rows > tokens) rows = (unsigned)tokens;
    const unsigned lanes = rows * per;
    const unsigned parts = (lanes + kMaxThreads - 1) / kMaxThreads;
    const unsigned threads = ((lanes + parts - 1) / parts + 31) / 32 * 32;
    const int64_t need = (tokens + rows - 1) / rows;
    int64_t x = (int64_t)sms * (1024 / threads) / parts;
    if (x < 1) x = 1;
    // rounds of equal length
    if (x > need) x = need;
    const int64_t rounds = (need + x - 1) / x;
    x = (need + rounds - 1) / rounds;
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

// CTAs of a narrow kernel that take `per` of n units at a time.
int64_t narrow_grid(int64_t n, int64_t per) {
    const int64_t need = (n + per - 1) / per;
    return need < kNarrowGrid ? need : kNarrowGrid;
}

template <typename T, bool INT8>
cudaError_t write_as(const CacheArgs &a, int vec, cudaStream_t s) {
    const unsigned per_row = (unsigned)(a.heads * (a.dim / a.group));
    const int64_t groups = a.tokens * a.tensors * (int64_t)per_row;
    if (vec) {
        int log2L = 0;
        while ((vec << log2L) < a.group) ++log2L;
        Shape shape;
        cudaError_t e = shape_for(
            a.tokens, (unsigned)(a.tensors * per_row) << log2L, log2L,
            &shape);
        if (e != cudaSuccess) return e;
        return vec == 16
                   ? launch_shape(write_wide_kernel<T, INT8, 16>, shape, a, s)
                   : launch_shape(write_wide_kernel<T, INT8, 8>, shape, a, s);
    }
    return launch_dependent(write_any_kernel<T, INT8>,
                            narrow_grid(groups, kThreads / 32), kThreads, 0, s,
                            a, per_row);
}

template <typename T, bool INT8>
cudaError_t read_as(const CacheArgs &a, int vec, cudaStream_t s) {
    const unsigned width = (unsigned)(a.heads * a.dim);
    if (vec) {
        Shape shape;
        cudaError_t e = shape_for(
            a.tokens, (unsigned)a.tensors * (width / (unsigned)vec), 0,
            &shape);
        if (e != cudaSuccess) return e;
        return vec == 16
                   ? launch_shape(read_wide_kernel<T, INT8, 16, 2>, shape, a, s)
                   : launch_shape(read_wide_kernel<T, INT8, 8, 2>, shape, a, s);
    }
    const int64_t n = a.tokens * a.tensors * (int64_t)width;
    return launch_dependent(read_any_kernel<T, INT8>,
                            narrow_grid(n, kThreads), kThreads, 0, s, a,
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

cudaError_t launch_cache_write(int dtype, const CacheArgs &a, int vec,
                               cudaStream_t s) {
    MT_CACHE_TYPES(write_as)
}
cudaError_t launch_cache_read(int dtype, const CacheArgs &a, int vec,
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

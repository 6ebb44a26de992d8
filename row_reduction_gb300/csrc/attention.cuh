// attention.cuh -- attention over the quantised cache: what its kernels share.
#pragma once

#include <cuda_fp8.h>

#include "mt_decoder.cuh"

namespace mt {

namespace {

constexpr float kLog2e = 1.4426950408889634f;

// 2^t: one MUFU operation (2^-inf = 0, NaN stays NaN, results below 2^-126
// flush to zero).
__device__ __forceinline__ float pow2(float t) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(t));
    return r;
}

// The largest of three; NaN where one is.
__device__ __forceinline__ float nanmax3(float a, float b, float c) {
    float r;
    asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}

// 1 / x, one unit in the last place (0 where that is below 2^-126).
__device__ __forceinline__ float reciprocal(float x) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

// cap tanh(z / cap).  Near 0, |z| < cap / 4, as z tanh(t) / t for t = z / cap, by
// Taylor's series in t^2 up to t^8 (alternating: the first term left out, 9e-9
// at 1/4, bounds the rest); farther away as cap - 2 cap / (1 + e^2t).  The latter
// is off by some 8 roundings of cap wherever z is, 36 of the value at t = -1/4,
// and of ever more of it towards 0; the series by 4.
struct Cap {
    float cap, near_to, inv, grow;
    // unit: of scores, log2(e) where they are exponents of two.
    __device__ __forceinline__ Cap(float c, float unit) {
        cap = c * unit;
        near_to = 0.25f * cap;
        inv = reciprocal(c) * (1.f / unit);
        grow = 2.f * kLog2e * inv;
    }
    // Two values, less something (pairs take one instruction).
    __device__ __forceinline__ float2 near(float2 z, float2 less) const {
        const float2 t = mul2(z, both(inv)), u = mul2(t, t);
        float2 p = fma2(both(kTanh4), u, both(kTanh3));
        p = fma2(p, u, both(kTanh2));
        p = fma2(p, u, both(kTanh1));
        return fma2(z, fma2(p, u, both(1.f)), less);
    }
    // less: with cap added to it.
    __device__ __forceinline__ float2 far(float2 z, float2 less) const {
        const float2 x = mul2(z, both(grow));
        const float2 e = add2(make_float2(pow2(x.x), pow2(x.y)), both(1.f));
        return fma2(make_float2(reciprocal(e.x), reciprocal(e.y)),
                    both(-2.f * cap), less);
    }
    // `about` less than cap tanh(z / cap).
    __device__ __forceinline__ float2 any(float2 z, float about) const {
        const float2 a = near(z, both(-about)), b = far(z, both(cap - about));
        return make_float2(fabsf(z.x) < near_to ? a.x : b.x,
                           fabsf(z.y) < near_to ? a.y : b.y);
    }
    static constexpr float kTanh1 = -1.f / 3.f, kTanh2 = 2.f / 15.f,
                           kTanh3 = -17.f / 315.f, kTanh4 = 62.f / 2835.f;
};
// A warp's scores of a chunk: where none is far, the series alone (64 sequences
// to 16384 keys, FP16 on int8 codes, 234 us; with a far one in every chunk 241,
// uncapped 225).
template <int N>
__device__ __forceinline__ void cap_scores(const Cap &cap, float (&z)[N][4]) {
    float most = 0.f;
#pragma unroll
    for (int i = 0; i < N; ++i) {
        most = nanmax3(most, fabsf(z[i][0]), fabsf(z[i][1]));
        most = nanmax3(most, fabsf(z[i][2]), fabsf(z[i][3]));
    }
    if (!__any_sync(kFull, !(most < cap.near_to))) {
#pragma unroll
        for (int i = 0; i < N; ++i)
#pragma unroll
            for (int e = 0; e < 4; e += 2) {
                const float2 y = cap.near(make_float2(z[i][e], z[i][e + 1]),
                                          both(0.f));
                z[i][e] = y.x;
                z[i][e + 1] = y.y;
            }
    } else {
#pragma unroll
        for (int i = 0; i < N; ++i)
#pragma unroll
            for (int e = 0; e < 4; e += 2) {
                const float2 y = cap.any(make_float2(z[i][e], z[i][e + 1]),
                                         0.f);
                z[i][e] = y.x;
                z[i][e + 1] = y.y;
            }
    }
}

// Where sequence s begins among the call's rows (ends at s + 1): whatever
// stands in offsets, no row is past them.
__device__ __forceinline__ int32_t begin_of(const mt_attention_call_t &c,
                                            int s) {
    return min(max(c.offsets[s], 0), (int32_t)c.rows);
}

// The sequence of a row of the batch (offsets[0] <= r < offsets[sequences]).
__device__ __forceinline__ int sequence_of(const int32_t *offsets, int n,
                                           int64_t r) {
    int lo = 0, hi = n;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (offsets[mid] <= r) lo = mid; else hi = mid;
    }
    return lo;
}

// The keys that a row at position p sees, of `held` keys: lo..hi (none before
// position 0, whatever its bounds say).
__device__ __forceinline__ void row_sees(const mt_attention_call_t &c,
                                         int64_t row, int64_t p, int64_t held,
                                         int64_t &lo, int64_t &hi) {
    lo = c.first ? (int64_t)c.first[row] : 0;
    hi = c.last ? (int64_t)c.last[row] : p;
    if (c.window) lo = max(lo, p - c.window + 1);
    lo = max(lo, (int64_t)0);
    hi = c.slots > 0 && p >= 0
             ? min(hi, min(held, (int64_t)c.pages * c.page_size) - 1) : -1;
}

// The slot of key j of a sequence, or -1.
__device__ __forceinline__ int64_t slot_of(const mt_attention_call_t &c,
                                           const int32_t *pages, int64_t j) {
    const int32_t id = pages[j / c.page_size];
    const int64_t slot = (int64_t)id * c.page_size + j % c.page_size;
    return id >= 0 && slot < c.slots ? slot : -1;
}

}  // namespace
}  // namespace mt

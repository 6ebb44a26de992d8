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

// cap tanh(z / cap) as cap (1 - 2 / (1 + e^(2 z / cap))): off by a few
// roundings of cap, where tanh.approx would be off by 2^-11 of it.
__device__ __forceinline__ float capped(float z, float cap, float inv_cap) {
    const float e = pow2(z * inv_cap * (2.f * kLog2e));
    return cap - 2.f * cap / (1.f + e);
}

// The same for z2 = 2 z / cap and cap2 = cap, both times log2(e), with the
// hardware's reciprocal (one unit in the last place).
__device__ __forceinline__ float capped2(float z2, float cap2) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.f + pow2(z2)));
    return fmaf(-2.f * cap2, r, cap2);
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

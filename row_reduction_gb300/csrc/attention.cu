// attention.cu -- attention over the quantised cache for any head and group: a
// warp per row and query head, a key at a time.
//
// For what the matrix kernels do not take (attention_head in step.cpp).  Bound by
// instructions and the sum over the warp, five exchanges a key; every query head
// reads its key head's keys for itself.  64 sequences to 16384 keys: heads of 32
// 36 ms, of 96 in three groups 53, of 192 84; prompts of 2 x 512 rows at 4096 keys
// 59, 91 and 78.  That is 3 to 5 times the time of plain torch operations for
// the former, 22 to 37 times for the latter.
#include "attention.cuh"

namespace mt {

namespace {

constexpr int kAnyThreads = 32 * kAttentionAnyWarps;
constexpr int kPerLane = kAttentionMaxDim / 32;

__device__ __forceinline__ float code_value(uint8_t code, bool int8) {
    if (int8) return (float)(int8_t)code;
    return __half2float(__half(__nv_cvt_fp8_to_halfraw(code, __NV_E4M3)));
}

// Lane l holds the values l, l + 32, ... of its head.  Key by key: the product
// summed over the warp, the running maximum and sum, the values added.
template <typename T>
__global__ void __launch_bounds__(kAnyThreads)
    attention_any_kernel(const mt_attention_call_t c) {
    grid_launch_dependents();
    grid_wait_prerequisites();
    const int lane = threadIdx.x & 31;
    const int64_t n = (int64_t)blockIdx.x * (kAnyThreads / 32) +
                      (threadIdx.x >> 5);
    const int64_t row = n / c.q_heads;
    const int head = (int)(n - row * c.q_heads);
    if (row >= c.rows || c.sequences == 0 || row < c.offsets[0] ||
        row >= c.offsets[c.sequences])
        return;
    const int s = sequence_of(c.offsets, c.sequences, row);
    const int64_t start = c.starts[s], from = begin_of(c, s);
    const int64_t p = start + (row - from);
    int64_t lo, hi;
    row_sees(c, row, p, start + (begin_of(c, s + 1) - from), lo, hi);
    const int key_head = head / (c.q_heads / c.k_heads);
    const int groups = c.dim / c.group;
    const int32_t *pages = c.table + s * c.table_stride;
    const T *q = static_cast<const T *>(c.q) + row * c.q_row +
                 (int64_t)head * c.q_head;
    const float slope = c.slopes ? c.slopes[head] : 0.f;
    const Cap cap(c.cap, 1.f);
    const bool int8 = c.format == MT_CACHE_INT8;
    float qv[kPerLane], o[kPerLane];
    bool bad = false;
#pragma unroll
    for (int i = 0; i < kPerLane; ++i) {
        const int d = lane + 32 * i;
        qv[i] = d < c.dim ? to_f(q[d]) : 0.f;
        bad |= !(fabsf(qv[i]) < INFINITY);
        o[i] = 0.f;
    }
    bad = __any_sync(kFull, bad);
    float top = -INFINITY, sum = 0.f;
    bool seen = false;
    for (int64_t j = lo; j <= hi; ++j) {
        const int64_t slot = slot_of(c, pages, j);
        if (slot < 0) continue;
        seen = true;
        const int64_t at = slot * c.k_heads + key_head;
        const uint8_t *kc = static_cast<const uint8_t *>(c.k_codes) +
                            at * c.dim;
        const uint8_t *vc = static_cast<const uint8_t *>(c.v_codes) +
                            at * c.dim;
        const float *ks = c.k_scales + at * groups;
        const float *vs = c.v_scales + at * groups;
        float z = 0.f;
#pragma unroll
        for (int i = 0; i < kPerLane; ++i) {
            const int d = lane + 32 * i;
            if (d < c.dim)
                z = fmaf(qv[i], code_value(kc[d], int8) * ks[d / c.group], z);
        }
#pragma unroll
        for (int off = 16; off > 0; off >>= 1)
            z += __shfl_xor_sync(kFull, z, off);
        z *= c.scale;
        if (c.cap > 0.f) z = cap.any(make_float2(z, z), 0.f).x;
        if (c.slopes) z -= slope * fabsf((float)(p - j));
        const float next = nanmax(top, z);
        const float keep = top == -INFINITY ? 0.f
                                            : pow2((top - next) * kLog2e);
        const float e = pow2((z - next) * kLog2e);
        sum = sum * keep + e;
        top = next;
#pragma unroll
        for (int i = 0; i < kPerLane; ++i) {
            const int d = lane + 32 * i;
            if (d < c.dim)
                o[i] = fmaf(e, code_value(vc[d], int8) * vs[d / c.group],
                            o[i] * keep);
        }
    }
    bad = bad && seen;
    const float inv = bad ? NAN : seen ? 1.f / sum : 0.f;
    T *out = static_cast<T *>(c.out) + row * c.out_row +
             (int64_t)head * c.out_head;
#pragma unroll
    for (int i = 0; i < kPerLane; ++i) {
        const int d = lane + 32 * i;
        if (d < c.dim) out[d] = from_f<T>(seen ? o[i] * inv : 0.f);
    }
    if (c.lse != nullptr && lane == 0)
        c.lse[row * c.q_heads + head] =
            bad ? NAN : seen ? top + logf(sum) : -INFINITY;
}

}  // namespace

cudaError_t launch_attention_any(int dtype, const mt_attention_call_t &c,
                                 cudaStream_t s) {
    const int64_t grid =
        (c.rows * c.q_heads + kAttentionAnyWarps - 1) / kAttentionAnyWarps;
    switch (dtype) {
        case DT_F32:
            return launch_dependent(attention_any_kernel<float>, grid,
                                    kAnyThreads, 0, s, c);
        case DT_F16:
            return launch_dependent(attention_any_kernel<__half>, grid,
                                    kAnyThreads, 0, s, c);
        default:
            return launch_dependent(attention_any_kernel<__nv_bfloat16>, grid,
                                    kAnyThreads, 0, s, c);
    }
}

}  // namespace mt

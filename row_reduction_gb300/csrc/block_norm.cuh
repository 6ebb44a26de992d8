// block_norm.cuh -- the norms around a block with its gate and the residual's
// scale, forward and backward (one translation unit per storage type).
#pragma once

#include "mt_decoder.cuh"

namespace mt {
namespace {

constexpr int kLoop = 256;  // threads of the kernels for any row

// Sums of N values over the CTA, the same bits in every thread.
template <int N>
__device__ __forceinline__ void cta_sum(float (&v)[N]) {
    __shared__ float part[N][32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int warps = (int)blockDim.x >> 5;
#pragma unroll
    for (int i = 0; i < N; ++i)
#pragma unroll
        for (int o = 16; o > 0; o >>= 1)
            v[i] += __shfl_xor_sync(kFull, v[i], o);
    __syncthreads();  // readers of the call before
    if (lane == 0)
#pragma unroll
        for (int i = 0; i < N; ++i) part[i][warp] = v[i];
    __syncthreads();
#pragma unroll
    for (int i = 0; i < N; ++i) {
        float t = lane < warps ? part[i][lane] : 0.f;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) t += __shfl_xor_sync(kFull, t, o);
        v[i] = t;
    }
}

template <typename T>
__device__ __forceinline__ float at(const void *p, int64_t i, float absent) {
    return p == nullptr ? absent : to_f(static_cast<const T *>(p)[i]);
}

// Any row: a CTA per row, which reads it once per sum and once to write.
template <typename T>
__global__ void __launch_bounds__(kLoop)
    norm_any_kernel(const mt_block_norm_call_t c) {
    grid_launch_dependents();
    grid_wait_prerequisites();
    const int64_t r = blockIdx.x;
    const int64_t x = r * c.x_stride, res = r * c.residual_stride;
    const int64_t gate = r * c.gate_stride;
    const float inv = 1.f / (float)c.cols;
    float r1 = 1.f;
    if (c.norms & MT_NORM_AFTER) {
        float s[1] = {0.f};
        for (int i = threadIdx.x; i < c.cols; i += kLoop) {
            const float v = at<T>(c.x, x + i, 0.f);
            s[0] = fmaf(v, v, s[0]);
        }
        cta_sum(s);
        r1 = rsqrtf(fmaf(s[0], inv, c.eps));
    }
    const auto stream = [&](int i) {
        const float u = at<T>(c.x, x + i, 0.f) * r1 * at<T>(c.weight, i, 1.f);
        return fmaf(at<T>(c.residual, res + i, 0.f), c.residual_scale,
                    u * at<T>(c.gate, gate + i, 1.f));
    };
    float r2 = 0.f;
    if (c.norms & MT_NORM_BEFORE) {
        float s[1] = {0.f};
        for (int i = threadIdx.x; i < c.cols; i += kLoop) {
            const float h = stream(i);
            s[0] = fmaf(h, h, s[0]);
        }
        cta_sum(s);
        r2 = rsqrtf(fmaf(s[0], inv, c.eps));
    }
    for (int i = threadIdx.x; i < c.cols; i += kLoop) {
        const float h = stream(i);
        static_cast<T *>(c.h)[r * c.h_stride + i] = from_f<T>(h);
        if (c.norms & MT_NORM_BEFORE)
            static_cast<T *>(c.y)[r * c.y_stride + i] =
                from_f<T>(h * r2 * at<T>(c.next_weight, i, 1.f));
    }
}

// Any row, backward: a CTA takes every gridDim.x-th row and adds its weights'
// gradients up in its own row of partial sums.
template <typename T>
__global__ void __launch_bounds__(kLoop)
    norm_back_any_kernel(const mt_block_norm_back_t c, float *partial) {
    grid_launch_dependents();
    grid_wait_prerequisites();
    const float inv = 1.f / (float)c.cols;
    const bool after = c.norms & MT_NORM_AFTER, before = c.norms & MT_NORM_BEFORE;
    float *sums = partial + (int64_t)blockIdx.x * 3 * c.cols;
    if (partial != nullptr)
        for (int i = threadIdx.x; i < 3 * c.cols; i += kLoop) sums[i] = 0.f;
    __syncthreads();
    for (int64_t r = blockIdx.x; r < c.rows; r += gridDim.x) {
        const int64_t x = r * c.x_stride, h = r * c.h_stride;
        const int64_t gate = r * c.gate_stride;
        float s[3] = {0.f, 0.f, 0.f};
        for (int i = threadIdx.x; i < c.cols; i += kLoop) {
            if (after) {
                const float v = at<T>(c.x, x + i, 0.f);
                s[0] = fmaf(v, v, s[0]);
            }
            if (before) {
                const float v = at<T>(c.h, h + i, 0.f);
                s[1] = fmaf(v, v, s[1]);
                s[2] = fmaf(at<T>(c.dy, r * c.dy_stride + i, 0.f) *
                                at<T>(c.next_weight, i, 1.f), v, s[2]);
            }
        }
        cta_sum(s);
        const float r1 = after ? rsqrtf(fmaf(s[0], inv, c.eps)) : 1.f;
        const float r2 = before ? rsqrtf(fmaf(s[1], inv, c.eps)) : 0.f;
        const float m2 = s[2] * inv * r2 * r2;
        const auto grad = [&](int i) {
            float g = at<T>(c.dh, r * c.dh_stride + i, 0.f);
            if (before)
                g += r2 * (at<T>(c.dy, r * c.dy_stride + i, 0.f) *
                               at<T>(c.next_weight, i, 1.f) -
                           at<T>(c.h, h + i, 0.f) * m2);
            return g;
        };
        float m1 = 0.f;
        if (after) {
            float t[1] = {0.f};
            for (int i = threadIdx.x; i < c.cols; i += kLoop)
                t[0] = fmaf(grad(i) * at<T>(c.gate, gate + i, 1.f) *
                                at<T>(c.weight, i, 1.f),
                            at<T>(c.x, x + i, 0.f), t[0]);
            cta_sum(t);
            m1 = t[0] * inv * r1 * r1;
        }
        for (int i = threadIdx.x; i < c.cols; i += kLoop) {
            const float g = grad(i), xv = at<T>(c.x, x + i, 0.f);
            const float w = at<T>(c.weight, i, 1.f);
            const float e = g * at<T>(c.gate, gate + i, 1.f);
            const float dg = g * xv * r1 * w;
            if (partial != nullptr) {
                if (c.dgate_sum) sums[i] += dg;
                if (c.dweight) sums[c.cols + i] += e * xv * r1;
                if (c.dnext_weight)
                    sums[2 * c.cols + i] +=
                        at<T>(c.dy, r * c.dy_stride + i, 0.f) *
                        at<T>(c.h, h + i, 0.f) * r2;
            }
            const float dx = after ? r1 * (e * w - xv * m1) : e;
            static_cast<T *>(c.dx)[r * c.dx_stride + i] = from_f<T>(dx);
            static_cast<T *>(c.dresidual)[r * c.dresidual_stride + i] =
                from_f<T>(g * c.residual_scale);
            if (c.dgate)
                static_cast<T *>(c.dgate)[r * c.dgate_stride + i] =
                    from_f<T>(dg);
        }
    }
}

template <typename T>
cudaError_t norm_as(const mt_block_norm_call_t &c, cudaStream_t s) {
    return launch_dependent(norm_any_kernel<T>, c.rows, kLoop, 0, s, c);
}

}  // namespace

#define MT_DEFINE_BLOCK_NORM(T, dt)                                          \
    cudaError_t launch_block_norm_##dt(const mt_block_norm_call_t &c,        \
                                       cudaStream_t s) {                     \
        return norm_as<T>(c, s);                                             \
    }                                                                        \
    cudaError_t launch_block_norm_back_##dt(const mt_block_norm_back_t &c,   \
                                            float *partial, int blocks,      \
                                            cudaStream_t s) {                \
        return launch_dependent(norm_back_any_kernel<T>, blocks, kLoop, 0,   \
                                s, c, partial);                              \
    }

}  // namespace mt

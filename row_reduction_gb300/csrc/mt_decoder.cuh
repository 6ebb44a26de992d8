// mt_decoder.cuh -- what the kernels of the decoder's row operators share
// (rotary positions, quantised cache, logits); their C entry points are in
// decoder.cpp.
#pragma once

#include "mt_kernels.cuh"
#include "mt_decoder_internal.h"

namespace mt {

// A launch as a programmatic dependent of the previous kernel on the stream:
// the kernel may start while that one finishes and waits for it
// (grid_wait_prerequisites) before it touches memory.
template <typename... P, typename... A>
cudaError_t launch_dependent(void (*kernel)(P...), int64_t grid, int threads,
                             size_t smem, cudaStream_t stream, A... args) {
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)grid);
    cfg.blockDim = dim3((unsigned)threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

// ---- pairs of FP32 values ---------------------------------------------------
// Two FP32 operations per instruction (sm_100 family), each rounded as the
// single ones are.
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
    float2 d;
    asm("{\n\t.reg .b64 a, b, c, d;\n\t"
        "mov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\t"
        "mov.b64 c, {%6, %7};\n\tfma.rn.f32x2 d, a, b, c;\n\t"
        "mov.b64 {%0, %1}, d;\n\t}"
        : "=f"(d.x), "=f"(d.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
    return d;
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
    float2 d;
    asm("{\n\t.reg .b64 a, b, d;\n\t"
        "mov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\t"
        "mul.rn.f32x2 d, a, b;\n\tmov.b64 {%0, %1}, d;\n\t}"
        : "=f"(d.x), "=f"(d.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return d;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
    float2 d;
    asm("{\n\t.reg .b64 a, b, d;\n\t"
        "mov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\t"
        "add.rn.f32x2 d, a, b;\n\tmov.b64 {%0, %1}, d;\n\t}"
        : "=f"(d.x), "=f"(d.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return d;
}
__device__ __forceinline__ float2 both(float v) { return make_float2(v, v); }

// N values at a time, in pairs where there are pairs: o = a b + c, o = a b.
template <int N>
__device__ __forceinline__ void fma_n(float *o, const float *a,
                                      const float *b, const float *c) {
    if constexpr (N == 1) {
        o[0] = fmaf(a[0], b[0], c[0]);
    } else {
#pragma unroll
        for (int i = 0; i < N; i += 2) {
            const float2 v = fma2(make_float2(a[i], a[i + 1]),
                                  make_float2(b[i], b[i + 1]),
                                  make_float2(c[i], c[i + 1]));
            o[i] = v.x;
            o[i + 1] = v.y;
        }
    }
}
template <int N>
__device__ __forceinline__ void mul_n(float *o, const float *a,
                                      const float *b) {
    if constexpr (N == 1) {
        o[0] = a[0] * b[0];
    } else {
#pragma unroll
        for (int i = 0; i < N; i += 2) {
            const float2 v = mul2(make_float2(a[i], a[i + 1]),
                                  make_float2(b[i], b[i + 1]));
            o[i] = v.x;
            o[i + 1] = v.y;
        }
    }
}
// o = s a and o = s a + c for one factor s.
template <int N>
__device__ __forceinline__ void scale_n(float *o, const float *a, float s) {
    if constexpr (N == 1) {
        o[0] = a[0] * s;
    } else {
#pragma unroll
        for (int i = 0; i < N; i += 2) {
            const float2 v = mul2(make_float2(a[i], a[i + 1]), both(s));
            o[i] = v.x;
            o[i + 1] = v.y;
        }
    }
}
template <int N>
__device__ __forceinline__ void scale_add_n(float *o, const float *a, float s,
                                            const float *c) {
    if constexpr (N == 1) {
        o[0] = fmaf(a[0], s, c[0]);
    } else {
#pragma unroll
        for (int i = 0; i < N; i += 2) {
            const float2 v = fma2(make_float2(a[i], a[i + 1]), both(s),
                                  make_float2(c[i], c[i + 1]));
            o[i] = v.x;
            o[i + 1] = v.y;
        }
    }
}

// V values of T as they lie in memory (aligned to V*sizeof(T) bytes): loads
// can be issued long before their values are widened.
template <typename T, int V>
struct Raw {
    static constexpr int kBytes = V * (int)sizeof(T);
    static constexpr int kWords = kBytes < 4 ? 1 : kBytes / 4;
    unsigned w[kWords];
    __device__ __forceinline__ void load(const T *p) {
        if constexpr (kWords == 4) {
            const uint4 u = *reinterpret_cast<const uint4 *>(p);
            w[0] = u.x; w[1] = u.y; w[2] = u.z; w[3] = u.w;
        } else if constexpr (kWords == 2) {
            const uint2 u = *reinterpret_cast<const uint2 *>(p);
            w[0] = u.x; w[1] = u.y;
        } else if constexpr (kBytes == 4) {
            w[0] = *reinterpret_cast<const unsigned *>(p);
        } else {
            w[0] = *reinterpret_cast<const unsigned short *>(p);
        }
    }
    __device__ __forceinline__ void store(T *p) const {
        if constexpr (kWords == 4) {
            *reinterpret_cast<uint4 *>(p) = make_uint4(w[0], w[1], w[2], w[3]);
        } else if constexpr (kWords == 2) {
            *reinterpret_cast<uint2 *>(p) = make_uint2(w[0], w[1]);
        } else if constexpr (kBytes == 4) {
            *reinterpret_cast<unsigned *>(p) = w[0];
        } else {
            *reinterpret_cast<unsigned short *>(p) = (unsigned short)w[0];
        }
    }
    __device__ __forceinline__ void zero() {
#pragma unroll
        for (int i = 0; i < kWords; ++i) w[i] = 0;
    }
    __device__ __forceinline__ void widen(float *d) const {
        if constexpr (kBytes >= 4) {
#pragma unroll
            for (int i = 0; i < kWords; ++i)
                Pack<T>::unpack(w[i], d + i * Pack<T>::kPerWord);
        } else {
            const unsigned short h = (unsigned short)w[0];
            d[0] = to_f(*reinterpret_cast<const T *>(&h));
        }
    }
};

}  // namespace mt

// rotary.cuh -- rotary positions of query and key heads, with the RMSNorm of
// each head in front: forward, and backward (one translation unit per
// storage type).
//
//   turn:  y_a = s (a cos - b sin),  y_b = s (a sin + b cos),  angle = p f_i
//   norm:  x <- x r w,  r = 1/sqrt(mean(x^2) + eps)
//   back:  g = s R^T dy,  dx = r (g w - x r^2 mean(g w x)),  dw = sum g x r
//
// Every value is read once and written once and takes about ten flops, so
// HBM bandwidth is the bound.  A warp serves one token (or a part of its
// heads, where there are few tokens): the cosines and sines of a pair are
// computed once per token and reused for every head the warp serves.
//
// Ownership.  A head is served by L lanes (a power of two); lane l owns the
// slots l, l+L, ... of it.  A slot is two packs of V values holding V whole
// pairs: packs j and pairs/V + j in the half layout, packs 2j and 2j+1 in
// the interleaved one.  So no pair is split between lanes, and the only
// exchange is the norm's sum over L lanes.
//
// Angles.  turns[i] is the pair's frequency in units of 2^-64 turns; position
// times that, modulo 2^64, is the angle exactly (the frequency's own rounding
// of 2^-65 turns grows to 2^-34 turns at position 2^31).  Its top 32 bits,
// taken as signed, give the angle in [-pi, pi) to 2^-33 turns, and their
// conversion to FP32 rounds at 2^-25 of half a turn: 1e-7 radians, whatever
// the position.
#pragma once

#include "mt_decoder.cuh"

namespace mt {

template <typename T, int V, int K, bool ILV>
struct RotSlots {
    // Offsets of the two packs of slot j.
    static __device__ __forceinline__ void offsets(const RotArgs &a, int j,
                                                   int &lo, int &hi) {
        if (ILV || j >= a.rot_slots) {
            lo = 2 * j * V;
            hi = lo + V;
        } else {
            lo = j * V;
            hi = a.pairs + j * V;
        }
    }
    static __device__ __forceinline__ void load(const RotArgs &a, const T *p,
                                                int j, float *z) {
        int lo, hi;
        offsets(a, j, lo, hi);
        ld_vec<T, V>(p + lo, z);
        if (V > 1 || hi < a.dim)
            ld_vec<T, V>(p + hi, z + V);
        else
            z[V] = 0.f;  // an odd head's last value has no partner
    }
    static __device__ __forceinline__ void store(const RotArgs &a, T *p,
                                                 int j, const float *z) {
        int lo, hi;
        offsets(a, j, lo, hi);
        st_vec<T, V>(p + lo, z);
        if (V > 1 || hi < a.dim) st_vec<T, V>(p + hi, z + V);
    }
    static __device__ __forceinline__ void weights(const RotArgs &a,
                                                   const T *w, int j,
                                                   float *z) {
        if (w == nullptr) {
#pragma unroll
            for (int e = 0; e < 2 * V; ++e) z[e] = 1.f;
            return;
        }
        int lo, hi;
        offsets(a, j, lo, hi);
        ld_vec<T, V, true>(w + lo, z);
        if (V > 1 || hi < a.dim)
            ld_vec<T, V, true>(w + hi, z + V);
        else
            z[V] = 0.f;
    }
    // s cos and s sin of the slot's pairs at position p (1 and 0 for a slot
    // that is not rotated).
    static __device__ __forceinline__ void angles(const RotArgs &a,
                                                  int64_t pos, int j,
                                                  float *c, float *s) {
        const bool rot = j < a.rot_slots;
#pragma unroll
        for (int e = 0; e < V; ++e) {
            c[e] = 1.f;
            s[e] = 0.f;
            if (rot) {
                const uint64_t t =
                    (uint64_t)pos *
                    __ldg(reinterpret_cast<const unsigned long long *>(
                              a.turns) +
                          j * V + e);
                const float half_turns =
                    (float)(int32_t)(t >> 32) * 4.6566128730773926e-10f;
                float sn, cs;
                sincospif(half_turns, &sn, &cs);
                c[e] = cs * a.scale;
                s[e] = sn * a.scale * a.sign;
            }
        }
    }
    static __device__ __forceinline__ void turn(float *z, const float *c,
                                                const float *s) {
#pragma unroll
        for (int e = 0; e < V; ++e) {
            const int ia = ILV ? 2 * e : e, ib = ILV ? 2 * e + 1 : V + e;
            const float x = z[ia], y = z[ib];
            z[ia] = x * c[e] - y * s[e];
            z[ib] = x * s[e] + y * c[e];
        }
    }
};

__device__ __forceinline__ int64_t rot_position(const RotArgs &a, int64_t t) {
    return a.pos64 ? static_cast<const int64_t *>(a.pos)[t]
                   : (int64_t) static_cast<const int32_t *>(a.pos)[t];
}

// Sum over the L lanes of a head (xor butterfly; every lane gets it).
__device__ __forceinline__ float head_sum(float v, int log2L) {
    for (int off = (1 << log2L) >> 1; off > 0; off >>= 1)
        v += __shfl_xor_sync(kFull, v, off);
    return v;
}

template <typename T, int V, int K, bool ILV, bool NORM>
__global__ void __launch_bounds__(kRotThreads)
    rotary_kernel(const RotArgs a) {
    using S = RotSlots<T, V, K, ILV>;
    constexpr int U = K == 1 ? 2 : 1;  // groups of heads in flight
    grid_launch_dependents();
    grid_wait_prerequisites();
    const int lane = threadIdx.x & 31;
    const int L = 1 << a.log2L;
    const int l = lane & (L - 1), sub = lane >> a.log2L;
    const int heads_per_warp = 32 >> a.log2L;
    const int64_t unit = (int64_t)blockIdx.x * (kRotThreads / 32) +
                         (threadIdx.x >> 5);
    const int64_t t = unit >> a.log2S;
    if (t >= a.tokens) return;  // whole warps
    const int S_ = 1 << a.log2S;
    const int first = (int)(unit & (S_ - 1));
    const int64_t pos = rot_position(a, t);
    float c[K][V], s[K][V];
#pragma unroll
    for (int k = 0; k < K; ++k) S::angles(a, pos, l + k * L, c[k], s[k]);
#pragma unroll 1
    for (int i = 0; i < 2; ++i) {
        const RotHeads &h = a.t[i];
        if (h.heads == 0) continue;
        const T *x = static_cast<const T *>(h.x) + t * h.xt;
        T *y = static_cast<T *>(h.y) + t * h.yt;
        float w[NORM ? K : 1][2 * V];
        if (NORM) {
#pragma unroll
            for (int k = 0; k < K; ++k)
                if (l + k * L < a.slots)
                    S::weights(a, static_cast<const T *>(h.w), l + k * L,
                               w[k]);
        }
        // The warps of a token take its groups of heads in turn; the key
        // heads' groups follow the query heads'.
        const int g0 = i == 0 ? first : (first - a.t[0].groups) & (S_ - 1);
        for (int g = g0; g < h.groups; g += U * S_) {
            float z[U][K][2 * V];
            bool in[U][K];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int head = (g + u * S_) * heads_per_warp + sub;
#pragma unroll
                for (int k = 0; k < K; ++k) {
                    in[u][k] = head < h.heads && l + k * L < a.slots;
                    if (in[u][k])
                        S::load(a, x + head * h.xh, l + k * L, z[u][k]);
                }
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int head = (g + u * S_) * heads_per_warp + sub;
                if (NORM) {
                    float ss = 0.f;
#pragma unroll
                    for (int k = 0; k < K; ++k)
                        if (in[u][k]) {
#pragma unroll
                            for (int e = 0; e < 2 * V; ++e)
                                ss += z[u][k][e] * z[u][k][e];
                        }
                    const float r =
                        rsqrtf(head_sum(ss, a.log2L) * a.inv_dim + a.eps);
#pragma unroll
                    for (int k = 0; k < K; ++k)
#pragma unroll
                        for (int e = 0; e < 2 * V; ++e)
                            z[u][k][e] *= r * w[k][e];
                }
#pragma unroll
                for (int k = 0; k < K; ++k)
                    if (in[u][k]) {
                        S::turn(z[u][k], c[k], s[k]);
                        S::store(a, y + head * h.yh, l + k * L, z[u][k]);
                    }
            }
        }
    }
}

// Backward with norm.  A CTA serves the heads of one tensor and adds up its
// part of the weight's gradient in registers over all its tokens; at the end
// the lanes and warps that own the same slot are added in a fixed order and
// the CTA writes one row of partial sums, which rotary_dweight_kernel adds.
template <typename T, int V, int K, bool ILV>
__global__ void __launch_bounds__(kRotThreads)
    rotary_backward_kernel(const RotArgs a) {
    using S = RotSlots<T, V, K, ILV>;
    constexpr int kWarps = kRotThreads / 32;
    __shared__ float sums[kWarps][kRotMaxDim];
    grid_launch_dependents();
    grid_wait_prerequisites();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int L = 1 << a.log2L;
    const int l = lane & (L - 1), sub = lane >> a.log2L;
    const int heads_per_warp = 32 >> a.log2L;
    const int i = (int)blockIdx.x < a.blocks[0] ? 0 : 1;
    const int block = (int)blockIdx.x - (i ? a.blocks[0] : 0);
    const RotHeads &h = a.t[i];
    const int S_ = 1 << a.log2S;
    float w[K][2 * V], dw[K][2 * V];
#pragma unroll
    for (int k = 0; k < K; ++k) {
#pragma unroll
        for (int e = 0; e < 2 * V; ++e) w[k][e] = dw[k][e] = 0.f;
        if (l + k * L < a.slots)
            S::weights(a, static_cast<const T *>(h.w), l + k * L, w[k]);
    }
    const int64_t units = a.tokens << a.log2S;
    for (int64_t unit = (int64_t)block * kWarps + warp; unit < units;
         unit += (int64_t)a.blocks[i] * kWarps) {
        const int64_t t = unit >> a.log2S;
        const int64_t pos = rot_position(a, t);
        const T *x = static_cast<const T *>(h.x) + t * h.xt;
        const T *dy = static_cast<const T *>(h.dy) + t * h.dt;
        T *y = static_cast<T *>(h.y) + t * h.yt;
        float c[K][V], s[K][V];
#pragma unroll
        for (int k = 0; k < K; ++k) S::angles(a, pos, l + k * L, c[k], s[k]);
        for (int g = (int)(unit & (S_ - 1)); g < h.groups; g += S_) {
            const int head = g * heads_per_warp + sub;
            float z[K][2 * V], d[K][2 * V];
            float xx = 0.f, gx = 0.f;
#pragma unroll
            for (int k = 0; k < K; ++k) {
                if (head < h.heads && l + k * L < a.slots) {
                    S::load(a, x + head * h.xh, l + k * L, z[k]);
                    S::load(a, dy + head * h.dh, l + k * L, d[k]);
                } else {
#pragma unroll
                    for (int e = 0; e < 2 * V; ++e) z[k][e] = d[k][e] = 0.f;
                }
            }
#pragma unroll
            for (int k = 0; k < K; ++k) {
                S::turn(d[k], c[k], s[k]);
#pragma unroll
                for (int e = 0; e < 2 * V; ++e) {
                    xx += z[k][e] * z[k][e];
                    gx += d[k][e] * w[k][e] * z[k][e];
                }
            }
            xx = head_sum(xx, a.log2L);
            gx = head_sum(gx, a.log2L);
            // no head: r = 0, so that eps = 0 adds no 0 * inf to dw
            const float r = head < h.heads
                                ? rsqrtf(xx * a.inv_dim + a.eps) : 0.f;
            const float m = gx * a.inv_dim * r * r;
#pragma unroll
            for (int k = 0; k < K; ++k) {
#pragma unroll
                for (int e = 0; e < 2 * V; ++e) {
                    dw[k][e] += d[k][e] * (z[k][e] * r);
                    d[k][e] = r * (d[k][e] * w[k][e] - z[k][e] * m);
                }
                if (head < h.heads && l + k * L < a.slots)
                    S::store(a, y + head * h.yh, l + k * L, d[k]);
            }
        }
    }
    if (a.partial == nullptr) return;
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
        for (int e = 0; e < 2 * V; ++e)
            for (int off = L; off < 32; off <<= 1)
                dw[k][e] += __shfl_xor_sync(kFull, dw[k][e], off);
#pragma unroll
    for (int k = 0; k < K; ++k)
        if (sub == 0 && l + k * L < a.slots) {
            int lo, hi;
            S::offsets(a, l + k * L, lo, hi);
#pragma unroll
            for (int e = 0; e < V; ++e) {
                sums[warp][lo + e] = dw[k][e];
                if (hi + e < a.dim) sums[warp][hi + e] = dw[k][V + e];
            }
        }
    __syncthreads();
    for (int d = threadIdx.x; d < a.dim; d += kRotThreads) {
        float v = 0.f;
#pragma unroll
        for (int j = 0; j < kWarps; ++j) v += sums[j][d];
        a.partial[(int64_t)blockIdx.x * a.dim + d] = v;
    }
}

// The (V, K) pairs that are built: V values of 16, 8, 4 bytes or one value;
// K = 1 slot per lane, or as many as the widest head needs.
template <typename T, bool ILV, typename F>
cudaError_t rot_dispatch(int V, int K, F f) {
    constexpr int W = 16 / (int)sizeof(T);
#define MT_ROT_CASE(v, k)                                                    \
    if (V == v && K == k) return f(std::integral_constant<int, v>{},         \
                                   std::integral_constant<int, k>{});
    if constexpr (W == 8) {
        MT_ROT_CASE(8, 1)
    }
    MT_ROT_CASE(4, 1)
    MT_ROT_CASE(4, 2)
    MT_ROT_CASE(2, 1)
    MT_ROT_CASE(2, 4)
    MT_ROT_CASE(1, 1)
    MT_ROT_CASE(1, 8)
#undef MT_ROT_CASE
    return cudaErrorInvalidValue;
}

template <typename T, bool ILV, bool NORM>
cudaError_t launch_rotary_as(const RotArgs &a, int V, int K, cudaStream_t s) {
    const int64_t units = a.tokens << a.log2S;
    const int64_t grid =
        (units + kRotThreads / 32 - 1) / (kRotThreads / 32);
    return rot_dispatch<T, ILV>(V, K, [&](auto v, auto k) {
        return launch_dependent(
            rotary_kernel<T, decltype(v)::value, decltype(k)::value, ILV,
                          NORM>,
            grid, kRotThreads, 0, s, a);
    });
}

template <typename T>
cudaError_t launch_rotary_any(const RotArgs &a, int V, int K, bool ilv,
                              bool norm, cudaStream_t s) {
    if (ilv)
        return norm ? launch_rotary_as<T, true, true>(a, V, K, s)
                    : launch_rotary_as<T, true, false>(a, V, K, s);
    return norm ? launch_rotary_as<T, false, true>(a, V, K, s)
                : launch_rotary_as<T, false, false>(a, V, K, s);
}

template <typename T, bool ILV>
cudaError_t launch_rotary_backward_as(const RotArgs &a, int V, int K,
                                      cudaStream_t s) {
    return rot_dispatch<T, ILV>(V, K, [&](auto v, auto k) {
        return launch_dependent(
            rotary_backward_kernel<T, decltype(v)::value, decltype(k)::value,
                                   ILV>,
            a.blocks[0] + a.blocks[1], kRotThreads, 0, s, a);
    });
}

#define MT_DEFINE_ROTARY(T, dt)                                              \
    cudaError_t launch_rotary_##dt(const RotArgs &a, int V, int K,           \
                                   bool interleaved, bool norm,              \
                                   cudaStream_t s) {                         \
        return launch_rotary_any<T>(a, V, K, interleaved, norm, s);          \
    }                                                                        \
    cudaError_t launch_rotary_backward_##dt(const RotArgs &a, int V, int K,  \
                                            bool interleaved,                \
                                            cudaStream_t s) {                \
        return interleaved                                                   \
                   ? launch_rotary_backward_as<T, true>(a, V, K, s)          \
                   : launch_rotary_backward_as<T, false>(a, V, K, s);        \
    }

}  // namespace mt

// block_norm.cuh -- the norms around a block with its gate and the residual's
// scale, forward and backward (one translation unit per storage type).
//
// A row stays in the registers of the W threads that share it, K packs of V
// values each, asked for at once: each matrix is read and written once.  The
// forward pass has two sums one after the other (of x^2, and of h^2, which needs
// the first).  So has the backward pass: x^2, h^2 and dy w2 h together, then e w1
// x.  There a CTA goes through many rows, the next one on its way while one is
// worked on, and a thread, which has the same columns in all of them, keeps
// their parts of the weights' and the gate's gradients, in registers, or in
// shared memory where it has 16 columns or more; a second kernel adds up the
// CTAs' in order.
//
// Bound: memory.  BF16 16384 x 4096, both norms and a gate of one row, 93 us, 87%
// of the measured copy bandwidth; backward 8192 x 4096 68 us, 89%.  Rows of 16384
// leave one CTA on an SM, which has nothing on its way while it adds up: 4096 of
// them 125 us, 64%; of 200 columns, 25 lanes of a warp have one pack each: 65536
// rows 24 us, 65%.  Backward, rows of 16384 are past both the kernel with rows
// ahead and the registers (300 bytes spill): 2048 of them 281 us, 22%.
//
// Packs are as wide as every row's address allows.  Rows that 16-byte packs do
// not divide, from 512 columns on, are copied into shared memory with what lies
// around them up to the packs' bounds and read there value by value (one value
// per access of global memory: 12000 x 5001 BF16 350 us for 185, backward 6000 x
// 5001 930 for 184; short rows keep that).  Rows that neither registers nor that hold are gone through in
// loops, once per sum and once to write.
#pragma once

#include "mt_decoder.cuh"

namespace mt {
namespace {

constexpr int kLoop = 512;  // threads of the kernels for any row

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

// V values of a matrix or vector, or the value that stands for an absent one.
template <typename T, int V>
__device__ __forceinline__ void values(const void *p, int64_t i, float absent,
                                       float *v) {
    if (p == nullptr) {
#pragma unroll
        for (int e = 0; e < V; ++e) v[e] = absent;
    } else {
        ld_vec<T, V>(static_cast<const T *>(p) + i, v);
    }
}
template <typename T, int V>
__device__ __forceinline__ void put(void *p, int64_t i, const float *v) {
    st_vec<T, V>(static_cast<T *>(p) + i, v);
}

// Any row: a CTA per row, which reads it once per sum and once to write.
template <typename T, int V>
__global__ void __launch_bounds__(kLoop)
    norm_loop_kernel(const mt_block_norm_call_t c) {
    grid_launch_dependents();
    grid_wait_prerequisites();
    const int64_t r = blockIdx.x;
    const int64_t x = r * c.x_stride, res = r * c.residual_stride;
    const int64_t gate = r * c.gate_stride;
    const bool after = c.norms & MT_NORM_AFTER;
    const bool before = c.norms & MT_NORM_BEFORE;
    const float inv = 1.f / (float)c.cols;
    float r1 = 1.f;
    if (after) {
        float s[1] = {0.f};
        for (int i = threadIdx.x * V; i < c.cols; i += kLoop * V) {
            float v[V];
            values<T, V>(c.x, x + i, 0.f, v);
#pragma unroll
            for (int e = 0; e < V; ++e) s[0] = fmaf(v[e], v[e], s[0]);
        }
        cta_sum(s);
        r1 = rsqrtf(fmaf(s[0], inv, c.eps));
    }
    const auto stream = [&](int i, float *h) {
        float u[V], f[V];
        values<T, V>(c.x, x + i, 0.f, u);
        if (after) {
            values<T, V>(c.weight, i, 1.f, f);
#pragma unroll
            for (int e = 0; e < V; ++e) u[e] = u[e] * r1 * f[e];
        }
        values<T, V>(c.gate, gate + i, 1.f, f);
        values<T, V>(c.residual, res + i, 0.f, h);
#pragma unroll
        for (int e = 0; e < V; ++e)
            h[e] = fmaf(h[e], c.residual_scale, u[e] * f[e]);
    };
    float r2 = 0.f;
    if (before) {
        float s[1] = {0.f};
        for (int i = threadIdx.x * V; i < c.cols; i += kLoop * V) {
            float h[V];
            stream(i, h);
#pragma unroll
            for (int e = 0; e < V; ++e) s[0] = fmaf(h[e], h[e], s[0]);
        }
        cta_sum(s);
        r2 = rsqrtf(fmaf(s[0], inv, c.eps));
    }
    for (int i = threadIdx.x * V; i < c.cols; i += kLoop * V) {
        float h[V], f[V];
        stream(i, h);
        put<T, V>(c.h, r * c.h_stride + i, h);
        if (!before) continue;
        values<T, V>(c.next_weight, i, 1.f, f);
#pragma unroll
        for (int e = 0; e < V; ++e) h[e] = h[e] * r2 * f[e];
        put<T, V>(c.y, r * c.y_stride + i, h);
    }
}

// Any row, backward: a CTA takes every gridDim.x-th row and adds its weights'
// gradients up in shared memory where 3 x cols of them fit (`room`), else in
// its own row of partial sums.
template <typename T, int V>
__global__ void __launch_bounds__(kLoop)
    norm_back_loop_kernel(const mt_block_norm_back_t c, float *partial,
                          int room) {
    extern __shared__ float shared[];
    grid_launch_dependents();
    grid_wait_prerequisites();
    const float inv = 1.f / (float)c.cols;
    const bool after = c.norms & MT_NORM_AFTER;
    const bool before = c.norms & MT_NORM_BEFORE;
    float *own = partial + (int64_t)blockIdx.x * 3 * c.cols;
    float *sums = room ? shared : own;
    if (partial != nullptr)
        for (int i = threadIdx.x; i < 3 * c.cols; i += kLoop) sums[i] = 0.f;
    __syncthreads();
    for (int64_t r = blockIdx.x; r < c.rows; r += gridDim.x) {
        const int64_t x = r * c.x_stride, h = r * c.h_stride;
        const int64_t dy = r * c.dy_stride, gate = r * c.gate_stride;
        float s[3] = {0.f, 0.f, 0.f};
        for (int i = threadIdx.x * V; i < c.cols; i += kLoop * V) {
            float v[V], d[V], f[V];
            if (after) {
                values<T, V>(c.x, x + i, 0.f, v);
#pragma unroll
                for (int e = 0; e < V; ++e) s[0] = fmaf(v[e], v[e], s[0]);
            }
            if (before) {
                values<T, V>(c.h, h + i, 0.f, v);
                values<T, V>(c.dy, dy + i, 0.f, d);
                values<T, V>(c.next_weight, i, 1.f, f);
#pragma unroll
                for (int e = 0; e < V; ++e) {
                    s[1] = fmaf(v[e], v[e], s[1]);
                    s[2] = fmaf(d[e] * f[e], v[e], s[2]);
                }
            }
        }
        cta_sum(s);
        const float r1 = after ? rsqrtf(fmaf(s[0], inv, c.eps)) : 1.f;
        const float r2 = before ? rsqrtf(fmaf(s[1], inv, c.eps)) : 0.f;
        const float m2 = s[2] * inv * r2 * r2;
        // The stream's gradient; dy and h on the way.
        const auto grad = [&](int i, float *g, float *d, float *v) {
            values<T, V>(c.dh, r * c.dh_stride + i, 0.f, g);
            if (!before) return;
            float f[V];
            values<T, V>(c.dy, dy + i, 0.f, d);
            values<T, V>(c.h, h + i, 0.f, v);
            values<T, V>(c.next_weight, i, 1.f, f);
#pragma unroll
            for (int e = 0; e < V; ++e)
                g[e] += r2 * (d[e] * f[e] - v[e] * m2);
        };
        float m1 = 0.f;
        if (after) {
            float t[1] = {0.f};
            for (int i = threadIdx.x * V; i < c.cols; i += kLoop * V) {
                float g[V], d[V], v[V], f[V], w[V];
                grad(i, g, d, v);
                values<T, V>(c.gate, gate + i, 1.f, f);
                values<T, V>(c.weight, i, 1.f, w);
                values<T, V>(c.x, x + i, 0.f, v);
#pragma unroll
                for (int e = 0; e < V; ++e)
                    t[0] = fmaf(g[e] * f[e] * w[e], v[e], t[0]);
            }
            cta_sum(t);
            m1 = t[0] * inv * r1 * r1;
        }
        for (int i = threadIdx.x * V; i < c.cols; i += kLoop * V) {
            float g[V], d[V], v[V], xv[V], f[V], w[V], o[V], dg[V];
            grad(i, g, d, v);
            values<T, V>(c.x, x + i, 0.f, xv);
            values<T, V>(c.weight, i, 1.f, w);
            values<T, V>(c.gate, gate + i, 1.f, f);
            float dx[V];
#pragma unroll
            for (int e = 0; e < V; ++e) {
                dg[e] = g[e] * (xv[e] * r1 * w[e]);
                dx[e] = g[e] * f[e];
                if (c.dgate_sum) sums[i + e] += dg[e];
                if (c.dweight)
                    sums[c.cols + i + e] += dx[e] * xv[e] * r1;
                if (c.dnext_weight)
                    sums[2 * c.cols + i + e] += d[e] * v[e] * r2;
                o[e] = g[e] * c.residual_scale;
                if (after) dx[e] = r1 * (dx[e] * w[e] - xv[e] * m1);
            }
            put<T, V>(c.dx, r * c.dx_stride + i, dx);
            put<T, V>(c.dresidual, r * c.dresidual_stride + i, o);
            if (c.dgate) put<T, V>(c.dgate, r * c.dgate_stride + i, dg);
        }
    }
    if (partial == nullptr || !room) return;
    __syncthreads();
    for (int i = threadIdx.x; i < 3 * c.cols; i += kLoop) own[i] = shared[i];
}

// ---- rows in registers -------------------------------------------------------
// Sums of N values over the W threads of a row: lanes of a warp (W <= 32) or
// the whole CTA; `turn` alternates between two places of the exchange, so that
// one barrier per call is enough.
template <int N>
__device__ __forceinline__ void row_sums(float (&v)[N], int W, int &turn) {
    __shared__ float part[2][N][32];
    if (W <= 32) {
        for (int o = W >> 1; o > 0; o >>= 1)
#pragma unroll
            for (int i = 0; i < N; ++i)
                v[i] += __shfl_xor_sync(kFull, v[i], o);
        return;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] += __shfl_xor_sync(kFull, v[i], o);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int warps = (int)blockDim.x >> 5;
    float (&to)[N][32] = part[turn];
    turn ^= 1;
    if (lane == 0)
#pragma unroll
        for (int i = 0; i < N; ++i) to[i][warp] = v[i];
    __syncthreads();
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = lane < warps ? to[i][lane] : 0.f;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] += __shfl_xor_sync(kFull, v[i], o);
}

// How a row's packs lie: pack k of thread `w` of a row has the columns from
// (w + k W) V on.
struct Lay {
    int W, rows;  // threads of a row, rows of a CTA
};

template <typename T, int V, int K>
struct Packs {
    Raw<T, V> p[K];
    __device__ __forceinline__ void load(const void *m, int64_t at, int w,
                                         int W, int cols, bool on) {
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const int col = (w + k * W) * V;
            if (on && col < cols)
                p[k].load(static_cast<const T *>(m) + at + col);
            else
                p[k].zero();
        }
    }
};
template <typename T, int V>
__device__ __forceinline__ void vector_pack(const void *p, int col, float *v) {
    if (p == nullptr) {
#pragma unroll
        for (int e = 0; e < V; ++e) v[e] = 1.f;
    } else {
        ld_vec<T, V, true>(static_cast<const T *>(p) + col, v);
    }
}

template <typename T, int V, int K>
__global__ void __launch_bounds__(K * V >= 32 ? 512 : 1024)
    norm_kernel(const mt_block_norm_call_t c, const Lay lay) {
    grid_launch_dependents();
    grid_wait_prerequisites();
    const int w = (int)threadIdx.x & (lay.W <= 32 ? lay.W - 1 : ~0);
    const int64_t r = (int64_t)blockIdx.x * lay.rows +
                      (lay.W <= 32 ? (int)threadIdx.x / lay.W : 0);
    const bool on = r < c.rows;
    const bool after = c.norms & MT_NORM_AFTER;
    const bool before = c.norms & MT_NORM_BEFORE;
    const float inv = 1.f / (float)c.cols;
    int turn = 0;
    Packs<T, V, K> x, res;
    x.load(c.x, r * c.x_stride, w, lay.W, c.cols, on);
    res.load(c.residual, r * c.residual_stride, w, lay.W, c.cols, on);
    float r1 = 1.f;
    if (after) {
        float s[1] = {0.f};
#pragma unroll
        for (int k = 0; k < K; ++k) {
            float v[V];
            x.p[k].widen(v);
#pragma unroll
            for (int e = 0; e < V; ++e) s[0] = fmaf(v[e], v[e], s[0]);
        }
        row_sums(s, lay.W, turn);
        r1 = rsqrtf(fmaf(s[0], inv, c.eps));
    }
    float h[K][V];
    float s[1] = {0.f};
#pragma unroll
    for (int k = 0; k < K; ++k) {
        const int col = (w + k * lay.W) * V;
        if (!on || col >= c.cols) continue;
        float u[V], f[V];
        x.p[k].widen(u);
        if (after) {
            vector_pack<T, V>(c.weight, col, f);
#pragma unroll
            for (int e = 0; e < V; ++e) u[e] = u[e] * r1 * f[e];
        }
        if (c.gate != nullptr) {
            vector_pack<T, V>(static_cast<const T *>(c.gate) +
                                  r * c.gate_stride, col, f);
#pragma unroll
            for (int e = 0; e < V; ++e) u[e] *= f[e];
        }
        res.p[k].widen(f);
#pragma unroll
        for (int e = 0; e < V; ++e) {
            h[k][e] = fmaf(f[e], c.residual_scale, u[e]);
            s[0] = fmaf(h[k][e], h[k][e], s[0]);
        }
        st_vec<T, V>(static_cast<T *>(c.h) + r * c.h_stride + col, h[k]);
    }
    if (!before) return;
    row_sums(s, lay.W, turn);
    const float r2 = rsqrtf(fmaf(s[0], inv, c.eps));
#pragma unroll
    for (int k = 0; k < K; ++k) {
        const int col = (w + k * lay.W) * V;
        if (!on || col >= c.cols) continue;
        float f[V];
        vector_pack<T, V>(c.next_weight, col, f);
#pragma unroll
        for (int e = 0; e < V; ++e) h[k][e] = h[k][e] * r2 * f[e];
        st_vec<T, V>(static_cast<T *>(c.y) + r * c.y_stride + col, h[k]);
    }
}

// The matrices of a row of the backward pass.
template <typename T, int V, int K>
struct BackRow {
    Packs<T, V, K> dy, dh, x, h;
    __device__ __forceinline__ void load(const mt_block_norm_back_t &c,
                                         int64_t r, int w, int W) {
        const bool on = r < c.rows;
        if (c.dy) dy.load(c.dy, r * c.dy_stride, w, W, c.cols, on);
        if (c.h) h.load(c.h, r * c.h_stride, w, W, c.cols, on);
        if (c.dh) dh.load(c.dh, r * c.dh_stride, w, W, c.cols, on);
        if (c.x) x.load(c.x, r * c.x_stride, w, W, c.cols, on);
    }
};

// Where a thread's sums of its columns are: registers, or shared memory (value
// i of every thread side by side).
template <int N, bool SHARED>
struct Sums {
    float v[SHARED ? 1 : N];
    float *at;
    __device__ __forceinline__ void begin(float *shared) {
        at = shared + threadIdx.x;
#pragma unroll
        for (int i = 0; i < N; ++i) {
            if constexpr (SHARED) at[i * blockDim.x] = 0.f;
            else v[i] = 0.f;
        }
    }
    __device__ __forceinline__ void add(int i, float d) {
        if constexpr (SHARED) at[i * blockDim.x] += d;
        else v[i] += d;
    }
    __device__ __forceinline__ float get(int i) const {
        if constexpr (SHARED) return at[i * blockDim.x];
        else return v[i];
    }
};

// 16 columns' sums and the rows of a thread do not fit its registers.
__host__ __device__ constexpr bool norm_sums_shared(int columns) {
    return columns >= 16;
}

// The next row is on its way where both fit (8 words of each matrix or less).
template <typename T, int V, int K>
__global__ void __launch_bounds__(512)
    norm_back_kernel(const mt_block_norm_back_t c, const Lay lay,
                     float *partial) {
    constexpr bool kShared = norm_sums_shared(K * V);
    constexpr bool kAhead = Raw<T, V>::kWords * K <= 8;
    extern __shared__ float shared[];
    grid_launch_dependents();
    grid_wait_prerequisites();
    const int w = (int)threadIdx.x & (lay.W <= 32 ? lay.W - 1 : ~0);
    const int group = lay.W <= 32 ? (int)threadIdx.x / lay.W : 0;
    const bool after = c.norms & MT_NORM_AFTER;
    const bool before = c.norms & MT_NORM_BEFORE;
    const float inv = 1.f / (float)c.cols;
    int turn = 0;
    // dgate, dweight, dnext_weight of the thread's columns
    Sums<3 * K * V, kShared> sums;
    if (partial != nullptr) sums.begin(shared);
    BackRow<T, V, K> a, next;
    const int64_t step = (int64_t)gridDim.x * lay.rows;
    int64_t base = (int64_t)blockIdx.x * lay.rows;
    if (kAhead) next.load(c, base + group, w, lay.W);
    for (; base < c.rows; base += step) {
        const int64_t r = base + group;
        const bool on = r < c.rows;
        if (kAhead) {
            a = next;
            next.load(c, r + step, w, lay.W);
        } else {
            a.load(c, r, w, lay.W);
        }
        float s[3] = {0.f, 0.f, 0.f};
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const int col = (w + k * lay.W) * V;
            if (!on || col >= c.cols) continue;
            if (after) {
                float v[V];
                a.x.p[k].widen(v);
#pragma unroll
                for (int e = 0; e < V; ++e) s[0] = fmaf(v[e], v[e], s[0]);
            }
            if (before) {
                float v[V], d[V], f[V];
                a.h.p[k].widen(v);
                a.dy.p[k].widen(d);
                vector_pack<T, V>(c.next_weight, col, f);
#pragma unroll
                for (int e = 0; e < V; ++e) {
                    s[1] = fmaf(v[e], v[e], s[1]);
                    s[2] = fmaf(d[e] * f[e], v[e], s[2]);
                }
            }
        }
        row_sums(s, lay.W, turn);
        const float r1 = after ? rsqrtf(fmaf(s[0], inv, c.eps)) : 1.f;
        const float r2 = before ? rsqrtf(fmaf(s[1], inv, c.eps)) : 0.f;
        const float m2 = s[2] * inv * r2 * r2;
        float g[K][V];
        float t[1] = {0.f};
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const int col = (w + k * lay.W) * V;
            if (!on || col >= c.cols) continue;
            float x[V];
            if (c.dh != nullptr) {
                a.dh.p[k].widen(g[k]);
            } else {
#pragma unroll
                for (int e = 0; e < V; ++e) g[k][e] = 0.f;
            }
            if (before) {
                float v[V], d[V], f[V];
                a.h.p[k].widen(v);
                a.dy.p[k].widen(d);
                vector_pack<T, V>(c.next_weight, col, f);
#pragma unroll
                for (int e = 0; e < V; ++e)
                    g[k][e] += r2 * (d[e] * f[e] - v[e] * m2);
                if (c.dnext_weight != nullptr) {
#pragma unroll
                    for (int e = 0; e < V; ++e)
                        sums.add((2 * K + k) * V + e, d[e] * v[e] * r2);
                }
            }
            // outputs may lie on inputs: nothing is written before the gate is
            // read
            float o[V], down[V];
#pragma unroll
            for (int e = 0; e < V; ++e) down[e] = g[k][e] * c.residual_scale;
            if (c.x != nullptr) a.x.p[k].widen(x);
            if (c.gate != nullptr) {
                float f[V];
                if (c.dgate != nullptr || c.dgate_sum != nullptr) {
                    vector_pack<T, V>(c.weight, col, f);
#pragma unroll
                    for (int e = 0; e < V; ++e)
                        o[e] = g[k][e] * (x[e] * r1 * f[e]);
                    if (c.dgate_sum != nullptr) {
#pragma unroll
                        for (int e = 0; e < V; ++e) sums.add(k * V + e, o[e]);
                    }
                }
                vector_pack<T, V>(static_cast<const T *>(c.gate) +
                                      r * c.gate_stride, col, f);
#pragma unroll
                for (int e = 0; e < V; ++e) g[k][e] *= f[e];
                if (c.dgate != nullptr)
                    st_vec<T, V>(static_cast<T *>(c.dgate) +
                                     r * c.dgate_stride + col, o);
            }
            st_vec<T, V>(static_cast<T *>(c.dresidual) +
                             r * c.dresidual_stride + col, down);
            if (after) {
                float f[V];
                vector_pack<T, V>(c.weight, col, f);
#pragma unroll
                for (int e = 0; e < V; ++e) {
                    if (c.dweight != nullptr)
                        sums.add((K + k) * V + e, g[k][e] * x[e] * r1);
                    g[k][e] *= f[e];
                    t[0] = fmaf(g[k][e], x[e], t[0]);
                }
            }
        }
        float m1 = 0.f;
        if (after) {
            row_sums(t, lay.W, turn);
            m1 = t[0] * inv * r1 * r1;
        }
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const int col = (w + k * lay.W) * V;
            if (!on || col >= c.cols) continue;
            if (after) {
                float x[V];
                a.x.p[k].widen(x);
#pragma unroll
                for (int e = 0; e < V; ++e)
                    g[k][e] = r1 * (g[k][e] - x[e] * m1);
            }
            st_vec<T, V>(static_cast<T *>(c.dx) + r * c.dx_stride + col, g[k]);
        }
    }
    if (partial == nullptr) return;
    // Groups of a CTA's rows one after the other, then the CTA's row of sums.
    float *to = partial + (int64_t)blockIdx.x * 3 * c.cols;
#pragma unroll 1
    for (int q = 0; q < lay.rows; ++q) {
        if (q == group) {
#pragma unroll
            for (int i = 0; i < 3; ++i)
#pragma unroll
                for (int k = 0; k < K; ++k)
#pragma unroll
                    for (int e = 0; e < V; ++e) {
                        const int col = (w + k * lay.W) * V + e;
                        if (col >= c.cols) continue;
                        float &p = to[(int64_t)i * c.cols + col];
                        const float v = sums.get((i * K + k) * V + e);
                        p = q == 0 ? v : p + v;
                    }
        }
        __syncthreads();
    }
}

// The same for rows of whole 16-byte packs, with the rows on their way in shared
// memory: each thread copies and reads its own packs (no barrier), two rows
// ahead.  Its columns' weights stay widened, arithmetic goes in pairs, and a
// gate of one row and the weight have one sum between them, A = sum of g x r1:
// dgate = weight A, dweight = gate A.  Packs past the row's end are zeros, which
// add nothing; only what is stored is guarded.
//
// Bound by instructions: some 25 for a value.  BF16 8192 x 4096 with one gate
// and both weights 68 us, where the kernel that widened everything for each row
// took 135.
__device__ __forceinline__ void copy_pack(void *to, const void *from,
                                          bool on) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(
                     smem_addr(to)),
                 "l"(from), "r"(on ? 16 : 0)
                 : "memory");
}
constexpr int kAheadRows = 2;
enum { GATE_NONE, GATE_ROW, GATE_MATRIX };
// Threads of a CTA: 256, two CTAs to an SM, where a row needs no more.
template <typename T, int K, int THREADS, int NORMS, int GATE>
__global__ void __launch_bounds__(THREADS, 512 / THREADS)
    norm_back_ahead_kernel(const mt_block_norm_back_t c, const Lay lay,
                           float *partial) {
    constexpr int V = 16 / (int)sizeof(T);
    constexpr bool after = NORMS & MT_NORM_AFTER;
    constexpr bool before = NORMS & MT_NORM_BEFORE;
    constexpr int kMatrices = GATE == GATE_MATRIX ? 5 : 4;
    extern __shared__ __align__(16) uint4 packs[];
    grid_wait_prerequisites();
    const int w = (int)threadIdx.x & (lay.W <= 32 ? lay.W - 1 : ~0);
    const int group = lay.W <= 32 ? (int)threadIdx.x / lay.W : 0;
    const float inv = 1.f / (float)c.cols;
    int turn = 0;
    enum { DY, DH, X, H, G };
    // pack k of matrix m of the row in place `stage`
    const auto pack = [&](int stage, int m, int k) -> uint4 * {
        return packs + ((stage * kMatrices + m) * K + k) * blockDim.x +
               threadIdx.x;
    };
    const auto load = [&](int64_t r, int stage) {
        const bool on = r < c.rows;
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const int col = (w + k * lay.W) * V;
            const bool in = on && col < c.cols;
            const auto one = [&](const void *m, int64_t stride, int which) {
                copy_pack(pack(stage, which, k),
                          static_cast<const T *>(m) +
                              (in ? r * stride + col : 0), in);
            };
            if (before) one(c.dy, c.dy_stride, DY);
            if (before) one(c.h, c.h_stride, H);
            if (after || GATE != GATE_NONE) one(c.x, c.x_stride, X);
            if (c.dh != nullptr) one(c.dh, c.dh_stride, DH);
            if (GATE == GATE_MATRIX) one(c.gate, c.gate_stride, G);
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
    const auto get = [&](int stage, int m, int k, float *v) {
        ld_vec<T, V>(reinterpret_cast<const T *>(pack(stage, m, k)), v);
    };
    // next_weight; weight times a gate of one row.
    float w2[K][V], wg[K][V], shared_sum[K][V], next_sum[K][V];
#pragma unroll
    for (int k = 0; k < K; ++k) {
        const int col = (w + k * lay.W) * V;
        float f[V];
        const bool in = col < c.cols;
        vector_pack<T, V>(in ? c.next_weight : nullptr, in ? col : 0, w2[k]);
        vector_pack<T, V>(in ? c.weight : nullptr, in ? col : 0, wg[k]);
        vector_pack<T, V>(in && GATE == GATE_ROW ? c.gate : nullptr,
                          in ? col : 0, f);
        mul_n<V>(wg[k], wg[k], f);
#pragma unroll
        for (int e = 0; e < V; ++e) shared_sum[k][e] = next_sum[k][e] = 0.f;
        if (c.dh == nullptr)
#pragma unroll
            for (int i = 0; i < kAheadRows; ++i)
                *pack(i, DH, k) = make_uint4(0, 0, 0, 0);
    }
    const int64_t step = (int64_t)gridDim.x * lay.rows;
    int64_t base = (int64_t)blockIdx.x * lay.rows;
#pragma unroll
    for (int i = 0; i < kAheadRows; ++i) load(base + group + i * step, i);
    int stage = 0;
#pragma unroll 1
    for (; base < c.rows; base += step) {
        const int64_t r = base + group;
        const bool on = r < c.rows;
        asm volatile("cp.async.wait_group %0;" ::"n"(kAheadRows - 1)
                     : "memory");
        float r1 = 1.f, r2 = 0.f, m2 = 0.f;
        if (after || before) {
            float2 q[3] = {};
#pragma unroll
            for (int k = 0; k < K; ++k) {
                float v[V], d[V];
                if (after) {
                    get(stage, X, k, v);
#pragma unroll
                    for (int e = 0; e < V; e += 2) {
                        const float2 p = make_float2(v[e], v[e + 1]);
                        q[0] = fma2(p, p, q[0]);
                    }
                }
                if (before) {
                    get(stage, H, k, v);
                    get(stage, DY, k, d);
                    mul_n<V>(d, d, w2[k]);
#pragma unroll
                    for (int e = 0; e < V; e += 2) {
                        const float2 p = make_float2(v[e], v[e + 1]);
                        q[1] = fma2(p, p, q[1]);
                        q[2] = fma2(make_float2(d[e], d[e + 1]), p, q[2]);
                    }
                }
            }
            float s[3];
#pragma unroll
            for (int i = 0; i < 3; ++i) s[i] = q[i].x + q[i].y;
            row_sums(s, lay.W, turn);
            if (after) r1 = rsqrtf(fmaf(s[0], inv, c.eps));
            if (before) r2 = rsqrtf(fmaf(s[1], inv, c.eps));
            m2 = s[2] * inv * r2 * r2;
            if (!on) r1 = r2 = m2 = 0.f;
        }
        float g[K][V];
        float2 t2 = make_float2(0.f, 0.f);
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const int col = (w + k * lay.W) * V;
            const bool in = on && col < c.cols;
            float x[V], f[V], o[V];
            get(stage, DH, k, g[k]);
            if (before) {
                float v[V], d[V];
                get(stage, H, k, v);
                get(stage, DY, k, d);
                mul_n<V>(o, d, w2[k]);
                scale_add_n<V>(o, v, -m2, o);
                scale_add_n<V>(g[k], o, r2, g[k]);
                scale_n<V>(v, v, r2);
                fma_n<V>(next_sum[k], d, v, next_sum[k]);
            }
            if (after || GATE != GATE_NONE) {
                get(stage, X, k, x);
                scale_n<V>(f, x, r1);     // x r1
            }
            if (in) {
                scale_n<V>(o, g[k], c.residual_scale);
                st_vec<T, V>(static_cast<T *>(c.dresidual) +
                                 r * c.dresidual_stride + col, o);
            }
            if (GATE == GATE_MATRIX) {
                float gate[V];
                get(stage, G, k, gate);
                mul_n<V>(o, g[k], f);
                mul_n<V>(o, o, wg[k]);
                if (in)
                    st_vec<T, V>(static_cast<T *>(c.dgate) +
                                     r * c.dgate_stride + col, o);
                mul_n<V>(g[k], g[k], gate);
            }
            if (after || GATE == GATE_ROW)
                fma_n<V>(shared_sum[k], g[k], f, shared_sum[k]);
            mul_n<V>(g[k], g[k], wg[k]);
            if (after) {
#pragma unroll
                for (int e = 0; e < V; e += 2)
                    t2 = fma2(make_float2(g[k][e], g[k][e + 1]),
                              make_float2(x[e], x[e + 1]), t2);
            }
        }
        float m1 = 0.f;
        if (after) {
            float t[1] = {t2.x + t2.y};
            row_sums(t, lay.W, turn);
            m1 = t[0] * inv * r1 * r1;
        }
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const int col = (w + k * lay.W) * V;
            if (after) {
                float x[V];
                get(stage, X, k, x);
                scale_add_n<V>(g[k], x, -m1, g[k]);
                scale_n<V>(g[k], g[k], r1);
            }
            if (on && col < c.cols)
                st_vec<T, V>(static_cast<T *>(c.dx) + r * c.dx_stride + col,
                             g[k]);
        }
        load(r + kAheadRows * step, stage);
        stage = stage + 1 == kAheadRows ? 0 : stage + 1;
    }
    asm volatile("cp.async.wait_group 0;" ::: "memory");
    grid_launch_dependents();
    if (partial == nullptr) return;
    // Groups of a CTA's rows one after the other, then the CTA's row of sums.
    float *to = partial + (int64_t)blockIdx.x * 3 * c.cols;
#pragma unroll 1
    for (int q = 0; q < lay.rows; ++q) {
        if (q == group) {
#pragma unroll
            for (int k = 0; k < K; ++k) {
                const int col = (w + k * lay.W) * V;
                if (col >= c.cols) continue;
                float f[V], u[V];
                vector_pack<T, V>(c.weight, col, u);
                vector_pack<T, V>(GATE == GATE_ROW ? c.gate : nullptr, col, f);
                mul_n<V>(u, u, shared_sum[k]);
                mul_n<V>(f, f, shared_sum[k]);
                const float *v[3] = {u, f, next_sum[k]};
#pragma unroll
                for (int i = 0; i < 3; ++i)
#pragma unroll
                    for (int e = 0; e < V; e += 4) {
                        float4 *p = reinterpret_cast<float4 *>(
                            to + (int64_t)i * c.cols + col + e);
                        float4 a = make_float4(v[i][e], v[i][e + 1],
                                               v[i][e + 2], v[i][e + 3]);
                        if (q != 0) {
                            const float4 b = *p;
                            a.x += b.x; a.y += b.y; a.z += b.z; a.w += b.w;
                        }
                        *p = a;
                    }
            }
        }
        __syncthreads();
    }
}

// ---- rows off the packs' bounds ----------------------------------------------
// A CTA goes through many rows, the next one on its way where there is room for
// two (`places`); a thread has every THREADS-th column of all of them, K at
// most, and its weights in registers.
//
// A row in shared memory: its place among 16-byte packs is kept, so that whole
// packs can be copied (the first of them with the end of the row before it, of
// the last one only what is the row's).
template <typename T>
struct OddRow {
    const uint8_t *at;  // the row's first value
    template <int THREADS>
    __device__ __forceinline__ void load(uint8_t *to, const void *m,
                                         int64_t row, int64_t stride,
                                         int cols) const {
        const uintptr_t first = reinterpret_cast<uintptr_t>(m) +
                                (uintptr_t)(row * stride) * sizeof(T);
        const unsigned shift = (unsigned)(first & 15);
        const unsigned bytes = (unsigned)cols * (unsigned)sizeof(T);
        for (unsigned j = threadIdx.x * 16; j < shift + bytes;
             j += THREADS * 16) {
            const uintptr_t from = first - shift + j;
            if (j == 0 && row == 0 && shift != 0) {
                // nothing of the matrix before it: value by value
                for (unsigned b = shift; b < 16 && b < shift + bytes;
                     b += sizeof(T))
                    *reinterpret_cast<T *>(to + b) =
                        *reinterpret_cast<const T *>(from + b);
                continue;
            }
            const unsigned left = shift + bytes - j;
            asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(
                             smem_addr(to + j)),
                         "l"(from), "r"(left < 16 ? left : 16u)
                         : "memory");
        }
    }
    __device__ __forceinline__ void begin(const uint8_t *region, const void *m,
                                          int64_t row, int64_t stride) {
        at = region + ((reinterpret_cast<uintptr_t>(m) +
                        (uintptr_t)(row * stride) * sizeof(T)) & 15);
    }
    __device__ __forceinline__ float operator[](int col) const {
        return to_f(reinterpret_cast<const T *>(at)[col]);
    }
};

template <typename T, int K, int THREADS>
__global__ void __launch_bounds__(THREADS, 1024 / THREADS)
    norm_odd_kernel(const mt_block_norm_call_t c, int region, int places) {
    extern __shared__ __align__(16) uint8_t rows[];
    grid_wait_prerequisites();
    const bool after = c.norms & MT_NORM_AFTER;
    const bool before = c.norms & MT_NORM_BEFORE;
    const bool wide = c.gate != nullptr && c.gate_stride != 0;
    const float inv = 1.f / (float)c.cols;
    const int tid = threadIdx.x;
    int turn = 0;
    float wg[K], w2[K];  // weight times a gate of one row; next_weight
#pragma unroll
    for (int k = 0; k < K; ++k) {
        const int col = tid + k * THREADS;
        const bool in = col < c.cols;
        wg[k] = in ? param_at(static_cast<const T *>(c.weight), col, 1.f) : 1.f;
        if (in && !wide)
            wg[k] *= param_at(static_cast<const T *>(c.gate), col, 1.f);
        w2[k] = in ? param_at(static_cast<const T *>(c.next_weight), col, 1.f)
                   : 1.f;
    }
    OddRow<T> x, res, gate;
    const auto load = [&](int64_t r, int stage) {
        uint8_t *to = rows + stage * 3 * region;
        if (r < c.rows) {
            x.template load<THREADS>(to, c.x, r, c.x_stride, c.cols);
            res.template load<THREADS>(to + region, c.residual, r,
                                       c.residual_stride, c.cols);
            if (wide)
                gate.template load<THREADS>(to + 2 * region, c.gate, r,
                                            c.gate_stride, c.cols);
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
    int stage = 0;
    if (places == 2) load(blockIdx.x, 0);
#pragma unroll 1
    for (int64_t r = blockIdx.x; r < c.rows; r += gridDim.x) {
        if (places == 1) {
            __syncthreads();  // the row before is done with
            load(r, 0);
        }
        asm volatile("cp.async.wait_group 0;" ::: "memory");
        __syncthreads();  // this row is there, the one before is done with
        if (places == 2) {
            stage ^= 1;
            load(r + gridDim.x, stage);
        }
        const uint8_t *from = rows + (stage ^ (places - 1)) * 3 * region;
        x.begin(from, c.x, r, c.x_stride);
        res.begin(from + region, c.residual, r, c.residual_stride);
        gate.begin(from + 2 * region, c.gate, r, c.gate_stride);
        float h[K];
        float s[1] = {0.f};
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const int col = tid + k * THREADS;
            h[k] = col < c.cols ? x[col] : 0.f;
            s[0] = fmaf(h[k], h[k], s[0]);
        }
        float r1 = 1.f;
        if (after) {
            row_sums(s, THREADS, turn);
            r1 = rsqrtf(fmaf(s[0], inv, c.eps));
        }
        s[0] = 0.f;
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const int col = tid + k * THREADS;
            if (col >= c.cols) continue;
            float u = h[k] * r1 * wg[k];
            if (wide) u *= gate[col];
            h[k] = fmaf(res[col], c.residual_scale, u);
            s[0] = fmaf(h[k], h[k], s[0]);
            static_cast<T *>(c.h)[r * c.h_stride + col] = from_f<T>(h[k]);
        }
        if (!before) continue;
        row_sums(s, THREADS, turn);
        const float r2 = rsqrtf(fmaf(s[0], inv, c.eps));
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const int col = tid + k * THREADS;
            if (col < c.cols)
                static_cast<T *>(c.y)[r * c.y_stride + col] =
                    from_f<T>(h[k] * r2 * w2[k]);
        }
    }
    grid_launch_dependents();
}

template <typename T, int K, int THREADS>
__global__ void __launch_bounds__(THREADS, 512 / THREADS)
    norm_back_odd_kernel(const mt_block_norm_back_t c, float *partial,
                         int region, int places) {
    extern __shared__ __align__(16) uint8_t rows[];
    grid_wait_prerequisites();
    const bool after = c.norms & MT_NORM_AFTER;
    const bool before = c.norms & MT_NORM_BEFORE;
    const bool wide = c.dgate != nullptr;
    const bool takes_x = after || c.gate != nullptr;
    const float inv = 1.f / (float)c.cols;
    const int tid = threadIdx.x;
    int turn = 0;
    float wg[K], w2[K], shared_sum[K], next_sum[K];
#pragma unroll
    for (int k = 0; k < K; ++k) {
        const int col = tid + k * THREADS;
        const bool in = col < c.cols;
        wg[k] = in ? param_at(static_cast<const T *>(c.weight), col, 1.f) : 1.f;
        if (in && !wide)
            wg[k] *= param_at(static_cast<const T *>(c.gate), col, 1.f);
        w2[k] = in ? param_at(static_cast<const T *>(c.next_weight), col, 1.f)
                   : 1.f;
        shared_sum[k] = next_sum[k] = 0.f;
    }
    OddRow<T> dy, dh, x, h, gate;
    const auto load = [&](int64_t r, int stage) {
        uint8_t *to = rows + stage * 5 * region;
        if (r < c.rows) {
            const auto one = [&](const OddRow<T> &m, const void *p,
                                 int64_t stride, int i) {
                m.template load<THREADS>(to + i * region, p, r, stride,
                                         c.cols);
            };
            if (before) one(dy, c.dy, c.dy_stride, 0);
            if (before) one(h, c.h, c.h_stride, 1);
            if (takes_x) one(x, c.x, c.x_stride, 2);
            if (c.dh) one(dh, c.dh, c.dh_stride, 3);
            if (wide) one(gate, c.gate, c.gate_stride, 4);
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
    int stage = 0;
    if (places == 2) load(blockIdx.x, 0);
#pragma unroll 1
    for (int64_t r = blockIdx.x; r < c.rows; r += gridDim.x) {
        if (places == 1) {
            __syncthreads();  // the row before is done with
            load(r, 0);
        }
        asm volatile("cp.async.wait_group 0;" ::: "memory");
        __syncthreads();  // this row is there, the one before is done with
        if (places == 2) {
            stage ^= 1;
            load(r + gridDim.x, stage);
        }
        const uint8_t *from = rows + (stage ^ (places - 1)) * 5 * region;
        dy.begin(from, c.dy, r, c.dy_stride);
        h.begin(from + region, c.h, r, c.h_stride);
        x.begin(from + 2 * region, c.x, r, c.x_stride);
        dh.begin(from + 3 * region, c.dh, r, c.dh_stride);
        gate.begin(from + 4 * region, c.gate, r, c.gate_stride);
        float s[3] = {0.f, 0.f, 0.f};
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const int col = tid + k * THREADS;
            if (col >= c.cols) continue;
            if (after) s[0] = fmaf(x[col], x[col], s[0]);
            if (before) {
                const float v = h[col];
                s[1] = fmaf(v, v, s[1]);
                s[2] = fmaf(dy[col] * w2[k], v, s[2]);
            }
        }
        row_sums(s, THREADS, turn);
        const float r1 = after ? rsqrtf(fmaf(s[0], inv, c.eps)) : 1.f;
        const float r2 = before ? rsqrtf(fmaf(s[1], inv, c.eps)) : 0.f;
        const float m2 = s[2] * inv * r2 * r2;
        float g[K];
        float t[1] = {0.f};
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const int col = tid + k * THREADS;
            if (col >= c.cols) continue;
            g[k] = c.dh ? dh[col] : 0.f;
            if (before) {
                const float d = dy[col], v = h[col];
                g[k] = fmaf(r2, fmaf(-v, m2, d * w2[k]), g[k]);
                next_sum[k] = fmaf(d, v * r2, next_sum[k]);
            }
            // outputs may lie on inputs: the row itself is in shared memory
            static_cast<T *>(c.dresidual)[r * c.dresidual_stride + col] =
                from_f<T>(g[k] * c.residual_scale);
            if (!takes_x) continue;
            const float v = x[col], u = v * r1;
            if (wide) {
                static_cast<T *>(c.dgate)[r * c.dgate_stride + col] =
                    from_f<T>(g[k] * u * wg[k]);
                g[k] *= gate[col];
            }
            shared_sum[k] = fmaf(g[k], u, shared_sum[k]);
            g[k] *= wg[k];
            t[0] = fmaf(g[k], v, t[0]);
        }
        float m1 = 0.f;
        if (after) {
            row_sums(t, THREADS, turn);
            m1 = t[0] * inv * r1 * r1;
        }
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const int col = tid + k * THREADS;
            if (col >= c.cols) continue;
            if (after) g[k] = r1 * fmaf(-x[col], m1, g[k]);
            static_cast<T *>(c.dx)[r * c.dx_stride + col] = from_f<T>(g[k]);
        }
    }
    grid_launch_dependents();
    if (partial == nullptr) return;
    float *to = partial + (int64_t)blockIdx.x * 3 * c.cols;
#pragma unroll
    for (int k = 0; k < K; ++k) {
        const int col = tid + k * THREADS;
        if (col >= c.cols) continue;
        to[col] = shared_sum[k] *
                  param_at(static_cast<const T *>(c.weight), col, 1.f);
        to[c.cols + col] =
            shared_sum[k] *
            (wide ? 1.f : param_at(static_cast<const T *>(c.gate), col, 1.f));
        to[2 * c.cols + col] = next_sum[k];
    }
}

// Bytes of a row's place in shared memory.
inline int odd_region(int cols, int es) {
    return (int)(((int64_t)cols * es + 15 + 15) / 16 * 16);
}
// Whether a matrix's rows follow one another, so that what lies before a row
// but the first is the matrix's too.
inline bool odd_ok(const void *p, int64_t stride, int64_t rows, int cols) {
    return p == nullptr || rows <= 1 || stride >= cols;
}
constexpr int kOddFrom = 512, kOddMost = 8192;

// Threads per row and rows per CTA for K packs of V values.
inline Lay lay_of(int cols, int V, int K, int small) {
    const int packs = (cols + V - 1) / V;
    const int need = (packs + K - 1) / K;
    Lay l;
    if (need <= 32) {
        l.W = 1;
        while (l.W < need) l.W *= 2;
        l.rows = small / l.W;
    } else {
        l.W = (need + 31) / 32 * 32;
        l.rows = 1;
    }
    return l;
}

template <typename T, int V, int K>
cudaError_t norm_launch(const mt_block_norm_call_t &c, cudaStream_t s) {
    const Lay l = lay_of(c.cols, V, K, 128);
    return launch_dependent(norm_kernel<T, V, K>,
                            (c.rows + l.rows - 1) / l.rows, l.W * l.rows, 0, s,
                            c, l);
}

template <typename T, int K, int THREADS>
cudaError_t norm_odd(const mt_block_norm_call_t &c, cudaStream_t s) {
    const auto kernel = norm_odd_kernel<T, K, THREADS>;
    const int region = odd_region(c.cols, sizeof(T));
    const int places = (int64_t)6 * region <= 200 * 1024 ? 2 : 1;
    const size_t smem = (size_t)places * 3 * region;
    int sms = 0;
    cudaError_t e = current_sm_count(&sms);
    if (e == cudaSuccess && smem > 40 * 1024)
        e = allow_max_smem(reinterpret_cast<const void *>(kernel));
    if (e != cudaSuccess) return e;
    int64_t grid = (int64_t)sms * (1024 / THREADS);
    const int64_t fit = 220 * 1024 / (int64_t)(smem + 2048);
    if (grid > sms * fit) grid = sms * fit;
    if (grid > c.rows) grid = c.rows;
    return launch_dependent(kernel, grid, THREADS, smem, s, c, region, places);
}

template <typename T, int V>
cudaError_t norm_packs(const mt_block_norm_call_t &c, cudaStream_t s) {
    const int packs = (c.cols + V - 1) / V;
    if constexpr (V * sizeof(T) < 16) {
        if (c.cols >= kOddFrom && c.cols <= kOddMost &&
            odd_ok(c.x, c.x_stride, c.rows, c.cols) &&
            odd_ok(c.residual, c.residual_stride, c.rows, c.cols) &&
            (c.gate_stride == 0 ||
             odd_ok(c.gate, c.gate_stride, c.rows, c.cols)))
            return c.cols <= 1024   ? norm_odd<T, 4, 256>(c, s)
                   : c.cols <= 2048 ? norm_odd<T, 8, 256>(c, s)
                   : c.cols <= 4096 ? norm_odd<T, 8, 512>(c, s)
                                    : norm_odd<T, 16, 512>(c, s);
    }
    if (packs <= 256) return norm_launch<T, V, 1>(c, s);
    if (packs <= 1024) return norm_launch<T, V, 2>(c, s);
    if (packs <= 2048) return norm_launch<T, V, 4>(c, s);
    if constexpr (V < 8)
        if (packs <= 4096) return norm_launch<T, V, 8>(c, s);
    if constexpr (V == 1)
        if (packs <= 8192) return norm_launch<T, V, 16>(c, s);
    return launch_dependent(norm_loop_kernel<T, V>, c.rows, kLoop, 0, s, c);
}

template <typename T>
cudaError_t norm_as(const mt_block_norm_call_t &c, int V, cudaStream_t s) {
    if constexpr (sizeof(T) == 2)
        if (V == 8) return norm_packs<T, 8>(c, s);
    if (V >= 4) return norm_packs<T, 4>(c, s);
    if (V >= 2) return norm_packs<T, 2>(c, s);
    return norm_packs<T, 1>(c, s);
}

// CTAs of the backward pass that share an SM: as many as 128 registers per
// thread and the sums in shared memory allow, two at most (each leaves a row
// of partial sums).
inline int back_grid(int64_t rows, int threads, size_t smem, int sms) {
    const int per_sm = threads <= 256 && smem <= 100 * 1024 ? 2 : 1;
    int64_t grid = (int64_t)sms * per_sm;
    if (grid > kNormBackBlocks) grid = kNormBackBlocks;
    return (int)(grid < rows ? grid : rows);
}

template <typename T, int V, int K>
cudaError_t norm_back_launch(const mt_block_norm_back_t &c, float *partial,
                             int *blocks, cudaStream_t s) {
    const Lay l = lay_of(c.cols, V, K, 256);
    const int threads = l.W * l.rows;
    const auto kernel = norm_back_kernel<T, V, K>;
    size_t smem = 0;
    int sms = 0;
    cudaError_t e = current_sm_count(&sms);
    if (norm_sums_shared(K * V) && partial != nullptr) {
        smem = (size_t)3 * K * V * threads * sizeof(float);
        if (smem > 40 * 1024 && e == cudaSuccess)
            e = allow_max_smem(reinterpret_cast<const void *>(kernel));
    }
    if (e != cudaSuccess) return e;
    *blocks = back_grid((c.rows + l.rows - 1) / l.rows, threads, smem, sms);
    return launch_dependent(kernel, *blocks, threads, smem, s, c, l, partial);
}

inline int back_grid_of(int64_t rows, int cols, int64_t grid) {
    if (grid > norm_back_blocks(cols)) grid = norm_back_blocks(cols);
    return (int)(grid < rows ? grid : rows);
}
template <typename T, int K, int THREADS, int NORMS, int GATE>
cudaError_t norm_back_ahead_as(const mt_block_norm_back_t &c, float *partial,
                               int *blocks, cudaStream_t s) {
    constexpr int V = 16 / (int)sizeof(T);
    const Lay l = lay_of(c.cols, V, K, 256);
    const int threads = l.W * l.rows;
    const auto kernel = norm_back_ahead_kernel<T, K, THREADS, NORMS, GATE>;
    const size_t smem = (size_t)kAheadRows * (GATE == GATE_MATRIX ? 5 : 4) *
                        K * 16 * threads;
    int sms = 0;
    cudaError_t e = current_sm_count(&sms);
    if (e == cudaSuccess && smem > 40 * 1024)
        e = allow_max_smem(reinterpret_cast<const void *>(kernel));
    if (e != cudaSuccess) return e;
    int64_t grid = (int64_t)sms * (512 / THREADS);
    const int64_t need = (c.rows + l.rows - 1) / l.rows;
    if (grid > kNormBackBlocks) grid = kNormBackBlocks;
    if (grid > need) grid = need;
    *blocks = (int)grid;
    return launch_dependent(kernel, grid, threads, smem, s, c, l, partial);
}
template <typename T, int K, int THREADS>
cudaError_t norm_back_ahead(const mt_block_norm_back_t &c, float *partial,
                            int *blocks, cudaStream_t s) {
    const int gate = c.gate == nullptr     ? GATE_NONE
                     : c.dgate == nullptr ? GATE_ROW : GATE_MATRIX;
#define MT_NORM_AHEAD(n, g)                                                  \
    if (c.norms == n && gate == g)                                           \
        return norm_back_ahead_as<T, K, THREADS, n, g>(c, partial, blocks, s);
    MT_NORM_AHEAD(1, GATE_NONE)
    MT_NORM_AHEAD(1, GATE_ROW)
    MT_NORM_AHEAD(1, GATE_MATRIX)
    MT_NORM_AHEAD(2, GATE_NONE)
    MT_NORM_AHEAD(2, GATE_ROW)
    MT_NORM_AHEAD(2, GATE_MATRIX)
    MT_NORM_AHEAD(3, GATE_NONE)
    MT_NORM_AHEAD(3, GATE_ROW)
    MT_NORM_AHEAD(3, GATE_MATRIX)
#undef MT_NORM_AHEAD
    return cudaErrorInvalidValue;
}

template <typename T, int K, int THREADS>
cudaError_t norm_back_odd(const mt_block_norm_back_t &c, float *partial,
                          int *blocks, cudaStream_t s) {
    const auto kernel = norm_back_odd_kernel<T, K, THREADS>;
    const int region = odd_region(c.cols, sizeof(T));
    const int places = (int64_t)10 * region <= 200 * 1024 ? 2 : 1;
    const size_t smem = (size_t)places * 5 * region;
    int sms = 0;
    cudaError_t e = current_sm_count(&sms);
    if (e == cudaSuccess && smem > 40 * 1024)
        e = allow_max_smem(reinterpret_cast<const void *>(kernel));
    if (e != cudaSuccess) return e;
    // 62, 80 and 112 registers for 4, 8 and 16 columns
    int per_sm = THREADS == 512 ? 1 : K == 4 ? 4 : K == 8 ? 3 : 2;
    while (per_sm > 1 && per_sm * (smem + 2048) > 228 * 1024) --per_sm;
    *blocks = back_grid_of(c.rows, c.cols, (int64_t)sms * per_sm);
    return launch_dependent(kernel, *blocks, THREADS, smem, s, c, partial,
                            region, places);
}

template <typename T, int V>
cudaError_t norm_back_packs(const mt_block_norm_back_t &c, float *partial,
                            int *blocks, cudaStream_t s) {
    constexpr int kWords = Raw<T, V>::kWords;  // of a pack
    const int packs = (c.cols + V - 1) / V;
    if (V * sizeof(T) < 16 && c.cols >= kOddFrom && c.cols <= kOddMost &&
        gate_plain(c) &&
        odd_ok(c.dy, c.dy_stride, c.rows, c.cols) &&
        odd_ok(c.dh, c.dh_stride, c.rows, c.cols) &&
        odd_ok(c.x, c.x_stride, c.rows, c.cols) &&
        odd_ok(c.h, c.h_stride, c.rows, c.cols) &&
        (c.dgate == nullptr ||
         odd_ok(c.gate, c.gate_stride, c.rows, c.cols))) {
        if constexpr (V * sizeof(T) < 16)
            return c.cols <= 1024
                       ? norm_back_odd<T, 4, 256>(c, partial, blocks, s)
                   : c.cols <= 2048
                       ? norm_back_odd<T, 8, 256>(c, partial, blocks, s)
                   : c.cols <= 4096
                       ? norm_back_odd<T, 16, 256>(c, partial, blocks, s)
                       : norm_back_odd<T, 16, 512>(c, partial, blocks, s);
    }
    if (V * sizeof(T) == 16 && packs <= 1024 && gate_plain(c)) {
        if constexpr (V * sizeof(T) == 16)
            return packs <= 256 ? norm_back_ahead<T, 1, 256>(c, partial,
                                                             blocks, s)
                   : packs <= 512 ? norm_back_ahead<T, 2, 256>(c, partial,
                                                               blocks, s)
                                  : norm_back_ahead<T, 2, 512>(c, partial,
                                                               blocks, s);
    } else {
        if (packs <= 512)
            return norm_back_launch<T, V, 1>(c, partial, blocks, s);
        if (packs <= 1024)
            return norm_back_launch<T, V, 2>(c, partial, blocks, s);
    }
    if (packs <= 2048) return norm_back_launch<T, V, 4>(c, partial, blocks, s);
    if constexpr (kWords * 8 <= 16)
        if (packs <= 4096)
            return norm_back_launch<T, V, 8>(c, partial, blocks, s);
    if constexpr (kWords * 16 <= 16)
        if (packs <= 8192)
            return norm_back_launch<T, V, 16>(c, partial, blocks, s);
    const auto kernel = norm_back_loop_kernel<T, V>;
    const size_t need = (size_t)3 * c.cols * sizeof(float);
    const bool room = partial != nullptr && need <= 200 * 1024;
    int sms = 0;
    cudaError_t e = current_sm_count(&sms);
    if (e == cudaSuccess && room)
        e = allow_max_smem(reinterpret_cast<const void *>(kernel));
    if (e != cudaSuccess) return e;
    *blocks = back_grid(c.rows, kLoop, room ? need : 0, sms);
    return launch_dependent(kernel, *blocks, kLoop, room ? need : 0, s, c,
                            partial, room ? 1 : 0);
}

template <typename T>
cudaError_t norm_back_as(const mt_block_norm_back_t &c, int V, float *partial,
                         int *blocks, cudaStream_t s) {
    if constexpr (sizeof(T) == 2)
        if (V == 8) return norm_back_packs<T, 8>(c, partial, blocks, s);
    if (V >= 4) return norm_back_packs<T, 4>(c, partial, blocks, s);
    if (V >= 2) return norm_back_packs<T, 2>(c, partial, blocks, s);
    return norm_back_packs<T, 1>(c, partial, blocks, s);
}

}  // namespace

#define MT_DEFINE_BLOCK_NORM(T, dt)                                          \
    cudaError_t launch_block_norm_##dt(const mt_block_norm_call_t &c, int V, \
                                       cudaStream_t s) {                     \
        return norm_as<T>(c, V, s);                                          \
    }                                                                        \
    cudaError_t launch_block_norm_back_##dt(const mt_block_norm_back_t &c,   \
                                            int V, float *partial,           \
                                            int *blocks, cudaStream_t s) {   \
        return norm_back_as<T>(c, V, partial, blocks, s);                    \
    }

}  // namespace mt

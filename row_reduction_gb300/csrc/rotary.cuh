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
// times that, modulo 2^64, is the angle exactly (the frequency's own rounding,
// at most 2^-63 turns, grows to 2^-32 turns at position 2^31).  Its top 32
// bits, taken as signed, give the angle in [-pi, pi), cut off by less than
// 2^-32 turns (1.5e-9 radians), and their conversion to FP32 rounds at 2^-25
// of half a turn: 1e-7 radians in all, whatever the position.  FP32 storage
// then takes sincospif (2 ulp).  For 16-bit storage __sinf and __cosf are
// enough: on [-pi, pi] they are off by at most 2^-21.4 and 2^-21.2, with the
// angle's three roundings 1e-6 in all, where the output's own rounding is up
// to 2^-12 (FP16) or 2^-9 (BF16); sincospif there costs as much as the rest of
// a token.
#pragma once

#include "mt_decoder.cuh"

namespace mt {

// Groups of heads whose loads a warp has in flight, for K slots per lane.
template <int K>
constexpr int kRotFlight = K == 1 ? 4 : (K == 2 ? 2 : 1);

// A lane's slot: where its two packs are, and its values as V first and V
// second members of pairs (a, b).
template <typename T, int V, bool ILV>
struct RotSlot {
    int lo, hi;    // offsets of the packs
    bool in;       // the head has such a slot
    bool rot;      // ... and its pairs are turned
    bool second;   // the second pack exists (not in an odd head's last slot)

    __device__ __forceinline__ RotSlot(const RotArgs &a, int j) {
        in = j < a.slots;
        rot = j < a.rot_slots;
        lo = ILV || !rot ? 2 * j * V : j * V;
        hi = ILV || !rot ? lo + V : a.pairs + j * V;
        second = V > 1 || hi < a.dim;
    }
    struct Packs {
        Raw<T, V> lo, hi;
        __device__ __forceinline__ void zero() {
            lo.zero();
            hi.zero();
        }
    };
    // Leaves r as it was where there is no such slot: zeroed once, it adds
    // nothing to its head's sums.  (A head that is not there may leave the
    // values of another, of which nothing is stored.)
    __device__ __forceinline__ void load(const T *p, bool there,
                                         Packs &r) const {
        if (there && in) {
            r.lo.load(p + lo);
            if (second) r.hi.load(p + hi);
        }
    }
    static __device__ __forceinline__ void split(const Packs &r, float *a,
                                                 float *b) {
        if (!ILV) {
            r.lo.widen(a);
            r.hi.widen(b);
        } else {
            float z[2 * V];
            r.lo.widen(z);
            r.hi.widen(z + V);
#pragma unroll
            for (int e = 0; e < V; ++e) {
                a[e] = z[2 * e];
                b[e] = z[2 * e + 1];
            }
        }
    }
    __device__ __forceinline__ void store(T *p, const float *a,
                                          const float *b) const {
        if (!ILV) {
            st_vec<T, V>(p + lo, a);
            if (second) st_vec<T, V>(p + hi, b);
        } else {
            float z[2 * V];
#pragma unroll
            for (int e = 0; e < V; ++e) {
                z[2 * e] = a[e];
                z[2 * e + 1] = b[e];
            }
            st_vec<T, V>(p + lo, z);
            if (second) st_vec<T, V>(p + hi, z + V);
        }
    }
    __device__ __forceinline__ void weights(const T *w, float *a,
                                            float *b) const {
#pragma unroll
        for (int e = 0; e < V; ++e) a[e] = b[e] = 1.f;
        if (w != nullptr && in) {
            Packs r;
            r.zero();
            load(w, true, r);
            split(r, a, b);
        }
    }
    // s cos and s sin of the slot's pairs at position p; 1 and 0 for a slot
    // that is not turned.
    __device__ __forceinline__ void angles(const RotArgs &a, int64_t pos,
                                           int j, float *c, float *s) const {
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
                const float turned = (float)(int32_t)(t >> 32);
                float sn, cs;
                if (sizeof(T) == 4) {
                    // half turns, in [-1, 1)
                    sincospif(turned * 4.6566128730773926e-10f, &sn, &cs);
                } else {
                    // radians, in [-pi, pi)
                    const float x = turned * 1.4629180792671596e-09f;
                    sn = __sinf(x);
                    cs = __cosf(x);
                }
                c[e] = cs * a.scale;
                s[e] = sn * a.scale * a.sign;
            }
        }
    }
};

__device__ __forceinline__ int64_t rot_position(const RotArgs &a, int64_t t) {
    return a.pos64 ? static_cast<const int64_t *>(a.pos)[t]
                   : (int64_t) static_cast<const int32_t *>(a.pos)[t];
}

// Sum over the L lanes of a head (xor butterfly; every lane gets it).
__device__ __forceinline__ float head_sum(float v, int log2L) {
#pragma unroll
    for (int i = 0; i < 5; ++i)
        if (i < log2L) v += __shfl_xor_sync(kFull, v, 1 << i);
    return v;
}

// What the forward pass multiplies a pair with, once per token and tensor:
//     y_a = r (a k1 + b k2),  y_b = r (a k3 + b k4).
template <int V>
struct RotFactors {
    float k1[V], k2[V], k3[V], k4[V];
};

// Works on and stores U groups of heads of one tensor (the first `here` of
// them exist, for whole warps): x's packs in raw, the lane's head of the
// first group in `head`, `stride` heads and `ys` values of y between groups.
template <typename T, int V, int K, bool ILV, bool NORM, int U>
__device__ __forceinline__ void rot_groups(
    const RotArgs &a, int l, int L, const typename RotSlot<T, V, ILV>::Packs
    (*raw)[K], const RotFactors<V> *f, T *y, int64_t ys, int head, int stride,
    int heads, int here, bool all_rot) {
    using S = RotSlot<T, V, ILV>;
#pragma unroll
    for (int u = 0; u < U; ++u) {
        if (u >= here) break;
        float va[K][V], vb[K][V];
        float r = 1.f;
        if (NORM) {
            float sq[V];
#pragma unroll
            for (int k = 0; k < K; ++k) {
                S::split(raw[u][k], va[k], vb[k]);
                if (k == 0)
                    mul_n<V>(sq, va[k], va[k]);
                else
                    fma_n<V>(sq, va[k], va[k], sq);
                fma_n<V>(sq, vb[k], vb[k], sq);
            }
            float ss = sq[0];
#pragma unroll
            for (int e = 1; e < V; ++e) ss += sq[e];
            r = rsqrtf(head_sum(ss, a.log2L) * a.inv_dim + a.eps);
        }
        T *out = y + u * ys;
        const bool there = head + u * stride < heads;
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const S slot(a, l + k * L);
            if (!slot.in || !there) continue;
            if (!NORM) {
                if (!all_rot && !slot.rot) {  // copied bit for bit
                    raw[u][k].lo.store(out + slot.lo);
                    if (slot.second) raw[u][k].hi.store(out + slot.hi);
                    continue;
                }
                S::split(raw[u][k], va[k], vb[k]);
            }
            float oa[V], ob[V];
            mul_n<V>(oa, va[k], f[k].k1);
            mul_n<V>(ob, vb[k], f[k].k4);
            if (all_rot || slot.rot) {  // 0 times a neighbour may be NaN
                fma_n<V>(oa, vb[k], f[k].k2, oa);
                fma_n<V>(ob, va[k], f[k].k3, ob);
            }
            if (NORM) {
                scale_n<V>(oa, oa, r);
                scale_n<V>(ob, ob, r);
            }
            slot.store(out, oa, ob);
        }
    }
}

// Forward (and, with the sines' sign turned, backward without norm).  Bound by
// latency at 16 warps per SM (128 registers, and 24 bytes spilled: coefficients,
// and the loads of four groups; 24 warps with 8-byte packs and no norm): BF16,
// 16384 tokens of 32 + 8 heads of 128 with norm 60 us, 5.6 TB/s, 82% of the
// measured copy bandwidth.  With few heads the angles and weights of a token
// are worked out by each group of lanes (57359 tokens of 4 + 1 heads of 64
// 32 us, 34%).  The loads of U groups of heads are issued before the angles
// are computed and before any of them is used.  HQ < U: a warp has at most HQ
// groups of queries and U - HQ of keys, all of them asked for at once.
template <typename T, int V, int K, bool ILV, bool NORM, int HQ>
__global__ void __launch_bounds__(
    kRotThreads, sizeof(T) == 2 && V * K <= 4 && !NORM ? 3 : 2)
    rotary_kernel(const RotArgs a) {
    using S = RotSlot<T, V, ILV>;
    constexpr int U = kRotFlight<K>;
    constexpr bool kFew = HQ < U;
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
    const int split = 1 << a.log2S;
    const int first = (int)(unit & (split - 1));
    const int64_t pos = rot_position(a, t);
    // The warps of a token take its groups of heads in turn; the key heads'
    // groups follow the query heads'.
    const int first_k = (first - a.t[0].groups) & (split - 1);
    const int stride = split * heads_per_warp;  // heads between two groups
    const bool all_rot = a.rot_slots == a.slots;
    typename S::Packs raw[U][K];
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
        for (int k = 0; k < K; ++k) raw[u][k].zero();
    const auto load = [&](const T *x, int64_t step, int head, int heads,
                          auto from, auto to) {
        constexpr int at = decltype(from)::value, end = decltype(to)::value;
#pragma unroll
        for (int u = 0; u < end - at; ++u)
#pragma unroll
            for (int k = 0; k < K; ++k)
                S(a, l + k * L).load(x + u * step, head + u * stride < heads,
                                     raw[at + u][k]);
    };
    const std::integral_constant<int, 0> none{};
    const std::integral_constant<int, HQ> keys{};
    const std::integral_constant<int, U> all{};
    const int q0 = first * heads_per_warp + sub;
    load(static_cast<const T *>(a.t[0].x) + t * a.t[0].xt + q0 * a.t[0].xh,
         stride * a.t[0].xh, q0, a.t[0].heads, none, keys);
    if (kFew) {
        const int k0 = first_k * heads_per_warp + sub;
        load(static_cast<const T *>(a.t[1].x) + t * a.t[1].xt +
                 k0 * a.t[1].xh,
             stride * a.t[1].xh, k0, a.t[1].heads, keys, all);
    }
    float c[K][V], s[K][V];
#pragma unroll
    for (int k = 0; k < K; ++k)
        S(a, l + k * L).angles(a, pos, l + k * L, c[k], s[k]);
    const auto factors = [&](const T *weight, RotFactors<V> *f) {
#pragma unroll
        for (int k = 0; k < K; ++k) {
            float wa[V], wb[V];
            if (NORM) S(a, l + k * L).weights(weight, wa, wb);
#pragma unroll
            for (int e = 0; e < V; ++e) {
                f[k].k1[e] = NORM ? wa[e] * c[k][e] : c[k][e];
                f[k].k2[e] = NORM ? -wb[e] * s[k][e] : -s[k][e];
                f[k].k3[e] = NORM ? wa[e] * s[k][e] : s[k][e];
                f[k].k4[e] = NORM ? wb[e] * c[k][e] : c[k][e];
            }
        }
    };
    if constexpr (kFew) {
        const auto groups = [&](int i, auto from, auto to) {
            constexpr int at = decltype(from)::value;
            const RotHeads &h = a.t[i];
            const int g0 = i == 0 ? first : first_k;
            if (g0 >= h.groups) return;
            const int head = g0 * heads_per_warp + sub;
            RotFactors<V> f[K];
            factors(static_cast<const T *>(h.w), f);
            rot_groups<T, V, K, ILV, NORM, decltype(to)::value - at>(
                a, l, L, raw + at, f,
                static_cast<T *>(h.y) + t * h.yt + head * h.yh,
                stride * h.yh, head, stride, h.heads,
                (h.groups - g0 + split - 1) >> a.log2S, all_rot);
        };
        groups(0, none, keys);
        groups(1, keys, all);
    } else {
#pragma unroll 1
        for (int i = 0; i < 2; ++i) {
            const RotHeads &h = a.t[i];
            const int g0 = i == 0 ? first : first_k;
            if (g0 >= h.groups) continue;
            int head = g0 * heads_per_warp + sub;
            const int heads = h.heads;
            const int64_t xs = stride * h.xh, ys = stride * h.yh;
            const T *x = static_cast<const T *>(h.x) + t * h.xt + head * h.xh;
            T *y = static_cast<T *>(h.y) + t * h.yt + head * h.yh;
            RotFactors<V> f[K];
            factors(static_cast<const T *>(h.w), f);
#pragma unroll 1
            for (int g = g0; g < h.groups; g += U * split) {
                if (i != 0 || g != g0) load(x, xs, head, heads, none, all);
                rot_groups<T, V, K, ILV, NORM, U>(
                    a, l, L, raw, f, y, ys, head, stride, heads,
                    (h.groups - g + split - 1) >> a.log2S, all_rot);
                x += U * xs;
                y += U * ys;
                head += U * stride;
            }
        }
    }
}

// Backward with norm.  A CTA serves the heads of one tensor and adds up its
// part of the weight's gradient in registers over all its tokens; at the end
// the lanes and warps that own the same slot are added in a fixed order and
// the CTA writes one row of partial sums, which rotary_dweight_kernel adds.
// Bound by dependent arithmetic at 16 warps per SM, with one item's loads on
// their way: BF16, 8192 tokens of 32 + 8 heads of 128 54 us, 4.6 TB/s.  FP32
// packs hold half the values; at 80 registers (of 110, 40 bytes spilled) 24 warps
// fit: 86 us for 94 there.  (BF16 with half as many per lane: 56 us at 24 warps.)
template <typename T, int V, int K, bool ILV, int THREADS>
__global__ void __launch_bounds__(THREADS, 2)
    rotary_backward_kernel(const RotArgs a) {
    using S = RotSlot<T, V, ILV>;
    constexpr int kWarps = THREADS / 32;
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
    float wa[K][V], wb[K][V], da[K][V], db[K][V];
#pragma unroll
    for (int k = 0; k < K; ++k) {
        S(a, l + k * L).weights(static_cast<const T *>(h.w), wa[k], wb[k]);
#pragma unroll
        for (int e = 0; e < V; ++e) da[k][e] = db[k][e] = 0.f;
    }
    // A warp takes an equal share of the tensor's (token, group) items, in
    // order, so that no warp has more than one more than another and the
    // angles of a token are computed by few warps.
    int64_t left, t;
    int head;  // the lane's
    {
        const int64_t items = a.tokens * h.groups;
        const int64_t warps = (int64_t)a.blocks[i] * kWarps;
        const int64_t me = (int64_t)block * kWarps + warp;
        const int64_t each = items / warps, more = items - each * warps;
        const int64_t first = each * me + min(more, me);
        left = each + (me < more ? 1 : 0);
        t = first / h.groups;
        head = (int)(first - t * h.groups) * heads_per_warp + sub;
    }
    const int heads = h.heads;
    const int64_t xs = heads_per_warp * h.xh, ds = heads_per_warp * h.dh,
                  ys = heads_per_warp * h.yh;
    const T *x = static_cast<const T *>(h.x) + t * h.xt + head * h.xh;
    const T *dy = static_cast<const T *>(h.dy) + t * h.dt + head * h.dh;
    T *y = static_cast<T *>(h.y) + t * h.yt + head * h.yh;
    typename S::Packs nx[K], nd[K];
#pragma unroll
    for (int k = 0; k < K; ++k) {
        nx[k].zero();
        nd[k].zero();
    }
    const auto load = [&]() {
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const S slot(a, l + k * L);
            slot.load(x, left > 0 && head < heads, nx[k]);
            slot.load(dy, left > 0 && head < heads, nd[k]);
        }
    };
    int64_t pos = left > 0 ? rot_position(a, t) : 0;
    load();
    float c[K][V], s[K][V];
    const bool all_rot = a.rot_slots == a.slots;
    bool turned = true;
#pragma unroll 1
    while (left > 0) {
        float xa[K][V], xb[K][V], ga[K][V], gb[K][V];
#pragma unroll
        for (int k = 0; k < K; ++k) {
            S::split(nx[k], xa[k], xb[k]);
            S::split(nd[k], ga[k], gb[k]);
        }
        T *out = y;
        const bool there = head < heads;
        if (turned) {
#pragma unroll
            for (int k = 0; k < K; ++k)
                S(a, l + k * L).angles(a, pos, l + k * L, c[k], s[k]);
        }
        // The next item is on its way while this one is worked on.
        --left;
        head += heads_per_warp;
        x += xs;
        dy += ds;
        y += ys;
        turned = head - sub >= heads;  // whole warps
        if (turned) {
            head = sub;
            ++t;
            x = static_cast<const T *>(h.x) + t * h.xt + head * h.xh;
            dy = static_cast<const T *>(h.dy) + t * h.dt + head * h.dh;
            y = static_cast<T *>(h.y) + t * h.yt + head * h.yh;
            if (left > 0) pos = rot_position(a, t);
        }
        load();

        float sq[V], dot[V];
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const S slot(a, l + k * L);
            if (all_rot || slot.rot) {
                // g = R^T dy: a.sign has turned the sines, so that
                // g_a = a c - b s, g_b = a s + b c
                float ta[V], tb[V], m[V];
                mul_n<V>(ta, ga[k], c[k]);
                mul_n<V>(tb, gb[k], c[k]);
#pragma unroll
                for (int e = 0; e < V; ++e) m[e] = -gb[k][e];
                fma_n<V>(tb, ga[k], s[k], tb);
                fma_n<V>(ga[k], m, s[k], ta);
#pragma unroll
                for (int e = 0; e < V; ++e) gb[k][e] = tb[e];
            }
            float ta[V], tb[V];
            mul_n<V>(ta, ga[k], wa[k]);
            mul_n<V>(tb, gb[k], wb[k]);
            if (k == 0) {
                mul_n<V>(sq, xa[k], xa[k]);
                mul_n<V>(dot, ta, xa[k]);
            } else {
                fma_n<V>(sq, xa[k], xa[k], sq);
                fma_n<V>(dot, ta, xa[k], dot);
            }
            fma_n<V>(sq, xb[k], xb[k], sq);
            fma_n<V>(dot, tb, xb[k], dot);
        }
        float xx = 0.f, gx = 0.f;
#pragma unroll
        for (int e = 0; e < V; ++e) {
            xx += sq[e];
            gx += dot[e];
        }
        xx = head_sum(xx, a.log2L);
        gx = head_sum(gx, a.log2L);
        const float r = rsqrtf(xx * a.inv_dim + a.eps);
        const float m = -gx * a.inv_dim * r * r;
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const S slot(a, l + k * L);
            // g r: dw += (g r) x, dx = (g r) w - x (m r)
            scale_n<V>(ga[k], ga[k], r);
            scale_n<V>(gb[k], gb[k], r);
            // A lane without a head holds another's values: it adds nothing
            // (0 times an infinity would be NaN).
            if (there && slot.in) {
                fma_n<V>(da[k], ga[k], xa[k], da[k]);
                fma_n<V>(db[k], gb[k], xb[k], db[k]);
                float oa[V], ob[V];
                mul_n<V>(oa, ga[k], wa[k]);
                mul_n<V>(ob, gb[k], wb[k]);
                scale_add_n<V>(oa, xa[k], m * r, oa);
                scale_add_n<V>(ob, xb[k], m * r, ob);
                slot.store(out, oa, ob);
            }
        }
    }
    if (a.partial == nullptr) return;
#pragma unroll
    for (int k = 0; k < K; ++k) {
        const S slot(a, l + k * L);
#pragma unroll
        for (int e = 0; e < V; ++e)
            for (int off = L; off < 32; off <<= 1) {
                da[k][e] += __shfl_xor_sync(kFull, da[k][e], off);
                db[k][e] += __shfl_xor_sync(kFull, db[k][e], off);
            }
        if (sub == 0 && slot.in) {
#pragma unroll
            for (int e = 0; e < V; ++e) {
                const int ia = ILV ? slot.lo + 2 * e : slot.lo + e;
                const int ib = ILV ? slot.lo + 2 * e + 1 : slot.hi + e;
                sums[warp][ia] = da[k][e];
                if (ib < a.dim) sums[warp][ib] = db[k][e];
            }
        }
    }
    __syncthreads();
    for (int d = threadIdx.x; d < a.dim; d += THREADS) {
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

// All groups at once where a warp's loads in flight hold them: as many of
// queries as of keys (BF16, 57359 tokens of 15 + 3 heads of 64, norm: 70 us,
// and 93 us without it), or one group of keys and the rest of queries (FP32,
// 44536 tokens of 6 + 2 heads of 96: 41 us, and 64 us without it).
template <typename T, bool ILV, bool NORM>
cudaError_t launch_rotary_as(const RotArgs &a, int V, int K, cudaStream_t s) {
    const int64_t units = a.tokens << a.log2S;
    const int64_t grid =
        (units + kRotThreads / 32 - 1) / (kRotThreads / 32);
    const auto fits = [&](int queries, int keys) {
        return rotary_fits(a, queries, keys);
    };
    return rot_dispatch<T, ILV>(V, K, [&](auto v, auto k) {
        constexpr int VV = decltype(v)::value, KK = decltype(k)::value;
        constexpr int U = kRotFlight<KK>;
        const auto run = [&](auto queries) {
            return launch_dependent(
                rotary_kernel<T, VV, KK, ILV, NORM, decltype(queries)::value>,
                grid, kRotThreads, 0, s, a);
        };
        if constexpr (U > 1)
            if (fits(U / 2, U / 2))
                return run(std::integral_constant<int, U / 2>{});
        if constexpr (U > 2)
            if (fits(U - 1, 1))
                return run(std::integral_constant<int, U - 1>{});
        return run(std::integral_constant<int, U>{});
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
        constexpr int VV = decltype(v)::value, KK = decltype(k)::value;
        const int grid = a.blocks[0] + a.blocks[1];
        if constexpr (sizeof(T) == 4 && KK == 1) {
            if (a.threads == kRotBackThreads)
                return launch_dependent(
                    rotary_backward_kernel<T, VV, KK, ILV, kRotBackThreads>,
                    grid, kRotBackThreads, 0, s, a);
        }
        return launch_dependent(
            rotary_backward_kernel<T, VV, KK, ILV, kRotThreads>, grid,
            kRotThreads, 0, s, a);
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

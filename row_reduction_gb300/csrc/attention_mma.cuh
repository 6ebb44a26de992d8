// attention_mma.cuh -- attention over the quantised cache on matrix
// instructions (one translation unit per code format).
//
// Scores are formed transposed, keys x queries (S^T = K Q^T), so that the
// cache's codes, which are the long operand, fill the instruction's 16 rows and
// the few query heads that share a key head its 8 columns.  A warp goes through
// chunks of keys of its own: codes come straight into registers, in the order
// of the instruction's fragments (the order of the dimensions is free as long
// as queries have the same; see Q below), one chunk ahead of the one that is
// worked on, and are widened to FP16 there, exactly.  What the scores give
// turns into the other product's operand (O^T = V^T P^T) by one transposition
// of 8 x 8 values within the warp.
//
// Scales.  A key's factor multiplies its score's sum of each group, a value's
// the weight that goes into the product of that group.
//
// Roundings to FP16.  Codes are exact.  Queries are held as a power of two
// times FP16 with the head's largest value at 2^14..2^15, BF16 and FP16 values
// exactly (down to 2^-28 of the largest), FP32 in two parts (2^-22).  Weights
// times the values' scales are held against the chunk's largest likewise: one
// part for BF16 output (2^-11, a quarter of its own rounding), two for FP16 and
// FP32.  Sums over a chunk are the instruction's, in FP32; sums over chunks are
// rounded to nearest in FP32.
//
// Work is dealt out in units, a chunk of keys of one tile (rows of a sequence
// and the query heads of a key head, up to 8 NT columns): every CTA takes an
// equal run of all units of the batch in their order, wherever sequences begin
// and end in it, so that lengths of any mixture fill the device and nothing
// about them need be known on the host.  A tile that is cut by the ends of
// runs is left as partial sums, which a second kernel joins in order.
#pragma once

#include "attention.cuh"

namespace mt {
namespace {

constexpr int kWarps = 4;

// ---- sums of a tile's units ----------------------------------------------------
// sum over 0 <= t < n of floor((a t + b) / m), for a, b >= 0.
__device__ __forceinline__ int64_t floor_sum(int64_t n, int64_t m, int64_t a,
                                             int64_t b) {
    int64_t s = 0;
    while (n > 0) {
        s += (n - 1) * n / 2 * (a / m) + n * (b / m);
        a %= m;
        b %= m;
        const int64_t y = a * n + b;
        if (y < m) break;
        n = y / m;
        b = y % m;
        const int64_t x = m;
        m = a;
        a = x;
    }
    return s;
}

// How the rows of a sequence are cut into tiles and units of KEYS keys.
struct Tiles {
    int64_t start;   // position of the first row
    int32_t rows;    // of the sequence
    int32_t per;     // rows of a tile
    int32_t count;   // tiles
    int32_t window;
    bool all;        // every tile goes through all keys (last bounds)
    // Tile t's first and last unit of keys (of what its rows may see).
    template <int KEYS>
    __device__ __forceinline__ int64_t first(int t) const {
        if (window == 0) return 0;
        return max(start + (int64_t)t * per - window + 1, (int64_t)0) / KEYS;
    }
    template <int KEYS>
    __device__ __forceinline__ int64_t last(int t) const {
        const int64_t r = all ? rows : min((int64_t)(t + 1) * per,
                                           (int64_t)rows);
        return (start + r - 1) / KEYS;
    }
    // Units of the tiles before t (first <= last in every tile).
    template <int KEYS>
    __device__ __forceinline__ int64_t before(int t) const {
        if (t <= 0) return 0;
        int64_t s = t;
        if (all) {
            s += t * last<KEYS>(0);
        } else {
            // all tiles but the sequence's last are whole
            const int whole = t < count ? t : count - 1;
            s += floor_sum(whole, KEYS, per, start + per - 1);
            if (t > whole) s += last<KEYS>(count - 1);
        }
        if (window != 0) {
            // from tile z on the window's begin is not negative
            const int64_t short_of = window - 1 - start;
            const int64_t z = short_of <= 0 ? 0 : (short_of + per - 1) / per;
            if (t > z)
                s -= floor_sum(t - z, KEYS, per, start + z * per - window + 1);
        }
        return s;
    }
};

// What the call's tiles have in common.
struct Cut {
    int32_t times;   // query heads per key head
    int32_t per;     // rows of a tile
    int32_t parts;   // tiles that share a row's query heads
};

__device__ __forceinline__ Tiles tiles_of(const mt_attention_call_t &c,
                                          const Cut &cut, int s) {
    Tiles t;
    const int64_t n = (int64_t)c.offsets[s + 1] - c.offsets[s];
    t.start = max(c.starts[s], 0);
    t.rows = (int32_t)max(n, (int64_t)0);
    t.per = cut.per;
    t.count = (t.rows + cut.per - 1) / cut.per;
    t.window = c.window;
    t.all = c.last != nullptr;
    return t;
}

// A cut tile that begins in a CTA's run: where its parts lie and what it is.
struct Record {
    int32_t valid, last;      // last: the CTA that holds its end
    int32_t row, rows;        // rows of the batch
    int32_t head, part;       // key head; part of the row's query heads
};
struct Share {
    Record *records;          // one per CTA
    float *sums;              // two places per CTA: m, l, O of each column
};

__host__ __device__ constexpr int place_floats(int columns, int dim) {
    return columns * (dim + 2);
}

// ---- instructions --------------------------------------------------------------
__device__ __forceinline__ void mma16816(float (&d)[4], const unsigned (&a)[4],
                                         unsigned b0, unsigned b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 "
        "{%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ unsigned transpose8x8(unsigned v) {
    unsigned r;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;"
                 : "=r"(r) : "r"(v));
    return r;
}
__device__ __forceinline__ unsigned half_pair(float lo, float hi) {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const unsigned *>(&h);
}
__device__ __forceinline__ float2 from_half_pair(unsigned v) {
    return __half22float2(*reinterpret_cast<const __half2 *>(&v));
}

// Four codes as two pairs of FP16 values, exactly.  int8: byte b + 128 under
// the exponent of 2^10 is the value 1152 + b.
template <bool INT8>
__device__ __forceinline__ void widen4(unsigned w, unsigned &lo,
                                       unsigned &hi) {
    if (INT8) {
        const unsigned u = w ^ 0x80808080u;
        const unsigned off = 0x64806480u;  // 1152, twice
        unsigned a = __byte_perm(u, 0x64646464u, 0x4140);
        unsigned b = __byte_perm(u, 0x64646464u, 0x4342);
        const __half2 x = __hsub2(*reinterpret_cast<const __half2 *>(&a),
                                  *reinterpret_cast<const __half2 *>(&off));
        const __half2 y = __hsub2(*reinterpret_cast<const __half2 *>(&b),
                                  *reinterpret_cast<const __half2 *>(&off));
        lo = *reinterpret_cast<const unsigned *>(&x);
        hi = *reinterpret_cast<const unsigned *>(&y);
    } else {
        const __half2_raw x = __nv_cvt_fp8x2_to_halfraw2(
            (__nv_fp8x2_storage_t)(w & 0xffffu), __NV_E4M3);
        const __half2_raw y = __nv_cvt_fp8x2_to_halfraw2(
            (__nv_fp8x2_storage_t)(w >> 16), __NV_E4M3);
        lo = (unsigned)x.x | (unsigned)x.y << 16;
        hi = (unsigned)y.x | (unsigned)y.y << 16;
    }
}

// BYTES of codes into words; zeros where not `on`.
template <int BYTES>
__device__ __forceinline__ void load_codes(const uint8_t *p, bool on,
                                           unsigned *w) {
    if constexpr (BYTES == 32) {
#pragma unroll
        for (int i = 0; i < 8; ++i) w[i] = 0;
        if (on)
            asm volatile("ld.global.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, "
                         "[%8];"
                         : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]),
                           "=r"(w[4]), "=r"(w[5]), "=r"(w[6]), "=r"(w[7])
                         : "l"(p));
    } else if constexpr (BYTES == 16) {
        uint4 v = make_uint4(0, 0, 0, 0);
        if (on) v = *reinterpret_cast<const uint4 *>(p);
        w[0] = v.x; w[1] = v.y; w[2] = v.z; w[3] = v.w;
    } else if constexpr (BYTES == 8) {
        uint2 v = make_uint2(0, 0);
        if (on) v = *reinterpret_cast<const uint2 *>(p);
        w[0] = v.x; w[1] = v.y;
    } else if constexpr (BYTES == 4) {
        w[0] = on ? *reinterpret_cast<const unsigned *>(p) : 0u;
    } else {
        w[0] = on ? *reinterpret_cast<const unsigned short *>(p) : 0u;
    }
}
template <int N>
__device__ __forceinline__ void load_scales(const float *p, bool on,
                                            float *v) {
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = 0.f;
    if (!on) return;
    if constexpr (N % 4 == 0) {
#pragma unroll
        for (int i = 0; i < N; i += 4) {
            const float4 f = *reinterpret_cast<const float4 *>(p + i);
            v[i] = f.x; v[i + 1] = f.y; v[i + 2] = f.z; v[i + 3] = f.w;
        }
    } else if constexpr (N == 2) {
        const float2 f = *reinterpret_cast<const float2 *>(p);
        v[0] = f.x; v[1] = f.y;
    } else {
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] = p[i];
    }
}

// ---- a head's layout -------------------------------------------------------------
template <int DIM_, int GROUPS_>
struct Head {
    static constexpr int DIM = DIM_, GROUPS = GROUPS_;
    static constexpr int GROUP = DIM / GROUPS;
    // A group is cut into blocks of B dimensions, the largest power of two
    // that divides it, at most 128.  Of a block, lane l of a quad holds the
    // B/4 bytes from l B/4 on of a key (two steps of the instruction take a
    // word of 4), and lane l of eight the B/8 bytes from l B/8 on of a value.
    static constexpr int B = (GROUP & -GROUP) > 128 ? 128 : (GROUP & -GROUP);
    static constexpr int BLOCKS = DIM / B;
    static constexpr int KEYS = DIM > 128 ? 16 : 32;  // of a chunk
    static constexpr int STEPS = DIM / 16;
    static constexpr int VWORDS = B >= 32 ? DIM / 32 : BLOCKS;
};

// A column of a tile: one row's query head.
struct Column {
    float f;            // score = f (q . k): the scale and the query's power
    float slope;
    int32_t lo, hi;     // keys that it sees
    int32_t p;          // its row's position
    int32_t pad;
};

template <class H, int PARTS, int NT>
struct Shared {
    uint2 q[NT][PARTS][H::STEPS][32];   // fragments
    Column column[8 * NT];
    int32_t lo_any, hi_any, lo_all, hi_all;
    float m[kWarps][8 * NT], l[kWarps][8 * NT];
    float o[kWarps][8 * NT][H::DIM + 4];
    int64_t scan[kWarps];
    int64_t at;         // place of the CTA's first unit in its sequence
    int32_t sequence;
};

template <class H, bool INT8, int PARTS, int NT>
struct Warp {
    static constexpr int KT = H::KEYS / 16;     // rows of 16 keys
    static constexpr int C = 8 * NT;
    unsigned k[KT][2][H::STEPS];
    unsigned v[KT][4][H::VWORDS];
    float ks[KT][2][H::GROUPS], vs[KT][2][H::GROUPS];
    float o[NT][H::STEPS][4];
    float m[NT][2], l[NT][2];

    __device__ __forceinline__ void begin() {
#pragma unroll
        for (int n = 0; n < NT; ++n) {
#pragma unroll
            for (int i = 0; i < H::STEPS; ++i)
#pragma unroll
                for (int e = 0; e < 4; ++e) o[n][i][e] = 0.f;
            m[n][0] = m[n][1] = -INFINITY;
            l[n][0] = l[n][1] = 0.f;
        }
    }
    // slot: of the chunk's key `lane`, or -1.
    __device__ __forceinline__ void load_keys(const mt_attention_call_t &c,
                                              int head, int slot) {
        const int lane = threadIdx.x & 31, g = lane >> 2, q = lane & 3;
#pragma unroll
        for (int t = 0; t < KT; ++t)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int s = __shfl_sync(kFull, slot, 16 * t + 8 * i + g);
                const int64_t at = (int64_t)s * c.k_heads + head;
                const uint8_t *p = static_cast<const uint8_t *>(c.k_codes) +
                                   at * H::DIM + q * (H::B / 4);
#pragma unroll
                for (int b = 0; b < H::BLOCKS; ++b)
                    load_codes<H::B / 4>(p + b * H::B, s >= 0,
                                         &k[t][i][b * (H::B / 16)]);
                load_scales<H::GROUPS>(c.k_scales + at * H::GROUPS, s >= 0,
                                       ks[t][i]);
            }
    }
    __device__ __forceinline__ void load_values(const mt_attention_call_t &c,
                                                int head, int slot) {
        const int lane = threadIdx.x & 31, g = lane >> 2, q = lane & 3;
#pragma unroll
        for (int t = 0; t < KT; ++t) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int s = __shfl_sync(
                    kFull, slot, 16 * t + 2 * q + (i & 1) + 8 * (i >> 1));
                const uint8_t *p = static_cast<const uint8_t *>(c.v_codes) +
                                   ((int64_t)s * c.k_heads + head) * H::DIM +
                                   g * (H::B / 8);
#pragma unroll
                for (int b = 0; b < H::BLOCKS; ++b)
                    load_codes<H::B / 8>(
                        p + b * H::B, s >= 0,
                        &v[t][i][H::B >= 32 ? b * (H::B / 32) : b]);
            }
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int s = __shfl_sync(kFull, slot, 16 * t + 8 * i + g);
                load_scales<H::GROUPS>(
                    c.v_scales + ((int64_t)s * c.k_heads + head) * H::GROUPS,
                    s >= 0, vs[t][i]);
            }
        }
    }
    // Sums of codes times queries times the keys' scales.
    __device__ __forceinline__ void scores(
        const Shared<H, PARTS, NT> &sh, float (&z)[NT][KT][4]) {
        const int lane = threadIdx.x & 31;
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int t = 0; t < KT; ++t)
#pragma unroll
                for (int e = 0; e < 4; ++e) z[n][t][e] = 0.f;
        constexpr int kPer = H::STEPS / H::GROUPS;  // steps of a group
#pragma unroll
        for (int gr = 0; gr < H::GROUPS; ++gr) {
            float acc[NT][KT][4];
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int t = 0; t < KT; ++t)
#pragma unroll
                    for (int e = 0; e < 4; ++e) acc[n][t][e] = 0.f;
#pragma unroll
            for (int i = gr * kPer; i < (gr + 1) * kPer; ++i) {
                unsigned a[KT][4];
#pragma unroll
                for (int t = 0; t < KT; ++t) {
                    widen4<INT8>(k[t][0][i], a[t][0], a[t][2]);
                    widen4<INT8>(k[t][1][i], a[t][1], a[t][3]);
                }
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int part = 0; part < PARTS; ++part) {
                        const uint2 b = sh.q[n][part][i][lane];
#pragma unroll
                        for (int t = 0; t < KT; ++t)
                            mma16816(acc[n][t], a[t], b.x, b.y);
                    }
            }
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int t = 0; t < KT; ++t)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        z[n][t][e] = fmaf(acc[n][t][e], ks[t][e >> 1][gr],
                                          z[n][t][e]);
        }
    }
    // Scores to exponents of two; -infinity, and a bit of `hidden`, for keys
    // that a column does not see.  j0: the chunk's first key; there: its keys
    // that have a slot.
    __device__ __forceinline__ void bend(const mt_attention_call_t &c,
                                         const Shared<H, PARTS, NT> &sh,
                                         float inv_cap, int j0,
                                         unsigned there, unsigned &hidden,
                                         float (&z)[NT][KT][4]) {
        hidden = 0;
        const int lane = threadIdx.x & 31, g = lane >> 2, q = lane & 3;
        constexpr unsigned kAll = H::KEYS == 32 ? ~0u : 0xffffu;
        const bool whole = there == kAll && j0 >= sh.lo_all &&
                           j0 + H::KEYS - 1 <= sh.hi_all;
#pragma unroll
        for (int n = 0; n < NT; ++n) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const Column &col = sh.column[8 * n + 2 * q + h];
                const float f = col.f;
#pragma unroll
                for (int t = 0; t < KT; ++t)
#pragma unroll
                    for (int i = 0; i < 2; ++i) z[n][t][2 * i + h] *= f;
                if (c.cap > 0.f) {
#pragma unroll
                    for (int t = 0; t < KT; ++t)
#pragma unroll
                        for (int i = 0; i < 2; ++i)
                            z[n][t][2 * i + h] =
                                capped(z[n][t][2 * i + h], c.cap, inv_cap);
                }
                if (c.slopes != nullptr) {
#pragma unroll
                    for (int t = 0; t < KT; ++t)
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            const int j = j0 + 16 * t + 8 * i + g;
                            z[n][t][2 * i + h] -=
                                col.slope * (float)abs(col.p - j);
                        }
                }
                if (!whole) {
#pragma unroll
                    for (int t = 0; t < KT; ++t)
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            const int at = 16 * t + 8 * i + g;
                            const bool see = there >> at & 1u &&
                                             j0 + at >= col.lo &&
                                             j0 + at <= col.hi;
                            if (!see) {
                                z[n][t][2 * i + h] = -INFINITY;
                                hidden |= 1u << (4 * (n * KT + t) + 2 * i + h);
                            }
                        }
                }
            }
#pragma unroll
            for (int t = 0; t < KT; ++t)
#pragma unroll
                for (int e = 0; e < 4; ++e) z[n][t][e] *= kLog2e;
        }
    }
    // Weights about the running maximum, and what the sums so far take.
    __device__ __forceinline__ void weigh(float (&z)[NT][KT][4],
                                          float (&keep)[NT][2]) {
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                float top = z[n][0][h];
#pragma unroll
                for (int t = 0; t < KT; ++t)
#pragma unroll
                    for (int i = 0; i < 2; ++i)
                        top = nanmax(top, z[n][t][2 * i + h]);
#pragma unroll
                for (int off = 4; off < 32; off <<= 1)
                    top = nanmax(top, __shfl_xor_sync(kFull, top, off));
                top = nanmax(top, m[n][h]);
                // nothing seen yet: all weights are 2^-infinity
                const float ref = top == -INFINITY ? 0.f : top;
                keep[n][h] = pow2(m[n][h] - ref);
                m[n][h] = top;
                float sum = 0.f;
#pragma unroll
                for (int t = 0; t < KT; ++t)
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        float &w = z[n][t][2 * i + h];
                        w = pow2(w - ref);
                        sum += w;
                    }
                l[n][h] = fmaf(l[n][h], keep[n][h], sum);
            }
    }
    // Adds the chunk's weights times values.
    __device__ __forceinline__ void add(const float (&w)[NT][KT][4],
                                        const float (&keep)[NT][2],
                                        unsigned hidden) {
        constexpr int kPer = H::STEPS / H::GROUPS;
#pragma unroll
        for (int gr = 0; gr < H::GROUPS; ++gr) {
            unsigned b[NT][PARTS][KT][2];
            float back[NT][2];
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                float pv[KT][4];
                unsigned e0 = 0, e1 = 0;
#pragma unroll
                for (int t = 0; t < KT; ++t)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        pv[t][e] = w[n][t][e] * vs[t][e >> 1][gr];
                        // not seen: nothing, whatever stands in the scale
                        if (hidden >> (4 * (n * KT + t) + e) & 1u)
                            pv[t][e] = 0.f;
                        const unsigned bits = __float_as_uint(pv[t][e]);
                        if (e & 1) e1 = max(e1, bits & 0x7fffffffu);
                        else e0 = max(e0, bits & 0x7fffffffu);
                    }
                unsigned ex = e0 >> 23 | (e1 >> 23) << 16;
#pragma unroll
                for (int off = 4; off < 32; off <<= 1)
                    ex = __vmaxu2(ex, __shfl_xor_sync(kFull, ex, off));
                float up[2];
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    // the largest at 2^14..2^15
                    const unsigned x = max(h ? ex >> 16 : ex & 0xffffu, 15u);
                    up[h] = __uint_as_float((268u - x) << 23);
                    back[n][h] = __uint_as_float((x - 14u) << 23);
                }
#pragma unroll
                for (int t = 0; t < KT; ++t)
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const float x = pv[t][2 * i] * up[0];
                        const float y = pv[t][2 * i + 1] * up[1];
                        const unsigned hi = half_pair(x, y);
                        b[n][0][t][i] = transpose8x8(hi);
                        if constexpr (PARTS == 2) {
                            const float2 r = from_half_pair(hi);
                            b[n][1][t][i] =
                                transpose8x8(half_pair(x - r.x, y - r.y));
                        }
                    }
            }
            // Two rows of the output per lane and step: dimensions 2 i and
            // 2 i + 1 of its bytes; a pair of keys side by side.
#pragma unroll
            for (int i = gr * kPer; i < (gr + 1) * kPer; i += 2) {
                // words with the dimensions of steps i and i + 1
                unsigned a[2][KT][4];
#pragma unroll
                for (int t = 0; t < KT; ++t)
#pragma unroll
                    for (int y = 0; y < 2; ++y) {
                        const int word = H::B >= 32 ? i / 2 : i;
                        const unsigned u = v[t][2 * y][word];
                        const unsigned x = v[t][2 * y + 1][word];
                        widen4<INT8>(__byte_perm(u, x, 0x5140), a[0][t][2 * y],
                                     a[0][t][2 * y + 1]);
                        if constexpr (H::B >= 32)
                            widen4<INT8>(__byte_perm(u, x, 0x7362),
                                         a[1][t][2 * y], a[1][t][2 * y + 1]);
                        else if (i + 1 < (gr + 1) * kPer)
                            widen4<INT8>(
                                __byte_perm(v[t][2 * y][word + 1],
                                            v[t][2 * y + 1][word + 1],
                                            0x5140),
                                a[1][t][2 * y], a[1][t][2 * y + 1]);
                    }
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int y = 0; y < 2; ++y) {
                        if (i + y >= (gr + 1) * kPer) continue;
                        float acc[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                        for (int part = 0; part < PARTS; ++part)
#pragma unroll
                            for (int t = 0; t < KT; ++t)
                                mma16816(acc, a[y][t], b[n][part][t][0],
                                         b[n][part][t][1]);
                        float (&out)[4] = o[n][i + y];
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            out[e] = fmaf(acc[e], back[n][e & 1],
                                          out[e] * keep[n][e & 1]);
                    }
            }
        }
    }
};


// ---- a tile ------------------------------------------------------------------
struct Tile {
    int s, t, head, part;
    Tiles tiles;
};

template <typename T>
__device__ __forceinline__ float q_value(const void *p, int64_t i) {
    return to_f(static_cast<const T *>(p)[i]);
}
__device__ __forceinline__ float load_as(int dtype, const void *p, int64_t i) {
    return dtype == DT_BF16  ? q_value<__nv_bfloat16>(p, i)
           : dtype == DT_F16 ? q_value<__half>(p, i)
                             : q_value<float>(p, i);
}
__device__ __forceinline__ void store_as(int dtype, void *p, int64_t i,
                                         float v) {
    if (dtype == DT_BF16)
        static_cast<__nv_bfloat16 *>(p)[i] = __float2bfloat16_rn(v);
    else if (dtype == DT_F16)
        static_cast<__half *>(p)[i] = __float2half_rn(v);
    else
        static_cast<float *>(p)[i] = v;
}

// What column `col` of a tile is: its row of the batch and its query head.
struct Place {
    bool used;
    int32_t row, head;
};
template <int C>
__device__ __forceinline__ Place place_of(const Cut &cut, int first_row,
                                          int rows, int key_head, int part,
                                          int col) {
    const int wide = cut.times < C ? cut.times : C;
    const int r = col / wide, g = part * C + col % wide;
    Place p;
    p.used = r < cut.per && r < rows && g < cut.times;
    p.row = first_row + r;
    p.head = key_head * cut.times + g;
    return p;
}

// Queries and bounds of a tile into shared memory.
template <class H, int PARTS, int NT>
__device__ __forceinline__ void tile_begin(const mt_attention_call_t &c,
                                           const Cut &cut, int dtype,
                                           const Tile &a,
                                           Shared<H, PARTS, NT> &sh) {
    constexpr int C = 8 * NT, kPer = 32 * kWarps / C;  // threads per column
    constexpr int kEach = H::DIM / kPer;
    const int tid = threadIdx.x, col = tid / kPer, sub = tid % kPer;
    const int from = c.offsets[a.s] + a.t * cut.per;
    const int rows = min(cut.per, a.tiles.rows - a.t * cut.per);
    const Place at = place_of<C>(cut, from, rows, a.head, a.part, col);
    float x[kEach];
    float largest = 0.f;
    const int64_t q = (int64_t)at.row * c.q_row + (int64_t)at.head * c.q_head;
#pragma unroll
    for (int i = 0; i < kEach; ++i)
        x[i] = at.used ? load_as(PARTS == 1 ? (int)DT_BF16 : dtype, c.q,
                                 q + sub + kPer * i)
                       : 0.f;
#pragma unroll
    for (int i = 0; i < kEach; ++i) largest = nanmax(largest, fabsf(x[i]));
#pragma unroll
    for (int off = kPer / 2; off > 0; off >>= 1)
        largest = nanmax(largest, __shfl_xor_sync(kFull, largest, off));
    const unsigned e = max(__float_as_uint(largest) >> 23, 15u);
    const bool bad = !(largest < INFINITY);
    const float up = bad ? 0.f : __uint_as_float((268u - e) << 23);
    __half *halves = reinterpret_cast<__half *>(&sh.q[col / 8][0][0][0]);
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
        const int d = sub + kPer * i, r = d % H::B;
        const int step = d / H::B * (H::B / 16) + r % (H::B / 4) / 4;
        const int lane = col % 8 * 4 + r / (H::B / 4);
        const float v = bad ? 0.f : x[i] * up;
        const __half hi = __float2half_rn(v);
        halves[(step * 32 + lane) * 4 + r % 4] = hi;
        if constexpr (PARTS == 2)
            halves[((H::STEPS + step) * 32 + lane) * 4 + r % 4] =
                __float2half_rn(v - __half2float(hi));
    }
    if (sub == 0) {
        Column k = {};
        k.lo = INT32_MIN;
        k.hi = INT32_MAX;
        if (at.used) {
            const int64_t n = (int64_t)c.offsets[a.s + 1] - c.offsets[a.s];
            const int64_t p = (int64_t)c.starts[a.s] +
                              (at.row - c.offsets[a.s]);
            int64_t lo, hi;
            row_sees(c, at.row, p, c.starts[a.s] + n, lo, hi);
            k.f = bad ? NAN : c.scale * __uint_as_float((e - 14u) << 23);
            k.slope = c.slopes ? c.slopes[at.head] : 0.f;
            k.lo = (int32_t)min(lo, (int64_t)INT32_MAX);
            k.hi = (int32_t)max(min(hi, (int64_t)INT32_MAX), (int64_t)-1);
            k.p = (int32_t)min(p, (int64_t)INT32_MAX);
            k.pad = 1;
        }
        sh.column[col] = k;
    }
    __syncthreads();
    if (tid < 32) {
        const Column k = tid < C ? sh.column[tid] : Column{};
        const bool used = k.pad != 0, some = used && k.lo <= k.hi;
        const int lo_any = __reduce_min_sync(kFull, some ? k.lo : INT32_MAX);
        const int hi_any = __reduce_max_sync(kFull, some ? k.hi : -1);
        const int lo_all = __reduce_max_sync(kFull, used ? k.lo : INT32_MIN);
        const int hi_all = __reduce_min_sync(kFull, used ? k.hi : INT32_MAX);
        if (tid == 0) {
            sh.lo_any = lo_any;
            sh.hi_any = hi_any;
            sh.lo_all = lo_all;
            sh.hi_all = hi_all;
        }
    }
    __syncthreads();
}

// The slot of key j, or -1 where no column sees it or it has none.
__device__ __forceinline__ int slot_in(const mt_attention_call_t &c,
                                       const int32_t *pages, int64_t j,
                                       int lo, int hi) {
    if (j < lo || j > hi) return -1;
    const int page = (int)((unsigned)j / (unsigned)c.page_size);
    const int id = pages[page];
    const int64_t slot = (int64_t)id * c.page_size +
                         ((int)j - page * c.page_size);
    return id >= 0 && slot < c.slots ? (int)slot : -1;
}

// A warp's share of the units [u0, u1) of a tile.
template <class H, bool INT8, int PARTS, int NT>
__device__ __forceinline__ void tile_run(const mt_attention_call_t &c,
                                         const Tile &a, int64_t u0, int64_t u1,
                                         const Shared<H, PARTS, NT> &sh,
                                         Warp<H, INT8, PARTS, NT> &w) {
    constexpr int KT = H::KEYS / 16;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int lo = sh.lo_any, hi = sh.hi_any;
    const float inv_cap = c.cap > 0.f ? 1.f / c.cap : 0.f;
    const int32_t *pages = c.table + a.s * c.table_stride;
    if (lo > hi) return;
    u0 = max(u0, (int64_t)(lo / H::KEYS));
    u1 = min(u1, (int64_t)(hi / H::KEYS) + 1);
    int64_t u = u0 + warp;
    if (u >= u1) return;
    const auto slot_at = [&](int64_t v) {
        return v < u1 && lane < H::KEYS
                   ? slot_in(c, pages, v * H::KEYS + lane, lo, hi) : -1;
    };
    int slot = slot_at(u), next = slot_at(u + kWarps);
    w.load_keys(c, a.head, slot);
    w.load_values(c, a.head, slot);
#pragma unroll 1
    for (; u < u1; u += kWarps) {
        const unsigned there = __ballot_sync(kFull, slot >= 0);
        float z[NT][KT][4], keep[NT][2];
        unsigned hidden;
        w.scores(sh, z);
        w.load_keys(c, a.head, next);
        w.bend(c, sh, inv_cap, (int)(u * H::KEYS), there, hidden, z);
        slot = next;
        next = slot_at(u + 2 * kWarps);
        w.weigh(z, keep);
        w.add(z, keep, hidden);
        w.load_values(c, a.head, slot);
    }
}

// The warps' sums of a tile joined: written out where the tile is whole, left
// as partial sums where it is not.
template <class H, bool INT8, int PARTS, int NT>
__device__ __forceinline__ void tile_end(const mt_attention_call_t &c,
                                         const Cut &cut, int dtype,
                                         const Tile &a, bool whole,
                                         float *sums,
                                         Shared<H, PARTS, NT> &sh,
                                         Warp<H, INT8, PARTS, NT> &w) {
    constexpr int C = 8 * NT;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int g = lane >> 2, q = lane & 3;
#pragma unroll
    for (int n = 0; n < NT; ++n) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            float sum = w.l[n][h];
#pragma unroll
            for (int off = 4; off < 32; off <<= 1)
                sum += __shfl_xor_sync(kFull, sum, off);
            if (g == 0) {
                sh.m[warp][8 * n + 2 * q + h] = w.m[n][h];
                sh.l[warp][8 * n + 2 * q + h] = sum;
            }
        }
#pragma unroll
        for (int i = 0; i < H::STEPS; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int d = i / (H::B / 16) * H::B + g * (H::B / 8) +
                              2 * (i % (H::B / 16)) + (e >> 1);
                sh.o[warp][8 * n + 2 * q + (e & 1)][d] = w.o[n][i][e];
            }
    }
    __syncthreads();
    const int from = c.offsets[a.s] + a.t * cut.per;
    const int rows = min(cut.per, a.tiles.rows - a.t * cut.per);
#pragma unroll 1
    for (int i = threadIdx.x; i < C * H::DIM; i += 32 * kWarps) {
        const int col = i / H::DIM, d = i % H::DIM;
        const Place at = place_of<C>(cut, from, rows, a.head, a.part, col);
        if (!at.used) continue;
        float top = sh.m[0][col];
#pragma unroll
        for (int x = 1; x < kWarps; ++x) top = nanmax(top, sh.m[x][col]);
        const float ref = top == -INFINITY ? 0.f : top;
        float sum = 0.f, o = 0.f;
#pragma unroll
        for (int x = 0; x < kWarps; ++x) {
            const float f = pow2(sh.m[x][col] - ref);
            sum = fmaf(sh.l[x][col], f, sum);
            o = fmaf(sh.o[x][col][d], f, o);
        }
        if (whole) {
            store_as(PARTS == 1 ? (int)DT_BF16 : dtype, c.out,
                     (int64_t)at.row * c.out_row +
                         (int64_t)at.head * c.out_head + d,
                     top == -INFINITY ? 0.f : o / sum);
            if (c.lse != nullptr && d == 0)
                c.lse[(int64_t)at.row * c.q_heads + at.head] =
                    top == -INFINITY ? top
                                     : (top + log2f(sum)) * 0.6931471805599453f;
        } else {
            sums[2 * C + i] = o;
            if (d == 0) {
                sums[col] = top;
                sums[C + col] = sum;
            }
        }
    }
    __syncthreads();  // shared memory is the next tile's
}

// The least units that a CTA takes where there are few: one for each warp.
constexpr int kLeastUnits = kWarps;

template <class H, bool INT8, int PARTS, int NT>
__global__ void __launch_bounds__(32 * kWarps, NT == 1 && H::DIM <= 128 ? 3 : 2)
    attention_mma_kernel(const mt_attention_call_t c, const Cut cut,
                         const Share share, int dtype) {
    constexpr int C = 8 * NT, KEYS = H::KEYS, T = 32 * kWarps;
    __shared__ __align__(16) Shared<H, PARTS, NT> sh;
    grid_launch_dependents();
    grid_wait_prerequisites();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    Record record = {};
    // Units of the sequences of this thread, and where they begin.
    const int each = (c.sequences + T - 1) / T;
    const int s0 = min(tid * each, c.sequences);
    const int s1 = min(s0 + each, c.sequences);
    const int64_t wide = (int64_t)c.k_heads * cut.parts;
    const auto units_of = [&](int s) {
        const Tiles t = tiles_of(c, cut, s);
        return wide * t.template before<KEYS>(t.count);
    };
    int64_t mine = 0;
    for (int s = s0; s < s1; ++s) mine += units_of(s);
    int64_t upto = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t v = __shfl_up_sync(kFull, upto, o);
        if (lane >= o) upto += v;
    }
    if (lane == 31) sh.scan[warp] = upto;
    __syncthreads();
    int64_t total = 0, first = upto - mine;
#pragma unroll
    for (int x = 0; x < kWarps; ++x) {
        if (x < warp) first += sh.scan[x];
        total += sh.scan[x];
    }
    const int64_t ctas = min((int64_t)gridDim.x,
                             (total + kLeastUnits - 1) / kLeastUnits);
    int64_t at = 0, end = 0;
    if (blockIdx.x < ctas) {
        at = total * blockIdx.x / ctas;
        end = total * (blockIdx.x + 1) / ctas;
    }
    if (at < end) {
        if (first <= at && at < first + mine) {
            int64_t left = at - first;
            int s = s0;
            for (;; ++s) {
                const int64_t n = units_of(s);
                if (left < n) break;
                left -= n;
            }
            sh.sequence = s;
            sh.at = left;
        }
        __syncthreads();
        Tile a;
        a.s = sh.sequence;
        int64_t off = sh.at;
        a.tiles = tiles_of(c, cut, a.s);
        int lo = 0, hi = a.tiles.count;  // before(lo) <= off < before(hi)
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (wide * a.tiles.template before<KEYS>(mid) <= off) lo = mid;
            else hi = mid;
        }
        a.t = lo;
        off -= wide * a.tiles.template before<KEYS>(lo);
        int64_t base = a.tiles.template first<KEYS>(lo);
        int64_t units = a.tiles.template last<KEYS>(lo) - base + 1;
        int index = (int)(off / units);
        off -= index * units;
        Warp<H, INT8, PARTS, NT> w;
        while (at < end) {
            const int64_t n = min(units - off, end - at);
            a.head = index / cut.parts;
            a.part = index - a.head * cut.parts;
            tile_begin<H, PARTS, NT>(c, cut, dtype, a, sh);
            w.begin();
            tile_run<H, INT8, PARTS, NT>(c, a, base + off, base + off + n, sh,
                                         w);
            const bool whole = n == units;
            if (!whole && off == 0) {
                const int64_t x = at + units;
                record.valid = 1;
                record.last = (int)((x * ctas - 1) / total);
                record.row = c.offsets[a.s] + a.t * cut.per;
                record.rows = min(cut.per, a.tiles.rows - a.t * cut.per);
                record.head = a.head;
                record.part = a.part;
            }
            tile_end<H, INT8, PARTS, NT>(
                c, cut, dtype, a, whole,
                share.sums + (2 * (int64_t)blockIdx.x + (off == 0 ? 1 : 0)) *
                                 place_floats(C, H::DIM),
                sh, w);
            at += n;
            off = 0;
            if (at < end && ++index == wide) {
                index = 0;
                if (++a.t == a.tiles.count) {
                    a.t = 0;
                    do a.tiles = tiles_of(c, cut, ++a.s);
                    while (a.tiles.rows == 0);
                }
                base = a.tiles.template first<KEYS>(a.t);
                units = a.tiles.template last<KEYS>(a.t) - base + 1;
            }
        }
    }
    if (tid == 0) share.records[blockIdx.x] = record;
}

// Joins the parts of a cut tile, in the order of the CTAs that left them.
template <int DIM, int C>
__global__ void __launch_bounds__(128)
    attention_join_kernel(const mt_attention_call_t c, const Cut cut,
                          const Share share, int dtype) {
    grid_launch_dependents();
    grid_wait_prerequisites();
    const Record r = share.records[blockIdx.x];
    if (!r.valid) return;
    constexpr int64_t kPlace = place_floats(C, DIM);
    const float *begin = share.sums + (2 * (int64_t)blockIdx.x + 1) * kPlace;
    const float *others = share.sums + 2 * kPlace * (blockIdx.x + 1);
    const int more = r.last - (int)blockIdx.x;
    const auto part = [&](int i) {
        return i == 0 ? begin : others + 2 * kPlace * (i - 1);
    };
    for (int i = blockIdx.y * 128 + threadIdx.x; i < C * DIM;
         i += 128 * gridDim.y) {
        const int col = i / DIM, d = i % DIM;
        const Place at = place_of<C>(cut, r.row, r.rows, r.head, r.part, col);
        if (!at.used) continue;
        float top = -INFINITY, sum = 0.f, o = 0.f;
#pragma unroll 4
        for (int x = 0; x <= more; ++x) {
            const float *p = part(x);
            const float m = p[col], l = p[C + col], v = p[2 * C + i];
            const float next = nanmax(top, m);
            const float ref = next == -INFINITY ? 0.f : next;
            const float a = pow2(top - ref), b = pow2(m - ref);
            sum = sum * a + l * b;
            o = o * a + v * b;
            top = next;
        }
        store_as(dtype, c.out,
                 (int64_t)at.row * c.out_row + (int64_t)at.head * c.out_head +
                     d,
                 top == -INFINITY ? 0.f : o / sum);
        if (c.lse != nullptr && d == 0)
            c.lse[(int64_t)at.row * c.q_heads + at.head] =
                top == -INFINITY ? top
                                 : (top + log2f(sum)) * 0.6931471805599453f;
    }
}

template <class H, bool INT8, int PARTS, int NT>
cudaError_t launch_attention_as(const AttentionPlan &p,
                                const mt_attention_call_t &c, int dtype,
                                void *workspace, cudaStream_t s) {
    const Cut cut = {p.times, p.per, p.parts};
    Share share;
    share.sums = static_cast<float *>(workspace);
    share.records = reinterpret_cast<Record *>(
        share.sums + 2 * (int64_t)p.ctas * place_floats(8 * NT, H::DIM));
    cudaError_t e = launch_dependent(attention_mma_kernel<H, INT8, PARTS, NT>,
                                     p.ctas, 32 * kWarps, 0, s, c, cut, share,
                                     dtype);
    if (e != cudaSuccess) return e;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)p.ctas, 2);
    cfg.blockDim = dim3(128);
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, attention_join_kernel<H::DIM, 8 * NT>, c,
                              cut, share, dtype);
}

template <bool INT8, int PARTS, int NT>
cudaError_t launch_attention(const AttentionPlan &p,
                             const mt_attention_call_t &c, int dtype,
                             void *workspace, cudaStream_t s) {
#define MT_ATTENTION_HEAD(d, g)                                              \
    if (c.dim == d && c.dim / c.group == g)                                  \
        return launch_attention_as<Head<d, g>, INT8, PARTS, NT>(             \
            p, c, dtype, workspace, s);
    MT_ATTENTION_HEAD(64, 1)
    MT_ATTENTION_HEAD(64, 2)
    MT_ATTENTION_HEAD(80, 1)
    MT_ATTENTION_HEAD(96, 1)
    MT_ATTENTION_HEAD(128, 1)
    MT_ATTENTION_HEAD(128, 2)
    MT_ATTENTION_HEAD(128, 4)
    if constexpr (NT == 1) {
        MT_ATTENTION_HEAD(256, 1)
        MT_ATTENTION_HEAD(256, 2)
        MT_ATTENTION_HEAD(256, 8)
    }
#undef MT_ATTENTION_HEAD
    return cudaErrorInvalidValue;
}

}  // namespace

#define MT_DEFINE_ATTENTION(name, int8, parts, nt)                           \
    cudaError_t name(const AttentionPlan &p, const mt_attention_call_t &c,   \
                     int dtype, void *workspace, cudaStream_t s) {           \
        return launch_attention<int8, parts, nt>(p, c, dtype, workspace, s); \
    }

}  // namespace mt

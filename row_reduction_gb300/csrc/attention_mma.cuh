// attention_mma.cuh -- attention over the quantised cache on matrix
// instructions (one translation unit per code format).
//
// Scores are formed transposed, keys x queries (S^T = K Q^T), so that the
// cache's codes, which are the long operand, fill the instruction's 16 rows and
// the few query heads that share a key head its 8 columns.  A warp goes through
// chunks of keys of its own: codes are copied into shared
// memory of the warp's own by asynchronous copies, a chunk ahead of the one that
// is worked on, and widened to FP16 on the way into fragments, exactly (the
// order of the dimensions is free as long as queries have the same, so a lane
// reads up to 16 bytes of a key at once).  What the scores give
// turns into the other product's operand (O^T = V^T P^T) by one transposition
// of 8 x 8 values within the warp.
//
// The four warps of a CTA take key heads of the same keys, as many as divide the
// call's (4, 2 or 1; the warps that are left share a head's keys): rows and
// scales of neighbouring heads lie side by side, and a head's scale alone is 4
// bytes of a sector of 32, which the other heads' CTAs would fetch again.
//
// Scales.  A key's factor multiplies its score's sum of each group, a value's
// the weight that goes into the product of that group.
//
// Roundings to FP16.  Codes are exact.  Queries are held as a power of two
// times FP16 with the head's largest value at 2^14..2^15, BF16 and FP16 values
// exactly (down to 2^-28 of the largest), FP32 in two parts (2^-22).  Weights
// times the values' scales are held likewise, their largest so far at
// 2^11..2^12 or above: one part for BF16 output (half a step 2^-11 of a weight,
// an eighth of the output's own), two for FP16 and FP32.  Against 64 bits outputs
// are off by 1.7e-3 rms with one part and with two, which is the rounding to
// BF16; two would bring them within 1e-4 of FP32 sums rounded once for 9e-4, at 210
// us in place of 205 (64 sequences to 16384 keys), 128 of 121 (heads of 64) and
// 90 of 83 (one of 131072, capped).  Sums are FP32: for BF16 output the
// instruction's own all along, else its sums of a chunk, added up to nearest.
//
// References.  A column's weights are exponentials about a reference that
// follows its largest score only where that runs 2^8 ahead, and the power of
// two under a group's weights where they pass 2^15: one vote tells that neither
// is so, which holds for nearly all chunks, and saves the exchange of maxima
// among lanes and the scaling of the sums.
//
// Work is dealt out in units, one chunk for each warp of one tile (rows of a
// sequence and the query heads of a key head, up to 8 NT columns, for each of
// the CTA's key heads): every CTA takes an
// equal run of all units of the batch in their order, wherever sequences begin
// and end in it, so that lengths of any mixture fill the device and nothing
// about them need be known on the host.  A tile that is cut by the ends of
// runs is left as partial sums, which a second kernel joins in order.
//
// Bound.  Long contexts by memory: 64 sequences to 16384 keys, 8 key heads of
// 128, BF16 200-205 us, 6.2 TB/s, 93-91% of the measured copy bandwidth (heads of
// 64 121 us, 79%: more chunks to the byte).  Short ones by a chain of waits: plan,
// queries, first keys, two or three chunks of some 2000 cycles a warp, sums, and
// the second kernel: eight sequences to 2048 keys 21 us.  One sequence of 131072
// keys, two groups a head, capped, 83 us, 51% (uncapped 77): each CTA has 27
// chunks a warp.  Half of the variants spill some words, 92 bytes at most (two
// parts, tiles of 16 columns).
//
// Two CTAs per SM of heads of 128 (three: 250 us for 242 before key heads shared
// a CTA): registers for a chunk's fragments count for more than warps.
#pragma once

#include "attention.cuh"

namespace mt {
namespace {

constexpr int kWarps = 4;

// ---- sums of a tile's units ----------------------------------------------------
// a / b for a >= 0, b > 0; in 32 bits, many times quicker, where they fit.
__device__ __forceinline__ int64_t quotient(int64_t a, int64_t b) {
    if (((uint64_t)(a | b) >> 32) == 0)
        return (int64_t)((unsigned)a / (unsigned)b);
    return a / b;
}
// sum over 0 <= t < n of floor((a t + b) / 2^log2), for a, b >= 0: whole parts
// aside, the points under a line, counted along the other axis in turn (slopes
// below 2^log2 from there on).
__device__ __forceinline__ int64_t floor_sum(int64_t n, int log2, int64_t a,
                                             int64_t b) {
    const int64_t low = (1LL << log2) - 1;
    int64_t s = (n - 1) * n / 2 * (a >> log2) + n * (b >> log2);
    int m = 1 << log2, slope = (int)(a & low), at = (int)(b & low);
    for (int64_t y = slope * n + at; y >= m; y = slope * n + at) {
        n = quotient(y, m);
        at = (int)(y - n * m);
        const int x = m / slope;
        s += (n - 1) * n / 2 * x + n * (at / slope);
        const int rest = m - x * slope;
        at %= slope;
        m = slope;
        slope = rest;
    }
    return s;
}

// A tile's begin and end (queries, the first keys' way, the warps' sums
// joined) in units: without them runs of short sequences are the last to end.
constexpr int64_t kExtra = 2;

// How the call's rows and heads are cut.
struct Cut {
    int32_t times;   // query heads per key head
    int32_t per;     // rows of a tile
    int32_t parts;   // tiles that share a row's query heads
    int32_t heads;   // key heads of a CTA: 4, 2 or 1
    int32_t log2;    // keys of a unit
    int32_t wide;    // tiles of the same rows: groups of key heads, parts
    int32_t whole;   // bits: q, out take 4 values at a time
};

// How the rows of a sequence are cut into tiles and units.
struct Tiles {
    int64_t start;   // position of the first row
    int32_t rows;    // of the sequence
    int32_t per;     // rows of a tile
    int32_t count;   // tiles
    int32_t window;
    int32_t log2;
    bool all;        // every tile goes through all keys (last bounds)
    // Tile t's first and last unit of keys (of what its rows may see).
    __device__ __forceinline__ int64_t first(int t) const {
        if (window == 0) return 0;
        return max(start + (int64_t)t * per - window + 1, (int64_t)0) >> log2;
    }
    __device__ __forceinline__ int64_t last(int t) const {
        const int64_t r = all ? rows : min((int64_t)(t + 1) * per,
                                           (int64_t)rows);
        return (start + r - 1) >> log2;
    }
    // Units of the tiles before t (first <= last in every tile), kExtra to
    // each for what a tile costs besides.
    __device__ __forceinline__ int64_t before(int t) const {
        if (t <= 0) return 0;
        int64_t s = (1 + kExtra) * (int64_t)t;
        if (t == 1) return s + last(0) - first(0);
        if (all) {
            s += t * last(0);
        } else {
            // all tiles but the sequence's last are whole
            const int whole = t < count ? t : count - 1;
            s += floor_sum(whole, log2, per, start + per - 1);
            if (t > whole) s += last(count - 1);
        }
        if (window != 0) {
            // from tile z on the window's begin is not negative
            const int64_t short_of = window - 1 - start;
            const int64_t z = short_of <= 0 ? 0 : (short_of + per - 1) / per;
            if (t > z)
                s -= floor_sum(t - z, log2, per,
                               start + z * per - window + 1);
        }
        return s;
    }
};

__device__ __forceinline__ Tiles tiles_of(const mt_attention_call_t &c,
                                          const Cut &cut, int s) {
    Tiles t;
    const int64_t n = (int64_t)begin_of(c, s + 1) - begin_of(c, s);
    t.start = max(c.starts[s], 0);
    t.rows = (int32_t)max(n, (int64_t)0);
    t.per = cut.per;
    t.count = (t.rows + cut.per - 1) / cut.per;
    // rows at negative positions see nothing; their tiles begin at key 0
    t.window = c.starts[s] < 0 ? 0 : c.window;
    t.log2 = cut.log2;
    t.all = c.last != nullptr;
    return t;
}

// A cut tile that begins in a CTA's run: where its parts lie and what it is.
struct Record {
    int32_t last;             // the CTA that holds its end
    int32_t row, rows;        // rows of the batch
    int32_t head, part;       // first key head; part of the row's query heads
};
struct Share {
    Record *records;          // one per CTA, where it has a cut tile
    int32_t *cut;             // one per CTA: whether it has
    float *sums;              // two places per CTA: m, l, O of each column of
                              // each of its key heads
};

// columns: of all of a CTA's key heads.
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
        asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\t"
            "cvt.rn.f16x2.e4m3x2 %0, l;\n\tcvt.rn.f16x2.e4m3x2 %1, h;\n\t}"
            : "=r"(lo), "=r"(hi) : "r"(w));
    }
}

// `bytes` (a constant: 16, 8, 4 or 2) of codes from shared memory into words.
__device__ __forceinline__ void read_codes(const uint8_t *p, int bytes,
                                           unsigned *w) {
    if (bytes == 16) {
        const uint4 v = *reinterpret_cast<const uint4 *>(p);
        w[0] = v.x; w[1] = v.y; w[2] = v.z; w[3] = v.w;
    } else if (bytes == 8) {
        const uint2 v = *reinterpret_cast<const uint2 *>(p);
        w[0] = v.x; w[1] = v.y;
    } else if (bytes == 4) {
        w[0] = *reinterpret_cast<const unsigned *>(p);
    } else {
        w[0] = *reinterpret_cast<const uint16_t *>(p);
    }
}

// 16 bytes from global into shared memory, on their way; zeros where not `on`.
__device__ __forceinline__ void copy16(void *to, const void *from, bool on) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(
                     smem_addr(to)),
                 "l"(from), "r"(on ? 16 : 0)
                 : "memory");
}
// A key's scales into shared memory, on their way; zeros where not `on`.
template <int BYTES>
__device__ __forceinline__ void copy_scales(void *to, const void *from,
                                            bool on) {
    if constexpr (BYTES > 16) {
        copy_scales<16>(to, from, on);
        copy_scales<BYTES - 16>(static_cast<char *>(to) + 16,
                                static_cast<const char *>(from) + 16, on);
    } else {
        asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;" ::"r"(
                         (unsigned)__cvta_generic_to_shared(to)),
                     "l"(from), "n"(BYTES), "r"(on ? BYTES : 0)
                     : "memory");
    }
}

// ---- a head's layout -------------------------------------------------------------
struct Block {
    int base, size;
};
template <int DIM_, int GROUPS_>
struct Head {
    static constexpr int DIM = DIM_, GROUPS = GROUPS_;
    static constexpr int GROUP = DIM / GROUPS;
    static constexpr int KEYS = DIM > 128 ? 16 : 32;  // of a chunk
    static constexpr int STEPS = DIM / 16;            // of the instruction
    static constexpr int PER = GROUP / 16;            // of a group
    // A group's dimensions come in blocks of 128, 64, 32 and 16, the largest
    // that fit first.  Of a block, lane l of a quad holds the size/4 bytes from
    // l size/4 on of a key, a word of them for each step, and lane l of eight
    // the size/8 bytes from l size/8 on of a value, two of them for each step.
    static __host__ __device__ constexpr Block block(int step) {
        int base = 0;
        for (int size = 128; size >= 16; size /= 2)
            while (GROUP - base >= size) {
                if (step * 16 < base + size) return {base, size};
                base += size;
            }
        return {0, 0};
    }
    // Where byte `byte` of key `key` of a chunk is in shared memory: units of
    // 16 bytes permuted by the key, so that what a quarter of a warp reads at
    // once lies in different banks.
    static __device__ __forceinline__ int place(int key, int byte) {
        if (DIM % 128 == 0) return key * DIM + (byte ^ (key & 7) << 4);
        if (DIM == 64) return key * 64 + (byte ^ (key >> 1 & 3) << 4);
        return key * DIM + byte;
    }
};

// A column of a tile: one row's query head.
struct Column {
    int32_t lo, hi;     // keys that it sees
    int32_t p;          // its row's position
    int32_t pad;
};

struct Deal {
    int64_t scan[2 * kWarps];
    int64_t at;         // place of the CTA's first unit in its sequence
    int32_t sequence;
};

template <class H, int PARTS, int NT>
struct Shared {
    // Each warp's own: the codes of two chunks, then its sums.
    struct Codes {
        uint8_t k[H::KEYS * H::DIM], v[H::KEYS * H::DIM];
    };
    union Own {
        Codes codes[2];
        float o[8 * NT][H::DIM + 4];
    };
    struct Scales {
        float k[H::KEYS][H::GROUPS], v[H::KEYS][H::GROUPS];
    };
    Own own[kWarps];
    Scales scales[kWarps][2];
    uint2 q[kWarps][NT][PARTS][H::STEPS][32];  // fragments, of each key head
    Column column[8 * NT];
    // Of each key head's columns: what the product takes to be a score in units
    // of log 2, the scale and the query's power of two; the slope in those units.
    float f[kWarps][8 * NT], slope[kWarps][8 * NT];
    int32_t lo_any, hi_any, lo_all, hi_all;
    float m[kWarps][8 * NT], l[kWarps][8 * NT];
    Deal deal;
    static_assert(sizeof(Own) == 2 * sizeof(Codes), "room for the sums");
};

// A key head of the cache, at slot 0, and the strides of slots.
struct Cache {
    const uint8_t *k, *v;
    const float *ks, *vs;
    unsigned row, scales;
};

template <class H, bool INT8, int PARTS, int NT>
struct Warp {
    static constexpr int KT = H::KEYS / 16;     // rows of 16 keys
    using Codes = typename Shared<H, PARTS, NT>::Codes;
    using Scales = typename Shared<H, PARTS, NT>::Scales;
    float o[NT][H::STEPS][4];        // in units of 2^-(up of its group)
    float ref[NT][2], l[NT][2];
    int hs;                          // which of the CTA's key heads
    // Exponent bits of the largest weight times scale so far, of each column
    // and group; four to a word.
    unsigned most[NT][2][(H::GROUPS + 3) / 4];

    __device__ __forceinline__ void begin() {
#pragma unroll
        for (int n = 0; n < NT; ++n) {
#pragma unroll
            for (int i = 0; i < H::STEPS; ++i)
#pragma unroll
                for (int e = 0; e < 4; ++e) o[n][i][e] = 0.f;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                ref[n][h] = -INFINITY;
                l[n][h] = 0.f;
#pragma unroll
                for (int i = 0; i < (H::GROUPS + 3) / 4; ++i)
                    most[n][h][i] = 0;
            }
        }
    }
    __device__ __forceinline__ unsigned exponent(int n, int h, int gr) const {
        return max(most[n][h][gr / 4] >> gr % 4 * 8 & 0xffu, 12u);
    }
    // 2^11 over the power of two under the largest, and its inverse.
    static __device__ __forceinline__ float up(unsigned e) {
        return __uint_as_float((265u - e) << 23);
    }
    static __device__ __forceinline__ float down(unsigned e) {
        return __uint_as_float((e - 11u) << 23);
    }
    // A chunk's codes and scales on their way; slot: of the chunk's key `lane`,
    // or -1, whose place is filled with zeros (its weights will be zero, but
    // what stands elsewhere may be NaN).
    __device__ __forceinline__ void load(const Cache &c, int slot, Codes &to,
                                         Scales &scales) {
        constexpr int kPieces = H::DIM / 16;  // of a key
        const int lane = threadIdx.x & 31;
#pragma unroll
        for (int i = 0; i < H::KEYS * kPieces / 32; ++i) {
            const int piece = lane + 32 * i;
            const int key = piece / kPieces, at = piece % kPieces * 16;
            const int s = __shfl_sync(kFull, slot, key);
            const uint64_t from = (uint64_t)(unsigned)max(s, 0) * c.row + at;
            copy16(to.k + H::place(key, at), c.k + from, s >= 0);
            copy16(to.v + H::place(key, at), c.v + from, s >= 0);
        }
        if (lane < H::KEYS) {
            const uint64_t from = (uint64_t)(unsigned)max(slot, 0) * c.scales;
            copy_scales<4 * H::GROUPS>(scales.k[lane], c.ks + from, slot >= 0);
            copy_scales<4 * H::GROUPS>(scales.v[lane], c.vs + from, slot >= 0);
        }
    }
    // A group's products from step S on: half a block of 128 at a time, 16
    // bytes of a key (steps as template arguments: in loops whose step varies
    // the fragments went through local memory).
    template <int S>
    __device__ __forceinline__ void score_blocks(
        const Shared<H, PARTS, NT> &sh, const Codes &st, int gr,
        float (&acc)[NT][KT][4]) {
        if constexpr (S < H::PER) {
            constexpr Block block = H::block(S);
            constexpr int size = block.size > 64 ? 64 : block.size;
            const int lane = threadIdx.x & 31, g = lane >> 2, q = lane & 3;
            const int at = gr * H::GROUP + block.base + q * (block.size / 4) +
                           4 * (S - block.base / 16);
            unsigned k[KT][2][4];
#pragma unroll
            for (int t = 0; t < KT; ++t)
#pragma unroll
                for (int i = 0; i < 2; ++i)
                    read_codes(st.k + H::place(16 * t + 8 * i + g, at & ~15) +
                                   (at & 15),
                               size / 4, k[t][i]);
#pragma unroll
            for (int x = 0; x < size / 16; ++x) {
                unsigned a[KT][4];
#pragma unroll
                for (int t = 0; t < KT; ++t) {
                    widen4<INT8>(k[t][0][x], a[t][0], a[t][2]);
                    widen4<INT8>(k[t][1][x], a[t][1], a[t][3]);
                }
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int part = 0; part < PARTS; ++part) {
                        const uint2 v =
                            sh.q[hs][n][part][gr * H::PER + S + x][lane];
#pragma unroll
                        for (int t = 0; t < KT; ++t)
                            mma16816(acc[n][t], a[t], v.x, v.y);
                    }
            }
            score_blocks<S + size / 16>(sh, st, gr, acc);
        }
    }
    // Sums of codes times queries times the keys' scales.
    __device__ __forceinline__ void scores(const Shared<H, PARTS, NT> &sh,
                                           const Codes &st,
                                           const Scales &scales,
                                           float (&z)[NT][KT][4]) {
        const int g = (threadIdx.x & 31) >> 2;
#pragma unroll
        for (int gr = 0; gr < H::GROUPS; ++gr) {
            float acc[NT][KT][4];
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int t = 0; t < KT; ++t)
#pragma unroll
                    for (int e = 0; e < 4; ++e) acc[n][t][e] = 0.f;
            score_blocks<0>(sh, st, gr, acc);
#pragma unroll
            for (int t = 0; t < KT; ++t)
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const float f = scales.k[16 * t + 8 * i + g][gr];
#pragma unroll
                    for (int n = 0; n < NT; ++n)
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            float &to = z[n][t][2 * i + h];
                            const float from = acc[n][t][2 * i + h];
                            to = gr == 0 ? from * f : fmaf(from, f, to);
                        }
                }
        }
    }
    // Scores to exponents of two; -infinity, and a bit of `hidden`, for keys
    // that a column does not see.  j0: the chunk's first key; there: its keys
    // that have a slot.  Returns whether there may be any such key.
    __device__ __forceinline__ bool bend(const mt_attention_call_t &c,
                                         const Shared<H, PARTS, NT> &sh,
                                         int j0, unsigned there,
                                         unsigned &hidden,
                                         float (&z)[NT][KT][4]) {
        hidden = 0;
        const int lane = threadIdx.x & 31, g = lane >> 2, q = lane & 3;
        constexpr unsigned kAll = H::KEYS == 32 ? ~0u : 0xffffu;
        const bool whole = there == kAll && j0 >= sh.lo_all &&
                           j0 + H::KEYS - 1 <= sh.hi_all;
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const float f = sh.f[hs][8 * n + 2 * q + h];
#pragma unroll
                for (int t = 0; t < KT; ++t)
#pragma unroll
                    for (int i = 0; i < 2; ++i) z[n][t][2 * i + h] *= f;
            }
        if (c.cap > 0.f) {
            const Cap cap(c.cap, kLog2e);
#pragma unroll
            for (int n = 0; n < NT; ++n) cap_scores(cap, z[n]);
        }
        if (c.slopes == nullptr && whole) return false;
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const Column &col = sh.column[8 * n + 2 * q + h];
                const float slope = sh.slope[hs][8 * n + 2 * q + h];
#pragma unroll
                for (int t = 0; t < KT; ++t)
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const int at = 16 * t + 8 * i + g;
                        float &v = z[n][t][2 * i + h];
                        if (c.slopes != nullptr)
                            v -= slope * (float)abs(col.p - (j0 + at));
                        if (!whole &&
                            !(there >> at & 1u && j0 + at >= col.lo &&
                              j0 + at <= col.hi)) {
                            v = -INFINITY;
                            hidden |= 1u << (4 * (n * KT + t) + 2 * i + h);
                        }
                    }
            }
        return !whole;
    }
    // Weights about the columns' references, which move where a score is 2^8
    // ahead of one (or there is none yet, or something is NaN).
    __device__ __forceinline__ void weigh(float (&z)[NT][KT][4]) {
        bool ahead = false;
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                float top = nanmax(z[n][0][h], z[n][0][2 + h]);
#pragma unroll
                for (int t = 1; t < KT; ++t)
                    top = nanmax3(top, z[n][t][h], z[n][t][2 + h]);
                ahead |= !(top <= ref[n][h] + 8.f);
            }
        if (__any_sync(kFull, ahead)) move(z);
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const float about = ref[n][h] == -INFINITY ? 0.f : ref[n][h];
#pragma unroll
                for (int t = 0; t < KT; ++t)
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        float &w = z[n][t][2 * i + h];
                        w = pow2(w - about);
                        l[n][h] += w;
                    }
            }
    }
    // References to the columns' largest scores; sums and exponents follow.
    __device__ __forceinline__ void move(const float (&z)[NT][KT][4]) {
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            float keep[2];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                float top = ref[n][h];
#pragma unroll
                for (int t = 0; t < KT; ++t)
#pragma unroll
                    for (int i = 0; i < 2; ++i)
                        top = nanmax(top, z[n][t][2 * i + h]);
#pragma unroll
                for (int off = 4; off < 32; off <<= 1)
                    top = nanmax(top, __shfl_xor_sync(kFull, top, off));
                keep[h] = pow2(ref[n][h] - (top == -INFINITY ? 0.f : top));
                ref[n][h] = top;
                l[n][h] *= keep[h];
                // the exponents of the largest so far in the new units: down by
                // as many powers of two, to the sums' own where that is less
                const unsigned less =
                    127u - min(__float_as_uint(keep[h]) >> 23, 127u);
#pragma unroll
                for (int gr = 0; gr < H::GROUPS; ++gr) {
                    const unsigned old = exponent(n, h, gr);
                    const unsigned now = max(old > less ? old - less : 0u, 12u);
                    set(n, h, gr, now);
                    const float f = keep[h] * up(now) * down(old);
#pragma unroll
                    for (int i = gr * H::PER; i < (gr + 1) * H::PER; ++i) {
                        o[n][i][h] *= f;
                        o[n][i][2 + h] *= f;
                    }
                }
            }
        }
    }
    __device__ __forceinline__ void set(int n, int h, int gr, unsigned e) {
        unsigned &w = most[n][h][gr / 4];
        w = (w & ~(0xffu << gr % 4 * 8)) | e << gr % 4 * 8;
    }
    // A group's weights times scales, a power of two up, within FP16's range:
    // where they pass it, or the largest so far is left far behind by the first
    // that come, that power moves.
    __device__ __forceinline__ void scaled(const float (&w)[NT][KT][4],
                                           unsigned hidden,
                                           bool masked,
                                           const Scales &scales, int gr,
                                           float (&x)[NT][KT][4]) {
        const int g = (threadIdx.x & 31) >> 2;
        float scale[KT][2];
#pragma unroll
        for (int t = 0; t < KT; ++t)
#pragma unroll
            for (int i = 0; i < 2; ++i)
                scale[t][i] = scales.v[16 * t + 8 * i + g][gr];
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int t = 0; t < KT; ++t)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    x[n][t][e] = w[n][t][e] * scale[t][e >> 1];
        if (masked) {
            // not seen: nothing, whatever stands in the scale
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int t = 0; t < KT; ++t)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        if (hidden >> (4 * (n * KT + t) + e) & 1u)
                            x[n][t][e] = 0.f;
        }
        float most_x = 0.f;
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            const float f[2] = {up(exponent(n, 0, gr)), up(exponent(n, 1, gr))};
#pragma unroll
            for (int t = 0; t < KT; ++t) {
#pragma unroll
                for (int e = 0; e < 4; ++e) x[n][t][e] *= f[e & 1];
                most_x = nanmax3(most_x, fabsf(x[n][t][0]), fabsf(x[n][t][1]));
                most_x = nanmax3(most_x, fabsf(x[n][t][2]), fabsf(x[n][t][3]));
            }
        }
        const bool out = !(most_x < 32768.f);
        if (__any_sync(kFull, out)) raise(w, hidden, scale, gr, x);
    }
    __device__ __forceinline__ void raise(const float (&w)[NT][KT][4],
                                       unsigned hidden,
                                       const float (&scale)[KT][2], int gr,
                                       float (&x)[NT][KT][4]) {
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            unsigned e0 = 0, e1 = 0;
#pragma unroll
            for (int t = 0; t < KT; ++t)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    x[n][t][e] = hidden >> (4 * (n * KT + t) + e) & 1u
                                     ? 0.f : w[n][t][e] * scale[t][e >> 1];
                    const unsigned bits =
                        __float_as_uint(fabsf(x[n][t][e])) >> 23;
                    if (e & 1) e1 = max(e1, bits);
                    else e0 = max(e0, bits);
                }
            unsigned ex = e0 | e1 << 16;
#pragma unroll
            for (int off = 4; off < 32; off <<= 1)
                ex = __vmaxu2(ex, __shfl_xor_sync(kFull, ex, off));
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                unsigned old = 0, now = 0;
#pragma unroll
                for (int r = 0; r < H::GROUPS; ++r)
                    if (r == gr) {
                        old = exponent(n, h, r);
                        now = max(old, h ? ex >> 16 : ex & 0xffffu);
                        set(n, h, r, now);
                        const float f = up(now) * down(old);
#pragma unroll
                        for (int i = r * H::PER; i < (r + 1) * H::PER; ++i) {
                            o[n][i][h] *= f;
                            o[n][i][2 + h] *= f;
                        }
                    }
#pragma unroll
                for (int t = 0; t < KT; ++t) {
                    x[n][t][h] *= up(now);
                    x[n][t][2 + h] *= up(now);
                }
            }
        }
    }
    // A group's weighted values from step S on.  Two rows of the output per
    // lane and step: two bytes of its own of a value; a pair of keys side by
    // side.
    template <int S>
    __device__ __forceinline__ void value_blocks(
        const Codes &st, int gr, const unsigned (&b)[NT][PARTS][KT][2]) {
        if constexpr (S < H::PER) {
            constexpr Block block = H::block(S);
            const int g = (threadIdx.x & 31) >> 2, q = threadIdx.x & 3;
            const int at = gr * H::GROUP + block.base + g * (block.size / 8);
            unsigned v[KT][4][4];
#pragma unroll
            for (int t = 0; t < KT; ++t)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    read_codes(st.v + H::place(16 * t + 2 * q + (i & 1) +
                                                   8 * (i >> 1),
                                               at & ~15) + (at & 15),
                               block.size / 8, v[t][i]);
#pragma unroll
            for (int m = 0; m < block.size / 16; ++m) {
                unsigned a[KT][4];
#pragma unroll
                for (int t = 0; t < KT; ++t)
#pragma unroll
                    for (int y = 0; y < 2; ++y)
                        widen4<INT8>(__byte_perm(v[t][2 * y][m / 2],
                                                 v[t][2 * y + 1][m / 2],
                                                 m & 1 ? 0x7362 : 0x5140),
                                     a[t][2 * y], a[t][2 * y + 1]);
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    float (&to)[4] = o[n][gr * H::PER + S + m];
                    if constexpr (PARTS == 1) {
#pragma unroll
                        for (int t = 0; t < KT; ++t)
                            mma16816(to, a[t], b[n][0][t][0], b[n][0][t][1]);
                    } else {
                        float acc[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                        for (int part = 0; part < PARTS; ++part)
#pragma unroll
                            for (int t = 0; t < KT; ++t)
                                mma16816(acc, a[t], b[n][part][t][0],
                                         b[n][part][t][1]);
#pragma unroll
                        for (int e = 0; e < 4; ++e) to[e] += acc[e];
                    }
                }
            }
            value_blocks<S + block.size / 16>(st, gr, b);
        }
    }
    // Adds the chunk's weights times values.
    __device__ __forceinline__ void add(const float (&w)[NT][KT][4],
                                        unsigned hidden, bool masked,
                                        const Codes &st,
                                        const Scales &scales) {
#pragma unroll
        for (int gr = 0; gr < H::GROUPS; ++gr) {
            unsigned b[NT][PARTS][KT][2];
            {
                float x[NT][KT][4];
                scaled(w, hidden, masked, scales, gr, x);
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int t = 0; t < KT; ++t)
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            const float lo = x[n][t][2 * i];
                            const float hi = x[n][t][2 * i + 1];
                            const unsigned h = half_pair(lo, hi);
                            b[n][0][t][i] = transpose8x8(h);
                            if constexpr (PARTS == 2) {
                                const float2 r = from_half_pair(h);
                                b[n][1][t][i] =
                                    transpose8x8(half_pair(lo - r.x,
                                                           hi - r.y));
                            }
                        }
            }
            value_blocks<0>(st, gr, b);
        }
    }
};

// ---- a tile ------------------------------------------------------------------
struct Tile {
    int s, t;
    int head;       // the first of the CTA's key heads
    int part;
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

// Columns of a tile that stand for something; they are the first ones.
template <int C>
__device__ __forceinline__ int columns_of(const Cut &cut, int rows, int part) {
    return cut.times <= C ? rows * cut.times : min(cut.times - part * C, C);
}

// A warp's part of the queries of a tile: the columns of its key head that are
// its own among the warps of that head, four values to a lane (one access each
// where they can: the CTAs of a sequence all ask for the same few lines).
template <class H, int PARTS, int NT>
struct Queries {
    static constexpr int C = 8 * NT, kEach = (H::DIM / 4 + 31) / 32;
    static constexpr int kWords = PARTS == 1 ? 2 : 4;
    unsigned x[C][kEach][kWords];
    template <typename T>
    static __device__ __forceinline__ void four(const void *q, int64_t at,
                                                bool whole, unsigned *w) {
        const T *p = static_cast<const T *>(q) + at;
        Raw<T, 4> r;
        if (whole) {
            r.load(p);
        } else {
            float v[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) v[e] = to_f(p[e]);
#pragma unroll
            for (int i = 0; i < r.kWords; ++i)
                r.w[i] = Pack<T>::pack(v + i * Pack<T>::kPerWord);
        }
#pragma unroll
        for (int i = 0; i < r.kWords; ++i) w[i] = r.w[i];
    }
    __device__ __forceinline__ void load(const mt_attention_call_t &c,
                                         const Cut &cut, int dtype,
                                         const Tile &a, int hs, int ks,
                                         int warps) {
        const int from = begin_of(c, a.s) + a.t * cut.per;
        const int rows = min(cut.per, a.tiles.rows - a.t * cut.per);
        const bool whole = cut.whole & 1;
#pragma unroll
        for (int col = 0; col < C; ++col) {
            const Place at =
                place_of<C>(cut, from, rows, a.head + hs, a.part, col);
            const bool on = at.used && (col & (warps - 1)) == ks;
            const int64_t q =
                (int64_t)at.row * c.q_row + (int64_t)at.head * c.q_head;
#pragma unroll
            for (int i = 0; i < kEach; ++i) {
                const int d = 4 * ((threadIdx.x & 31) + 32 * i);
#pragma unroll
                for (int e = 0; e < kWords; ++e) x[col][i][e] = 0;
                if (!on || d >= H::DIM) continue;
                if constexpr (PARTS == 1)
                    four<__nv_bfloat16>(c.q, q + d, whole, x[col][i]);
                else if (dtype == DT_F16)
                    four<__half>(c.q, q + d, whole, x[col][i]);
                else
                    four<float>(c.q, q + d, whole, x[col][i]);
            }
        }
    }
    __device__ __forceinline__ void widen(const unsigned *w, int dtype,
                                          float *v) const {
        if constexpr (PARTS == 1) {
            Pack<__nv_bfloat16>::unpack(w[0], v);
            Pack<__nv_bfloat16>::unpack(w[1], v + 2);
        } else if (dtype == DT_F16) {
            Pack<__half>::unpack(w[0], v);
            Pack<__half>::unpack(w[1], v + 2);
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e) v[e] = __uint_as_float(w[e]);
        }
    }
    // Fragments, and the columns' factors, into shared memory; columns from
    // `columns` on stand for nothing.
    __device__ __forceinline__ void put(const mt_attention_call_t &c,
                                        Shared<H, PARTS, NT> &sh, int dtype,
                                        int columns, int hs, int ks,
                                        int warps) {
        const int lane = threadIdx.x & 31;
        int place[kEach];  // of the lane's fours in a column's fragments
#pragma unroll
        for (int i = 0; i < kEach; ++i) {
            const int d = min(4 * (lane + 32 * i), H::DIM - 4);
            const int r = d % H::GROUP;
            const Block block = H::block(r / 16);
            const int in = r - block.base, wide = block.size / 4;
            const int step = d / H::GROUP * H::PER + block.base / 16 +
                             in % wide / 4;
            place[i] = step * 32 + in / wide;
        }
#pragma unroll
        for (int col = 0; col < C; ++col) {
            if ((col & (warps - 1)) != ks) continue;
            float v[kEach][4];
            float largest = 0.f;
            if (col < columns) {
#pragma unroll
                for (int i = 0; i < kEach; ++i) {
                    widen(x[col][i], dtype, v[i]);
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        largest = nanmax(largest, fabsf(v[i][e]));
                }
                largest = warp_nanmax(largest);
            }
            const unsigned e = max(__float_as_uint(largest) >> 23, 15u);
            const bool bad = !(largest < INFINITY);
            const bool none = bad || col >= columns;
            const float up = __uint_as_float((268u - e) << 23);
#pragma unroll
            for (int i = 0; i < kEach; ++i) {
                if (4 * (lane + 32 * i) >= H::DIM) continue;
                uint2 hi = make_uint2(0, 0), lo = hi;
                if (!none) {
                    const float a = v[i][0] * up, b = v[i][1] * up;
                    const float c_ = v[i][2] * up, d = v[i][3] * up;
                    hi = make_uint2(half_pair(a, b), half_pair(c_, d));
                    if constexpr (PARTS == 2) {
                        const float2 p = from_half_pair(hi.x);
                        const float2 q = from_half_pair(hi.y);
                        lo = make_uint2(half_pair(a - p.x, b - p.y),
                                        half_pair(c_ - q.x, d - q.y));
                    }
                }
                sh.q[hs][col / 8][0][0][place[i] + col % 8 * 4] = hi;
                if constexpr (PARTS == 2)
                    sh.q[hs][col / 8][1][0][place[i] + col % 8 * 4] = lo;
            }
            if (lane == 0)
                sh.f[hs][col] =
                    bad ? NAN
                        : c.scale * kLog2e * __uint_as_float((e - 14u) << 23);
        }
    }
};

// What the columns of a tile see, into shared memory.
template <class H, int PARTS, int NT>
__device__ __forceinline__ void tile_bounds(const mt_attention_call_t &c,
                                            const Cut &cut, const Tile &a,
                                            int hs, int ks,
                                            Shared<H, PARTS, NT> &sh) {
    constexpr int C = 8 * NT;
    const int col = threadIdx.x & 31;
    const int from = begin_of(c, a.s);
    const Place at = place_of<C>(cut, from + a.t * cut.per,
                                 min(cut.per, a.tiles.rows - a.t * cut.per),
                                 a.head + hs, a.part, col);
    const bool used = col < C && at.used;
    if (c.slopes != nullptr && ks == 0 && col < C)
        sh.slope[hs][col] = used ? c.slopes[at.head] * kLog2e : 0.f;
    if (threadIdx.x >= 32) return;
    Column k = {INT32_MIN, INT32_MAX, 0, 0};
    if (used) {
        const int64_t n = (int64_t)begin_of(c, a.s + 1) - from;
        const int64_t start = c.starts[a.s], p = start + (at.row - from);
        int64_t lo, hi;
        row_sees(c, at.row, p, start + n, lo, hi);
        k.lo = (int32_t)min(lo, (int64_t)INT32_MAX);
        k.hi = (int32_t)max(min(hi, (int64_t)INT32_MAX), (int64_t)-1);
        k.p = (int32_t)min(p, (int64_t)INT32_MAX);
    }
    if (col < C) sh.column[col] = k;
    const bool some = used && k.lo <= k.hi;
    const int lo_any = __reduce_min_sync(kFull, some ? k.lo : INT32_MAX);
    const int hi_any = __reduce_max_sync(kFull, some ? k.hi : -1);
    const int lo_all = __reduce_max_sync(kFull, k.lo);
    const int hi_all = __reduce_min_sync(kFull, k.hi);
    if (col == 0) {
        sh.lo_any = lo_any;
        sh.hi_any = hi_any;
        sh.lo_all = lo_all;
        sh.hi_all = hi_all;
    }
}

// A key's page, asked for a chunk before its slot is worked out (arithmetic on
// a loaded value would hold the warp up where it stands).
struct Page {
    int id, at;  // number (-1: no column sees the key), place in it
};
__device__ __forceinline__ Page page_of(const mt_attention_call_t &c,
                                        const int32_t *pages, int64_t j,
                                        int lo, int hi) {
    Page p = {-1, 0};
    if (j >= lo && j <= hi) {
        const unsigned page = (unsigned)j / (unsigned)c.page_size;
        p.at = (int)((unsigned)j - page * (unsigned)c.page_size);
        p.id = pages[page];
    }
    return p;
}
// Its slot, or -1 where it has none.
__device__ __forceinline__ int slot_in(const mt_attention_call_t &c, Page p) {
    const int64_t slot = (int64_t)p.id * c.page_size + p.at;
    return p.id >= 0 && slot < c.slots ? (int)slot : -1;
}

// The units [u0, u1) of a tile: its queries, and each warp's share of them.
template <class H, bool INT8, int PARTS, int NT>
__device__ __forceinline__ void tile_run(const mt_attention_call_t &c,
                                         const Cut &cut, int dtype,
                                         const Tile &a, int64_t u0, int64_t u1,
                                         Shared<H, PARTS, NT> &sh,
                                         Warp<H, INT8, PARTS, NT> &w) {
    constexpr int KT = H::KEYS / 16;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int warps = kWarps / cut.heads;  // of a key head
    const int hs = warp / warps, ks = warp & (warps - 1);
    w.hs = hs;
    // The queries are asked for first and needed last: the first keys' slots
    // and codes are on their way meanwhile.
    Queries<H, PARTS, NT> queries;
    queries.load(c, cut, dtype, a, hs, ks, warps);
    tile_bounds(c, cut, a, hs, ks, sh);
    __syncthreads();
    const int lo = sh.lo_any, hi = sh.hi_any;
    const int32_t *pages = c.table + a.s * c.table_stride;
    // chunks
    int64_t u = max(u0 * warps, (int64_t)(lo / H::KEYS));
    const int64_t end =
        lo > hi ? 0 : min(u1 * warps, (int64_t)(hi / H::KEYS) + 1);
    u += (ks - u) & (warps - 1);
    const auto page_at = [&](int64_t v) {
        return v < end && lane < H::KEYS
                   ? page_of(c, pages, v * H::KEYS + lane, lo, hi)
                   : Page{-1, 0};
    };
    const int head = a.head + hs;
    Cache m;
    m.row = (unsigned)(c.k_heads * H::DIM);
    m.scales = (unsigned)(c.k_heads * H::GROUPS);
    m.k = static_cast<const uint8_t *>(c.k_codes) + head * H::DIM;
    m.v = static_cast<const uint8_t *>(c.v_codes) + head * H::DIM;
    m.ks = c.k_scales + head * H::GROUPS;
    m.vs = c.v_scales + head * H::GROUPS;
    auto &codes = sh.own[warp].codes;
    auto &scales = sh.scales[warp];
    const Page first = page_at(u);
    Page next = page_at(u + warps);
    int slot = slot_in(c, first), stage = 0;
    if (u < end) w.load(m, slot, codes[0], scales[0]);
    asm volatile("cp.async.commit_group;" ::: "memory");
    queries.put(c, sh, dtype,
                columns_of<8 * NT>(
                    cut, min(cut.per, a.tiles.rows - a.t * cut.per), a.part),
                hs, ks, warps);
    __syncthreads();
    w.begin();
#pragma unroll 1
    for (; u < end; u += warps) {
        const unsigned there = __ballot_sync(kFull, slot >= 0);
        slot = slot_in(c, next);
        next = page_at(u + 2 * warps);
        if (u + warps < end)
            w.load(m, slot, codes[stage ^ 1], scales[stage ^ 1]);
        asm volatile("cp.async.commit_group;" ::: "memory");
        asm volatile("cp.async.wait_group 1;" ::: "memory");
        __syncwarp();
        if (there != 0) {
            float z[NT][KT][4];
            unsigned hidden;
            w.scores(sh, codes[stage], scales[stage], z);
            const bool masked =
                w.bend(c, sh, (int)(u * H::KEYS), there, hidden, z);
            w.weigh(z);
            w.add(z, hidden, masked, codes[stage], scales[stage]);
        }
        __syncwarp();  // the next round's copies go where this one read
        stage ^= 1;
    }
    asm volatile("cp.async.wait_group 0;" ::: "memory");
    __syncwarp();  // the warp's sums take the chunks' place
}

// Four values of a row of the output.
__device__ __forceinline__ void store4(int dtype, bool whole, void *p,
                                       int64_t i, const float *v) {
    if (!whole) {
#pragma unroll
        for (int e = 0; e < 4; ++e) store_as(dtype, p, i + e, v[e]);
    } else if (dtype == DT_BF16) {
        st_vec<__nv_bfloat16, 4>(static_cast<__nv_bfloat16 *>(p) + i, v);
    } else if (dtype == DT_F16) {
        st_vec<__half, 4>(static_cast<__half *>(p) + i, v);
    } else {
        st_vec<float, 4>(static_cast<float *>(p) + i, v);
    }
}
// A column's sums about `top` (-infinity: nothing seen), out.
__device__ __forceinline__ void finish(const mt_attention_call_t &c,
                                       const Cut &cut, int dtype,
                                       const Place &at, int d, float top,
                                       float sum, float *o) {
#pragma unroll
    for (int e = 0; e < 4; ++e) o[e] = top == -INFINITY ? 0.f : o[e] / sum;
    store4(dtype, (cut.whole & 2) != 0, c.out,
           (int64_t)at.row * c.out_row + (int64_t)at.head * c.out_head + d, o);
    if (c.lse != nullptr && d == 0)
        c.lse[(int64_t)at.row * c.q_heads + at.head] =
            top == -INFINITY ? top : (top + log2f(sum)) * 0.6931471805599453f;
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
                sh.m[warp][8 * n + 2 * q + h] = w.ref[n][h];
                sh.l[warp][8 * n + 2 * q + h] = sum;
            }
        }
#pragma unroll
        for (int i = 0; i < H::STEPS; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int gr = i / H::PER;
                const Block block = H::block(i % H::PER);
                const int d = gr * H::GROUP + block.base +
                              g * (block.size / 8) +
                              2 * (i % H::PER - block.base / 16) + (e >> 1);
                sh.own[warp].o[8 * n + 2 * q + (e & 1)][d] =
                    w.o[n][i][e] * w.down(w.exponent(n, e & 1, gr));
            }
    }
    __syncthreads();
    const int from = begin_of(c, a.s) + a.t * cut.per;
    const int rows = min(cut.per, a.tiles.rows - a.t * cut.per);
    const int columns = columns_of<C>(cut, rows, a.part);
    const int warps = kWarps / cut.heads;
#pragma unroll 1
    for (int hs = 0; hs < cut.heads; ++hs)
#pragma unroll 1
        for (int i = 4 * threadIdx.x; i < columns * H::DIM;
             i += 128 * kWarps) {
            const int col = i / H::DIM, d = i % H::DIM, w0 = hs * warps;
            float top = sh.m[w0][col];
            for (int x = 1; x < warps; ++x)
                top = nanmax(top, sh.m[w0 + x][col]);
            const float ref = top == -INFINITY ? 0.f : top;
            float sum = 0.f, o[4] = {0.f, 0.f, 0.f, 0.f};
            for (int x = 0; x < warps; ++x) {
                const float f = pow2(sh.m[w0 + x][col] - ref);
                const float4 v = *reinterpret_cast<const float4 *>(
                    &sh.own[w0 + x].o[col][d]);
                sum = fmaf(sh.l[w0 + x][col], f, sum);
                o[0] = fmaf(v.x, f, o[0]);
                o[1] = fmaf(v.y, f, o[1]);
                o[2] = fmaf(v.z, f, o[2]);
                o[3] = fmaf(v.w, f, o[3]);
            }
            if (whole) {
                finish(c, cut, PARTS == 1 ? (int)DT_BF16 : dtype,
                       place_of<C>(cut, from, rows, a.head + hs, a.part, col),
                       d, top, sum, o);
            } else {
                const int at = hs * C + col;
                *reinterpret_cast<float4 *>(sums + 2 * kWarps * C +
                                            at * H::DIM + d) =
                    make_float4(o[0], o[1], o[2], o[3]);
                if (d == 0) {
                    sums[at] = top;
                    sums[kWarps * C + at] = sum;
                }
            }
        }
    __syncthreads();  // shared memory is the next tile's
}

// The least units that a CTA takes where there are few: a tile's own, and one.
constexpr int kLeastUnits = (int)kExtra + 1;

// Deals the call's units out and goes through the CTA's run of them:
// body(tile, u0, u1, whole, place) for the units [u0, u1) of a tile, whole or
// not, whose partial sums belong in the CTA's place 0 or 1.
template <int WARPS = kWarps, class Body>
__device__ __forceinline__ void deal_units(const mt_attention_call_t &c,
                                           const Cut &cut, const Share &share,
                                           Deal &sh, Body body) {
    constexpr int T = 32 * WARPS;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    int cut_here = 0;
    // Units of the sequences of this thread, and where they begin.
    const int each = (c.sequences + T - 1) / T;
    const int s0 = min(tid * each, c.sequences);
    const int s1 = min(s0 + each, c.sequences);
    const int64_t wide = cut.wide;
    const auto units_of = [&](int s) {
        const Tiles t = tiles_of(c, cut, s);
        return wide * t.before(t.count);
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
    for (int x = 0; x < WARPS; ++x) {
        if (x < warp) first += sh.scan[x];
        total += sh.scan[x];
    }
    const int64_t ctas = min((int64_t)gridDim.x,
                             (total + kLeastUnits - 1) / kLeastUnits);
    int64_t at = 0, end = 0;
    if (blockIdx.x < ctas) {
        at = quotient(total * blockIdx.x, ctas);
        end = quotient(total * (blockIdx.x + 1), ctas);
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
        // before(lo) <= off < before(hi): every thread looks at one place of
        // the range, until it has one tile.
        int lo = 0, hi = a.tiles.count;
        int64_t units_before = 0;
        while (hi - lo > 1) {
            const int step = (hi - lo + T - 1) / T;
            const int mid = min(lo + (tid + 1) * step, hi);
            const int64_t here = mid < hi ? wide * a.tiles.before(mid) : 0;
            const int fewer = __syncthreads_count(mid < hi && here <= off);
            if (fewer > 0) {
                if (tid == fewer - 1) sh.at = here;
                __syncthreads();
                units_before = sh.at;
            }
            lo += fewer * step;
            hi = min(lo + step, hi);
        }
        a.t = lo;
        off -= units_before;
        int64_t base = a.tiles.first(lo);
        int64_t units = a.tiles.last(lo) - base + 1 + kExtra;
        int index = (int)quotient(off, units);
        off -= index * units;
        while (at < end) {
            const int64_t n = min(units - off, end - at);
            a.head = index / cut.parts;
            a.part = index - a.head * cut.parts;
            a.head *= cut.heads;
            const bool whole = n == units;
            if (!whole && off == 0) {
                const int64_t x = at + units;
                cut_here = 1;
                if (tid == 0)
                    share.records[blockIdx.x] = {
                        (int)quotient(x * ctas - 1, total),
                        begin_of(c, a.s) + a.t * cut.per,
                        min(cut.per, a.tiles.rows - a.t * cut.per), a.head,
                        a.part};
            }
            body(a, base + max(off - kExtra, (int64_t)0),
                 base + max(off + n - kExtra, (int64_t)0), whole,
                 off == 0 ? 1 : 0);
            at += n;
            off = 0;
            if (at < end && ++index == wide) {
                index = 0;
                if (++a.t == a.tiles.count) {
                    a.t = 0;
                    do a.tiles = tiles_of(c, cut, ++a.s);
                    while (a.tiles.rows == 0);
                }
                base = a.tiles.first(a.t);
                units = a.tiles.last(a.t) - base + 1 + kExtra;
            }
        }
    }
    // Not before: the next kernel's CTAs would take the place of this one's
    // (64 sequences to 16384 keys with three CTAs per SM: 331 us for 251).
    grid_launch_dependents();
    if (tid == 0) share.cut[blockIdx.x] = cut_here;
}

template <class H, bool INT8, int PARTS, int NT>
__global__ void __launch_bounds__(32 * kWarps,
                                  attention_ctas(H::DIM, H::GROUPS, PARTS, NT))
    attention_mma_kernel(const mt_attention_call_t c, const Cut cut,
                         const Share share, int dtype) {
    extern __shared__ __align__(16) uint8_t shared[];
    Shared<H, PARTS, NT> &sh =
        *reinterpret_cast<Shared<H, PARTS, NT> *>(shared);
    grid_wait_prerequisites();
    Warp<H, INT8, PARTS, NT> w;
    deal_units(c, cut, share, sh.deal,
               [&](const Tile &a, int64_t u0, int64_t u1, bool whole,
                   int place) {
                   tile_run<H, INT8, PARTS, NT>(c, cut, dtype, a, u0, u1, sh,
                                                w);
                   tile_end<H, INT8, PARTS, NT>(
                       c, cut, dtype, a, whole,
                       share.sums + (2 * (int64_t)blockIdx.x + place) *
                                        place_floats(kWarps * 8 * NT, H::DIM),
                       sh, w);
               });
}

// Joins the parts of cut tiles, in the order of the CTAs that left them: a
// column to a warp, four values to a lane, a part's factor in each lane first;
// where there are few columns, the warps of a CTA share the parts of one.
constexpr int kJoin = 256, kJoinWarps = kJoin / 32;
// CTAs that join for each that left parts, behind tiles of 64 and 128 columns:
// there a warp has many columns one after the other, each a chain of reads (two
// prompts of 512 rows 186 us with one, 175 with two, 173 with eight).
constexpr int kJoinCtas = 2;
template <int DIM, int C, int SLOTS>
__global__ void __launch_bounds__(kJoin)
    attention_join_kernel(const mt_attention_call_t c, const Cut cut,
                          const Share share, int dtype, int records) {
    constexpr int kQuads = (DIM / 4 + 31) / 32;  // of a lane
    __shared__ int16_t cuts[kAttentionMaxCtas];
    __shared__ int counts[kJoinWarps];
    __shared__ float tops[kJoinWarps], totals[kJoinWarps];
    __shared__ float4 part_o[kJoinWarps][DIM / 4];
    grid_wait_prerequisites();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int ctas = (int)gridDim.x;
    // The cut tiles, by the CTA in which they begin: a warp looks at a run of
    // them, four for each lane at a time.
    constexpr int kLooks = 4;
    int n = 0;
    for (int b0 = 0; b0 < records; b0 += kLooks * kJoin) {
        bool on[kLooks];
        unsigned mask[kLooks];
        int found = 0;
#pragma unroll
        for (int y = 0; y < kLooks; ++y) {
            const int b = b0 + (warp * kLooks + y) * 32 + lane;
            on[y] = b < records && share.cut[b] != 0;
        }
#pragma unroll
        for (int y = 0; y < kLooks; ++y) {
            mask[y] = __ballot_sync(kFull, on[y]);
            found += __popc(mask[y]);
        }
        if (lane == 0) counts[warp] = found;
        __syncthreads();
        int before = n;
        for (int x = 0; x < kJoinWarps; ++x) {
            if (x < warp) before += counts[x];
            n += counts[x];
        }
#pragma unroll
        for (int y = 0; y < kLooks; ++y) {
            if (on[y])
                cuts[before + __popc(mask[y] & ((1u << lane) - 1u))] =
                    (int16_t)(b0 + (warp * kLooks + y) * 32 + lane);
            before += __popc(mask[y]);
        }
        __syncthreads();
    }
    // columns that a tile has at most
    const int most = cut.times <= C ? cut.per * cut.times : C;
    constexpr int64_t kPlace = place_floats(SLOTS * C, DIM);
    const int columns = n * cut.heads * most;
    const bool few = columns <= ctas;
    const int share_of = few ? kJoinWarps : 1;
    const int mine = few ? warp : 0;  // which of the parts
    for (int p = few ? (int)blockIdx.x
                     : (int)blockIdx.x * kJoinWarps + warp;
         p < columns; p += ctas * (few ? 1 : kJoinWarps)) {
        const int tile = p / (cut.heads * most), in = p - tile * cut.heads * most;
        const int b = cuts[tile], hs = in / most, col = in - hs * most;
        const Record r = share.records[b];
        const Place at =
            place_of<C>(cut, r.row, r.rows, r.head + hs, r.part, col);
        if (!at.used) continue;  // the same for all that share the column
        const int parts = r.last - b + 1, i = hs * C + col;
        // part 0 is in its CTA's second place, the others in the first places
        // of the CTAs after it
        const auto part = [&](int x) {
            return share.sums + (2 * (int64_t)(b + x) + (x == 0 ? 1 : 0)) *
                                    kPlace;
        };
        float top = -INFINITY;
        for (int x = mine + share_of * lane; x < parts; x += share_of * 32)
            top = nanmax(top, part(x)[i]);
        top = warp_nanmax(top);
        const float ref = top == -INFINITY ? 0.f : top;
        float sum = 0.f;
        float4 o[kQuads] = {};
        for (int x0 = mine; x0 < parts; x0 += share_of * 32) {
            const int x = x0 + share_of * lane;
            const bool on = x < parts;
            const float f = on ? pow2(part(x)[i] - ref) : 0.f;
            if (on) sum = fmaf(part(x)[SLOTS * C + i], f, sum);
            const int many = min(32, (parts - x0 + share_of - 1) / share_of);
#pragma unroll 8
            for (int y = 0; y < many; ++y) {
                const float g = __shfl_sync(kFull, f, y);
                const float *from = part(x0 + share_of * y) + 2 * SLOTS * C +
                                    i * DIM;
#pragma unroll
                for (int k = 0; k < kQuads; ++k) {
                    const int at4 = lane + 32 * k;
                    if (at4 >= DIM / 4) continue;
                    const float4 v =
                        *reinterpret_cast<const float4 *>(from + 4 * at4);
                    o[k].x = fmaf(v.x, g, o[k].x);
                    o[k].y = fmaf(v.y, g, o[k].y);
                    o[k].z = fmaf(v.z, g, o[k].z);
                    o[k].w = fmaf(v.w, g, o[k].w);
                }
            }
        }
#pragma unroll
        for (int off = 16; off > 0; off >>= 1)
            sum += __shfl_xor_sync(kFull, sum, off);
        if (few) {
            if (lane == 0) {
                tops[warp] = top;
                totals[warp] = sum;
            }
#pragma unroll
            for (int k = 0; k < kQuads; ++k)
                if (lane + 32 * k < DIM / 4) part_o[warp][lane + 32 * k] = o[k];
            __syncthreads();
            if (warp == 0) {
                for (int x = 0; x < kJoinWarps; ++x)
                    top = nanmax(top, tops[x]);
                const float about = top == -INFINITY ? 0.f : top;
                sum = 0.f;
#pragma unroll
                for (int k = 0; k < kQuads; ++k)
                    o[k] = make_float4(0.f, 0.f, 0.f, 0.f);
                for (int x = 0; x < kJoinWarps; ++x) {
                    const float g = pow2(tops[x] - about);
                    sum = fmaf(totals[x], g, sum);
#pragma unroll
                    for (int k = 0; k < kQuads; ++k) {
                        if (lane + 32 * k >= DIM / 4) continue;
                        const float4 v = part_o[x][lane + 32 * k];
                        o[k].x = fmaf(v.x, g, o[k].x);
                        o[k].y = fmaf(v.y, g, o[k].y);
                        o[k].z = fmaf(v.z, g, o[k].z);
                        o[k].w = fmaf(v.w, g, o[k].w);
                    }
                }
            }
        }
        if (!few || warp == 0) {
#pragma unroll
            for (int k = 0; k < kQuads; ++k) {
                const int at4 = lane + 32 * k;
                if (at4 < DIM / 4)
                    finish(c, cut, dtype, at, 4 * at4, top, sum, &o[k].x);
            }
        }
        if (few) __syncthreads();  // the next column's
    }
    grid_launch_dependents();
}

template <class H, bool INT8, int PARTS, int NT>
cudaError_t launch_attention_as(const AttentionPlan &p,
                                const mt_attention_call_t &c, int dtype,
                                void *workspace, cudaStream_t s) {
    using Sh = Shared<H, PARTS, NT>;
    constexpr int kCtas = attention_ctas(H::DIM, H::GROUPS, PARTS, NT);
    constexpr size_t kBytes = sizeof(Sh);
    static_assert((kBytes + 1024) * kCtas <= 228 * 1024,
                  "the CTAs that share an SM fit its shared memory");
    const int warps = kWarps / p.heads;
    const Cut cut = {p.times, p.per, p.parts, p.heads,
                     (H::KEYS == 32 ? 5 : 4) + (warps == 4   ? 2
                                                : warps == 2 ? 1 : 0),
                     c.k_heads / p.heads * p.parts, p.whole};
    Share share;
    share.sums = static_cast<float *>(workspace);
    share.records = reinterpret_cast<Record *>(
        share.sums +
        2 * (int64_t)p.ctas * place_floats(kWarps * 8 * NT, H::DIM));
    share.cut = reinterpret_cast<int32_t *>(share.records + p.ctas);
    static_assert(sizeof(Record) + sizeof(int32_t) == kAttentionRecord, "");
    cudaError_t e = cudaSuccess;
    const auto kernel = attention_mma_kernel<H, INT8, PARTS, NT>;
    if (kBytes > 40 * 1024)
        e = allow_max_smem(reinterpret_cast<const void *>(kernel));
    if (e == cudaSuccess)
        e = launch_dependent(kernel, p.ctas, 32 * kWarps, kBytes, s, c, cut,
                             share, dtype);
    if (e != cudaSuccess) return e;
    return launch_dependent(attention_join_kernel<H::DIM, 8 * NT, kWarps>,
                            p.ctas, kJoin, 0, s, c, cut, share, dtype, p.ctas);
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

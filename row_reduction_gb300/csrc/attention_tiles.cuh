// attention_tiles.cuh -- attention over the quantised cache for prompts, BF16, on
// tensor memory (one translation unit per code format).
//
// A tile has 128 columns (rows of a sequence times the query heads of a key
// head) and goes through chunks of 64 keys.  Four warps have a column to a thread
// and to a lane of tensor memory: they take a chunk's scores from there, make
// weights of them and put these, as FP16, in the scores' place.  Nothing is
// exchanged among lanes for that.  Four other warps copy codes, widen them to
// FP16 in shared memory (swizzled by 128 bytes), 16 keys each, and issue the
// products: S = Q K^T, 128 x 64, a chunk ahead, and O += P V, 128 x dim, with P
// out of tensor memory.  Two CTAs to an SM share its 512 columns.
//
// Scores, references, scales and roundings are as in attention_mma.cuh, for one
// group a head and BF16; sums stay in tensor memory, and are brought out to be
// scaled only where a reference or a power of two has moved.  Units, cut tiles
// and their joining are the same as there.
//
// Bound.  Two sequences of up to 512 rows at 4096 keys, 32 + 8 heads of 128,
// capped: 178 us, 322 TFLOP/s, 308 on tiles of 64 columns with mma.sync (uncapped
// and causal 155 for 283); 2 x 2048 rows at 8192 keys 830 us, 425 TFLOP/s.  What
// is done for a score sets it, not the products (16% of the tensor pipe; heads of
// 64, half the products, 148 us): issue slots are 45% busy at 16 warps per SM, and
// weights wait for scales from shared memory, 52% of whose throughput operands,
// codes and scales share, and for each other's results.  Some 220 bytes of a
// thread's 128 registers spill.  All eight warps on weights, halves of a column
// each, took 239 us, all four on everything 214 (175 at the time).
//
// Waits have a limit; a CTA whose wait ran out gives NaN.  No barrier gets two
// phases ahead of who waits for it: weights of a chunk arrive only after the sums
// of the chunk before are through.
#pragma once

#include "attention_mma.cuh"

namespace mt {
namespace {

constexpr int kTileColumns = 128, kTileKeys = 64;
constexpr int kTensorColumns = 256;  // scores twice, sums

// ---- instructions ----------------------------------------------------------------
// An operand in shared memory, rows of 128 bytes in blocks of 8, swizzled; far:
// bytes between blocks of 64 values of an operand whose rows are keys' (K x N).
__device__ __forceinline__ uint64_t operand(unsigned at, unsigned far) {
    return (uint64_t)(at >> 4 & 0x3fffu) | (uint64_t)(far >> 4) << 16 |
           (uint64_t)(1024 >> 4) << 32 | 1ull << 46 | 2ull << 61;
}
// FP16 operands, FP32 sums, 128 rows; across: B's rows are keys'.
__host__ __device__ constexpr unsigned product_of(int n, bool across) {
    return 1u << 4 | (across ? 1u << 16 : 0u) | (unsigned)(n >> 3) << 17 |
           (128u >> 4) << 24;
}
__device__ __forceinline__ void tensor_product(unsigned d, uint64_t a,
                                               uint64_t b, unsigned kind,
                                               bool add) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(
            d),
        "l"(a), "l"(b), "r"(kind), "r"(add ? 1 : 0)
        : "memory");
}
// The same with the first operand in tensor memory, two values to a column.
__device__ __forceinline__ void tensor_product(unsigned d, unsigned a,
                                               uint64_t b, unsigned kind,
                                               bool add) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::
            "r"(d), "r"(a), "l"(b), "r"(kind), "r"(add ? 1 : 0)
        : "memory");
}
// The products so far arrive at `bar`.
__device__ __forceinline__ void tensor_arrive(uint64_t *bar) {
    asm volatile(
        "tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 "
        "[%0];" ::"r"(smem_addr(bar))
        : "memory");
}
__device__ __forceinline__ void tensor_before() {
    asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void tensor_after() {
    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
}
// The 32 columns from `at` on of the thread's own lane.  Loads and stores are
// the warp's: its lanes, which may have gone different ways, come together here.
__device__ __forceinline__ void tensor_load(unsigned (&r)[32], unsigned at) {
    __syncwarp();
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {"
        "%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
        "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31"
        "}, [%32];\n\ttcgen05.wait::ld.sync.aligned;"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]),
          "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]),
          "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
          "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]),
          "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]),
          "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]),
          "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]),
          "=r"(r[30]), "=r"(r[31])
        : "r"(at)
        : "memory");
}
__device__ __forceinline__ void tensor_store(unsigned at,
                                             const unsigned (&r)[32]) {
    __syncwarp();
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {"
        "%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, "
        "%17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32"
        "};\n\ttcgen05.wait::st.sync.aligned;" ::"r"(at),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]),
        "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
        "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]),
        "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]),
        "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]),
        "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]), "r"(r[29]),
        "r"(r[30]), "r"(r[31])
        : "memory");
}

template <int DIM>
struct TileShared {
    static constexpr int BLOCKS = DIM / 64;    // of 64 values, 128 bytes
    uint4 q[BLOCKS][kTileColumns * 8];
    uint4 k[BLOCKS][kTileKeys * 8], v[BLOCKS][kTileKeys * 8];
    uint8_t k_codes[kTileKeys * DIM], v_codes[kTileKeys * DIM];
    float ks[4][kTileKeys], vs[4][kTileKeys];  // of four chunks in turn
    alignas(16) unsigned there[4][kWarps];                 // keys with a slot, 16 to a warp
    int32_t lo_any[kWarps], hi_any[kWarps], lo_all[kWarps], hi_all[kWarps];
    Deal deal;
    uint64_t score_done[2], weights_there, value_done;
    unsigned tensor;
    int failed;                                // a wait ran out
    static_assert(DIM == 64 || DIM == 128, "whole blocks, 128 columns of sums");
};

// CAP: whether scores are capped (two kernels: what the one needs more takes
// the other's registers).
template <int DIM, bool INT8, bool CAP>
struct TileRun {
    static constexpr int PIECES = DIM / 16;    // of 16 codes, of a key
    static constexpr int OWN = kTileKeys / kWarps;
    using Sh = TileShared<DIM>;
    Sh &sh;
    unsigned scores_at, sums_at;               // in tensor memory, own lanes
    unsigned score_phase = 0, value_phase = 0, weights_phase = 0;
    // the thread's column
    float ref, l, f, slope;
    unsigned most;                             // exponent, as in Warp
    int lo, hi, p;
    bool any;                                  // sums there

    __device__ __forceinline__ explicit TileRun(Sh &s) : sh(s) {}
    static __device__ __forceinline__ float up(unsigned e) {
        return __uint_as_float((265u - e) << 23);
    }
    static __device__ __forceinline__ float down(unsigned e) {
        return __uint_as_float((e - 11u) << 23);
    }
    // bit: of `phase`, the barrier's.
    __device__ __forceinline__ void wait(uint64_t *bar, unsigned &phase,
                                         int bit = 0) {
        if (!mbar_try_wait(bar, phase >> bit & 1u) &&
            !*(volatile int *)&sh.failed &&
            !mbar_wait_bounded(bar, phase >> bit & 1u))
            *(volatile int *)&sh.failed = 1;
        phase ^= 1u << bit;
        tensor_after();
    }
    __device__ __forceinline__ void wait_all(uint64_t *bar, unsigned &phase,
                                             int bit = 0) {
        wait(bar, phase, bit);
        __syncwarp();  // what follows is the warp's
    }
    // By one lane, after all of the warp's.
    static __device__ __forceinline__ void arrive(uint64_t *bar) {
        __syncwarp();
        if ((threadIdx.x & 31) == 0)
            asm volatile("mbarrier.arrive.release.cta.shared::cta.b64 _, [%0];" ::"r"(
                             smem_addr(bar))
                         : "memory");
    }
    static __device__ __forceinline__ void four(const mt_attention_call_t &c,
                                                bool whole, int64_t at,
                                                float *v) {
        const __nv_bfloat16 *q = static_cast<const __nv_bfloat16 *>(c.q) + at;
        if (whole) {
            ld_vec<__nv_bfloat16, 4>(q, v);
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e) v[e] = to_f(q[e]);
        }
    }
    // The column's query into shared memory, its factor and bounds.
    __device__ __forceinline__ void begin(const mt_attention_call_t &c,
                                          const Cut &cut, const Tile &a) {
        const int col = threadIdx.x, lane = col & 31, warp = col >> 5;
        const int from = begin_of(c, a.s);
        const Place at = place_of<kTileColumns>(
            cut, from + a.t * cut.per,
            min(cut.per, a.tiles.rows - a.t * cut.per), a.head, a.part, col);
        const bool whole = cut.whole & 1;
        const int64_t x0 =
            (int64_t)at.row * c.q_row + (int64_t)at.head * c.q_head;
        float largest = 0.f;
        if (at.used) {
#pragma unroll 8
            for (int i = 0; i < DIM / 4; ++i) {
                float v[4];
                four(c, whole, x0 + 4 * i, v);
                largest = nanmax3(largest, fabsf(v[0]), fabsf(v[1]));
                largest = nanmax3(largest, fabsf(v[2]), fabsf(v[3]));
            }
        }
        const unsigned e = max(__float_as_uint(largest) >> 23, 15u);
        const bool bad = !(largest < INFINITY);
        const float by = __uint_as_float((268u - e) << 23);
#pragma unroll 4
        for (int i = 0; i < DIM / 8; ++i) {
            uint4 w = make_uint4(0, 0, 0, 0);
            if (at.used && !bad) {
                float v[8];
                four(c, whole, x0 + 8 * i, v);
                four(c, whole, x0 + 8 * i + 4, v + 4);
                w = make_uint4(half_pair(v[0] * by, v[1] * by),
                               half_pair(v[2] * by, v[3] * by),
                               half_pair(v[4] * by, v[5] * by),
                               half_pair(v[6] * by, v[7] * by));
            }
            sh.q[i / 8][col * 8 + ((i & 7) ^ (col & 7))] = w;
        }
        f = bad ? NAN
                : c.scale * kLog2e * __uint_as_float((e - 14u) << 23);
        slope = 0.f;
        lo = INT32_MIN;
        hi = INT32_MAX;
        p = 0;
        if (at.used) {
            const int64_t n = (int64_t)begin_of(c, a.s + 1) - from;
            const int64_t start = c.starts[a.s], pos = start + (at.row - from);
            int64_t b0, b1;
            row_sees(c, at.row, pos, start + n, b0, b1);
            if (c.slopes != nullptr) slope = c.slopes[at.head] * kLog2e;
            lo = (int)min(b0, (int64_t)INT32_MAX);
            hi = (int)max(min(b1, (int64_t)INT32_MAX), (int64_t)-1);
            p = (int)min(pos, (int64_t)INT32_MAX);
        }
        const bool some = at.used && lo <= hi;
        const int v[4] = {__reduce_min_sync(kFull, some ? lo : INT32_MAX),
                          __reduce_max_sync(kFull, some ? hi : -1),
                          __reduce_max_sync(kFull, lo),
                          __reduce_min_sync(kFull, hi)};
        if (lane == 0) {
            sh.lo_any[warp] = v[0];
            sh.hi_any[warp] = v[1];
            sh.lo_all[warp] = v[2];
            sh.hi_all[warp] = v[3];
        }
        ref = -INFINITY;
        l = 0.f;
        most = 12u;
    }
    // The warp's 16 keys of a chunk, widened.
    __device__ __forceinline__ void widen(const uint8_t *codes,
                                          uint4 (*to)[kTileKeys * 8],
                                          int warp) const {
        const int lane = threadIdx.x & 31;
#pragma unroll
        for (int y = 0; y < OWN * PIECES / 32; ++y) {
            const int piece = lane + 32 * y;
            const int key = warp * OWN + piece / PIECES, at = piece % PIECES;
            const uint4 w =
                *reinterpret_cast<const uint4 *>(codes + key * DIM + 16 * at);
            uint4 x0, x1;
            widen4<INT8>(w.x, x0.x, x0.y);
            widen4<INT8>(w.y, x0.z, x0.w);
            widen4<INT8>(w.z, x1.x, x1.y);
            widen4<INT8>(w.w, x1.z, x1.w);
            uint4 *row = to[at / 4] + key * 8;
            const int unit = at % 4 * 2, swap = key & 7;
            // a block's lanes begin with the first unit, the other's with the
            // second: both lie in the same banks
            const bool second = DIM == 128 && at >= 4;
            row[(unit + second) ^ swap] = second ? x1 : x0;
            row[(unit + !second) ^ swap] = second ? x0 : x1;
        }
    }
    // A chunk's scores to weights, packed by twos; returns what the sums so far
    // are to be multiplied by.  Pairs of values by one instruction each.
    __device__ __forceinline__ float weigh(const mt_attention_call_t &c, int i,
                                           int j0, int ring, int lo_all,
                                           int hi_all,
                                           unsigned (&out)[kTileKeys / 2]) {
        constexpr int N = kTileKeys / 2;
        float2 z[N];
        // Half of them at a time, as far as registers go; scales are asked for
        // ahead.
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            float4 k[N / 4];
#pragma unroll
            for (int j = 0; j < N / 4; ++j)
                k[j] = *reinterpret_cast<const float4 *>(
                    &sh.ks[ring][h * N + 4 * j]);
            unsigned r[N];
            tensor_load(r, scores_at + (i & 1) * kTileKeys + h * N);
#pragma unroll
            for (int j = 0; j < N / 4; ++j) {
                z[h * (N / 2) + 2 * j] =
                    mul2(make_float2(__uint_as_float(r[4 * j]),
                                     __uint_as_float(r[4 * j + 1])),
                         make_float2(k[j].x, k[j].y));
                z[h * (N / 2) + 2 * j + 1] =
                    mul2(make_float2(__uint_as_float(r[4 * j + 2]),
                                     __uint_as_float(r[4 * j + 3])),
                         make_float2(k[j].z, k[j].w));
            }
        }
        // Exponents of two, less the reference (none yet: 0).
        const float about = ref == -INFINITY ? 0.f : ref;
        const float2 f2 = make_float2(f, f);
        if constexpr (CAP) {
            const Cap cap(c.cap, kLog2e);
            // One vote of the warp for the whole chunk (one for every 16 keys
            // took 221 us for 178); with a far score in every chunk 233.
            float most_z = 0.f;
#pragma unroll
            for (int j = 0; j < N; ++j) {
                z[j] = mul2(z[j], f2);
                most_z = nanmax3(most_z, fabsf(z[j].x), fabsf(z[j].y));
            }
            if (!__any_sync(kFull, !(most_z < cap.near_to))) {
#pragma unroll
                for (int j = 0; j < N; ++j) z[j] = cap.near(z[j], both(-about));
            } else {
#pragma unroll
                for (int j = 0; j < N; ++j) z[j] = cap.any(z[j], about);
            }
        } else {
            const float2 less = make_float2(-about, -about);
#pragma unroll
            for (int j = 0; j < N; ++j) z[j] = fma2(z[j], f2, less);
        }
        const uint4 by_warp = *reinterpret_cast<const uint4 *>(sh.there[ring]);
        static_assert(kWarps == 4 && OWN == 16, "a word of each");
        uint64_t there = (uint64_t)(by_warp.z | by_warp.w << 16) << 32 |
                         (by_warp.x | by_warp.y << 16);
        const bool whole = ~there == 0 && j0 >= lo_all &&
                           j0 + kTileKeys - 1 <= hi_all;
        if (c.slopes != nullptr) {
#pragma unroll
            for (int j = 0; j < N; ++j) {
                z[j].x -= slope * (float)abs(p - (j0 + 2 * j));
                z[j].y -= slope * (float)abs(p - (j0 + 2 * j + 1));
            }
        }
        // (two words, so that a bit is at a constant place of one)
        unsigned w0 = 0, w1 = 0;
        if (!whole) {
            // keys lo - j0 .. hi - j0 of the chunk
            const int64_t a = (int64_t)lo - j0, b = (int64_t)hi - j0;
            if (a > 0) there &= a >= kTileKeys ? 0 : ~0ull << a;
            if (b < kTileKeys - 1) there &= b < 0 ? 0 : ~0ull >> (63 - b);
            w0 = (unsigned)there;
            w1 = (unsigned)(there >> 32);
#pragma unroll
            for (int j = 0; j < N; ++j) {
                const unsigned w = (j < N / 2 ? w0 : w1) >> (2 * j & 31);
                if (!(w & 1u)) z[j].x = -INFINITY;
                if (!(w & 2u)) z[j].y = -INFINITY;
            }
        }
        float tops[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) tops[j] = nanmax(z[j].x, z[j].y);
#pragma unroll
        for (int j = 4; j < N; ++j)
            tops[j & 3] = nanmax3(tops[j & 3], z[j].x, z[j].y);
        const float top = nanmax(nanmax(tops[0], tops[1]),
                                 nanmax(tops[2], tops[3]));
        float times = 1.f;
        if (ref == -INFINITY ? !(top == -INFINITY) : !(top <= 8.f)) {
            // the reference up to the largest so far, by what that really is
            const float next = about + top, moved = next - about;
            const float keep = ref == -INFINITY ? 0.f : pow2(-moved);
            const float2 less = make_float2(-moved, -moved);
#pragma unroll
            for (int j = 0; j < N; ++j) z[j] = add2(z[j], less);
            ref = next;
            l *= keep;
            const unsigned down_by =
                127u - min(__float_as_uint(keep) >> 23, 127u);
            const unsigned now = max(most > down_by ? most - down_by : 0u, 12u);
            times = keep * up(now) * down(most);
            most = now;
        }
        float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            float4 v[N / 4];
#pragma unroll
            for (int j = 0; j < N / 4; ++j)
                v[j] = *reinterpret_cast<const float4 *>(
                    &sh.vs[ring][h * N + 4 * j]);
#pragma unroll
            for (int j = 0; j < N / 4; ++j) {
                float2 &a = z[h * (N / 2) + 2 * j];
                float2 &b = z[h * (N / 2) + 2 * j + 1];
                a = make_float2(pow2(a.x), pow2(a.y));
                b = make_float2(pow2(b.x), pow2(b.y));
                sum[0] = add2(sum[0], a);
                sum[1] = add2(sum[1], b);
                a = mul2(a, make_float2(v[j].x, v[j].y));
                b = mul2(b, make_float2(v[j].z, v[j].w));
            }
        }
        l += (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y);
        if (!whole) {
            // not seen: nothing, whatever stands in the scale
#pragma unroll
            for (int j = 0; j < N; ++j) {
                const unsigned w = (j < N / 2 ? w0 : w1) >> (2 * j & 31);
                if (!(w & 1u)) z[j].x = 0.f;
                if (!(w & 2u)) z[j].y = 0.f;
            }
        }
        float bigs[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int j = 0; j < N; ++j)
            bigs[j & 3] = nanmax3(bigs[j & 3], fabsf(z[j].x), fabsf(z[j].y));
        const float big = nanmax(nanmax(bigs[0], bigs[1]),
                                 nanmax(bigs[2], bigs[3]));
        if (!(big * up(most) < 32768.f)) {
            const unsigned now =
                max(most, __float_as_uint(big) >> 23 & 0xffu);
            times *= up(now) * down(most);
            most = now;
        }
        const float2 by = make_float2(up(most), up(most));
#pragma unroll
        for (int j = 0; j < N; ++j) {
            z[j] = mul2(z[j], by);
            out[j] = half_pair(z[j].x, z[j].y);
        }
        return times;
    }
    // What the tile goes through: chunks u .. u + n - 1, of keys lo_any .. hi_any.
    struct Span {
        int64_t u;
        int n, lo_any, hi_any, lo_all, hi_all;
    };
    // Four warps: copies, widening, products.
    __device__ __forceinline__ void feed(const mt_attention_call_t &c,
                                         const Tile &a, const Span &t) {
        const int tid = threadIdx.x - 128, lane = tid & 31, warp = tid >> 5;
        const int32_t *pages = c.table + a.s * c.table_stride;
        const int n = t.n;
        const auto page_at = [&](int i) {
            return i < n && lane < OWN
                       ? page_of(c, pages,
                                 (t.u + i) * kTileKeys + warp * OWN + lane,
                                 t.lo_any, t.hi_any)
                       : Page{-1, 0};
        };
        const unsigned row = (unsigned)(c.k_heads * DIM);
        const uint8_t *kp =
            static_cast<const uint8_t *>(c.k_codes) + a.head * DIM;
        const uint8_t *vp =
            static_cast<const uint8_t *>(c.v_codes) + a.head * DIM;
        const auto copy = [&](const uint8_t *from, uint8_t *to, int slot) {
#pragma unroll
            for (int y = 0; y < OWN * PIECES / 32; ++y) {
                const int piece = lane + 32 * y;
                const int key = piece / PIECES, at = piece % PIECES * 16;
                const int s = __shfl_sync(kFull, slot, key);
                copy16(to + (warp * OWN + key) * DIM + at,
                       from + (uint64_t)(unsigned)max(s, 0) * row + at, s >= 0);
            }
        };
        // A chunk's keys and all its scales.
        const auto load_keys = [&](int slot, int ring) {
            copy(kp, sh.k_codes, slot);
            if (lane < OWN) {
                const uint64_t from =
                    (uint64_t)(unsigned)max(slot, 0) * (unsigned)c.k_heads +
                    a.head;
                copy_scales<4>(&sh.ks[ring][warp * OWN + lane],
                               c.k_scales + from, slot >= 0);
                copy_scales<4>(&sh.vs[ring][warp * OWN + lane],
                               c.v_scales + from, slot >= 0);
            }
            const unsigned there = __ballot_sync(kFull, slot >= 0);
            if (lane == 0) sh.there[ring][warp] = there & 0xffffu;
        };
        const auto commit = [] {
            asm volatile("cp.async.commit_group;" ::: "memory");
        };
        // What the four warps have written is there for products.
        const auto written = [] {
            fence_proxy_async_smem();
            tensor_before();
            asm volatile("barrier.cta.sync 1, 128;" ::: "memory");
        };
        const unsigned q_at = smem_addr(sh.q), k_at = smem_addr(sh.k);
        const unsigned v_at = smem_addr(sh.v);
        // (a warp's keys and scales: each warp arrives, and the products)
        const auto scores = [&](int i) {
            arrive(&sh.score_done[i & 1]);
            if (tid != 0) return;
            tensor_after();
#pragma unroll
            for (int s = 0; s < DIM / 16; ++s)
                tensor_product(
                    sh.tensor + (i & 1) * kTileKeys,
                    operand(q_at + s / 4 * (kTileColumns * 128) + s % 4 * 32, 0),
                    operand(k_at + s / 4 * (kTileKeys * 128) + s % 4 * 32, 0),
                    product_of(kTileKeys, false), s > 0);
            tensor_arrive(&sh.score_done[i & 1]);
        };
        const auto values = [&](int i) {
            if (tid != 0) return;
            wait(&sh.weights_there, weights_phase);
#pragma unroll
            for (int s = 0; s < kTileKeys / 16; ++s)
                tensor_product(sh.tensor + 2 * kTileKeys,
                               sh.tensor + (i & 1) * kTileKeys + s * 8,
                               operand(v_at + s * 2048, kTileKeys * 128),
                               product_of(DIM, true), i > 0 || s > 0);
            tensor_arrive(&sh.value_done);
        };
        // In flight: the keys of the chunk after the one whose scores are under
        // way, then the values of that.
        int slot = slot_in(c, page_at(0)), slot_v = slot;
        Page next = page_at(1);
        load_keys(slot, 0);
        commit();
        asm volatile("cp.async.wait_group 0;" ::: "memory");
        __syncwarp();
        widen(sh.k_codes, sh.k, warp);
        __syncwarp();
        int slot_next = slot_in(c, next);
        next = page_at(2);
        if (n > 1) load_keys(slot_next, 1);
        commit();
        copy(vp, sh.v_codes, slot_v);
        commit();
        written();
        scores(0);
        __syncwarp();
#pragma unroll 1
        for (int i = 0; i < n; ++i) {
            slot_v = slot_next;
            // a chunk's keys are through: the next one's in their place
            wait_all(&sh.score_done[i & 1], score_phase, i & 1);
            if (i + 1 < n) {
                asm volatile("cp.async.wait_group 1;" ::: "memory");
                __syncwarp();
                widen(sh.k_codes, sh.k, warp);
                __syncwarp();
                slot_next = slot_in(c, next);
                next = page_at(i + 3);
                if (i + 2 < n) load_keys(slot_next, i + 2 & 3);
            }
            commit();
            // the sums of the chunk before are through: its values' place and
            // its weights', which is that of the next scores, are free
            if (i > 0) wait_all(&sh.value_done, value_phase);
            if (i + 1 < n) {
                written();
                scores(i + 1);
                __syncwarp();
            }
            asm volatile("cp.async.wait_group 1;" ::: "memory");
            __syncwarp();
            widen(sh.v_codes, sh.v, warp);
            __syncwarp();
            if (i + 1 < n) copy(vp, sh.v_codes, slot_v);
            commit();
            written();
            values(i);
            __syncwarp();
        }
        asm volatile("cp.async.wait_group 0;" ::: "memory");
    }
    // Four warps: a column to a thread.
    __device__ __forceinline__ void weights(const mt_attention_call_t &c,
                                            const Span &t) {
#pragma unroll 1
        for (int i = 0; i < t.n; ++i) {
            wait_all(&sh.score_done[i & 1], score_phase, i & 1);
            unsigned w[kTileKeys / 2];
            const float times = weigh(c, i, (int)((t.u + i) * kTileKeys), i & 3,
                                      t.lo_all, t.hi_all, w);
            if (i > 0) {
                // The sums so far are complete before they are touched, and
                // the chunk before has been taken before this one arrives: no
                // barrier gets two phases ahead of who waits for it.
                wait_all(&sh.value_done, value_phase);
                if (__any_sync(kFull, !(times == 1.f))) {
#pragma unroll 1
                    for (int d = 0; d < DIM; d += 32) {
                        unsigned o[32];
                        tensor_load(o, sums_at + d);
#pragma unroll
                        for (int e = 0; e < 32; ++e)
                            o[e] = __float_as_uint(__uint_as_float(o[e]) *
                                                   times);
                        tensor_store(sums_at + d, o);
                    }
                }
            }
            // in the scores' place
            tensor_store(scores_at + (i & 1) * kTileKeys, w);
            tensor_before();
            arrive(&sh.weights_there);
        }
    }
    __device__ __forceinline__ void run(const mt_attention_call_t &c,
                                        const Cut &cut, const Tile &a,
                                        int64_t u0, int64_t u1) {
        any = false;
        if (threadIdx.x < 128) {
            begin(c, cut, a);
            fence_proxy_async_smem();
        }
        __syncthreads();
        Span t = {0, 0, INT32_MAX, -1, INT32_MIN, INT32_MAX};
#pragma unroll
        for (int x = 0; x < kWarps; ++x) {
            t.lo_any = min(t.lo_any, sh.lo_any[x]);
            t.hi_any = max(t.hi_any, sh.hi_any[x]);
            t.lo_all = max(t.lo_all, sh.lo_all[x]);
            t.hi_all = min(t.hi_all, sh.hi_all[x]);
        }
        t.u = max(u0, (int64_t)(t.lo_any / kTileKeys));
        const int64_t end =
            t.lo_any > t.hi_any
                ? 0 : min(u1, (int64_t)(t.hi_any / kTileKeys) + 1);
        if (t.u >= end) return;  // the same for all threads
        any = true;
        t.n = (int)(end - t.u);
        if (threadIdx.x < 128) weights(c, t);
        else feed(c, a, t);
        wait_all(&sh.value_done, value_phase);
    }
    __device__ __forceinline__ void end(const mt_attention_call_t &c,
                                        const Cut &cut, const Tile &a,
                                        bool whole, float *sums) {
        if (threadIdx.x < 128) put(c, cut, a, whole, sums);
        tensor_before();
        __syncthreads();  // shared and tensor memory are the next tile's
    }
    __device__ __forceinline__ void put(const mt_attention_call_t &c,
                                        const Cut &cut, const Tile &a,
                                        bool whole, float *sums) {
        const int col = threadIdx.x;
        const Place at = place_of<kTileColumns>(
            cut, begin_of(c, a.s) + a.t * cut.per,
            min(cut.per, a.tiles.rows - a.t * cut.per), a.head, a.part, col);
        if (*(volatile int *)&sh.failed) ref = NAN;
        const bool none = ref == -INFINITY;
        if (at.used && !whole) {
            sums[col] = ref;
            sums[kTileColumns + col] = l;
        }
        if (at.used && whole && c.lse != nullptr)
            c.lse[(int64_t)at.row * c.q_heads + at.head] =
                none ? ref : (ref + log2f(l)) * 0.6931471805599453f;
        const float by = down(most);
        const int64_t to =
            (int64_t)at.row * c.out_row + (int64_t)at.head * c.out_head;
#pragma unroll 1
        for (int d = 0; d < DIM; d += 32) {
            unsigned o[32];
#pragma unroll
            for (int e = 0; e < 32; ++e) o[e] = 0;
            if (any) tensor_load(o, sums_at + d);  // the same for the CTA
            if (at.used) {
#pragma unroll
                for (int e = 0; e < 32; e += 4) {
                    float v[4];
#pragma unroll
                    for (int x = 0; x < 4; ++x)
                        v[x] = __uint_as_float(o[e + x]) * by;
                    if (whole) {
#pragma unroll
                        for (int x = 0; x < 4; ++x)
                            v[x] = ref != ref ? NAN : none ? 0.f : v[x] / l;
                        store4(DT_BF16, (cut.whole & 2) != 0, c.out,
                               to + d + e, v);
                    } else {
                        *reinterpret_cast<float4 *>(sums + 2 * kTileColumns +
                                                    col * DIM + d + e) =
                            make_float4(v[0], v[1], v[2], v[3]);
                    }
                }
            }
        }
    }
};

template <int DIM, bool INT8, bool CAP>
__global__ void __launch_bounds__(64 * kWarps, 2)
    attention_tiles_kernel(const mt_attention_call_t c, const Cut cut,
                           const Share share, int) {
    extern __shared__ uint8_t tiles_shared[];
    // operands begin at multiples of 1024
    TileShared<DIM> &sh = *reinterpret_cast<TileShared<DIM> *>(
        tiles_shared + (-smem_addr(tiles_shared) & 1023u));
    const int warp = threadIdx.x >> 5;
    grid_wait_prerequisites();
    if (warp == 0) {
        asm volatile(
            "tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;\n\t"
            "tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::"r"(
                smem_addr(&sh.tensor)),
            "n"(kTensorColumns)
            : "memory");
    }
    if (threadIdx.x == 0) {
        for (int b = 0; b < 2; ++b)
            mbar_init(&sh.score_done[b], 1 + kWarps);
        mbar_init(&sh.weights_there, kWarps);
        mbar_init(&sh.value_done, 1);
        mbar_init_fence();
        sh.failed = 0;
    }
    tensor_before();
    __syncthreads();
    tensor_after();
    TileRun<DIM, INT8, CAP> r(sh);
    r.scores_at = sh.tensor + ((unsigned)(warp & 3) * 32 << 16);
    r.sums_at = r.scores_at + 2 * kTileKeys;
    deal_units<2 * kWarps>(
               c, cut, share, sh.deal,
               [&](const Tile &a, int64_t u0, int64_t u1, bool whole,
                   int place) {
                   r.run(c, cut, a, u0, u1);
                   r.end(c, cut, a, whole,
                         share.sums + (2 * (int64_t)blockIdx.x + place) *
                                          place_floats(kTileColumns, DIM));
               });
    if (*(volatile int *)&sh.failed) {  // once more, for what is under way
        for (int b = 0; b < 2; ++b)
            mbar_wait_bounded(&sh.score_done[b], (r.score_phase >> b & 1) ^ 1);
        mbar_wait_bounded(&sh.value_done, r.value_phase ^ 1);
    }
    __syncthreads();
    if (warp == 0)
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(
                         sh.tensor),
                     "n"(kTensorColumns)
                     : "memory");
}

template <int DIM, bool INT8, bool CAP>
cudaError_t launch_tiles_as(const AttentionPlan &p,
                            const mt_attention_call_t &c, int dtype,
                            void *workspace, cudaStream_t s) {
    constexpr size_t kBytes = sizeof(TileShared<DIM>) + 1024;
    static_assert((kBytes + 1024) * 2 <= 228 * 1024,
                  "two CTAs fit an SM's shared memory");
    const Cut cut = {p.times, p.per, p.parts, 1, 6, c.k_heads * p.parts,
                     p.whole};
    Share share;
    share.sums = static_cast<float *>(workspace);
    share.records = reinterpret_cast<Record *>(
        share.sums + 2 * (int64_t)p.ctas * place_floats(kTileColumns, DIM));
    share.cut = reinterpret_cast<int32_t *>(share.records + p.ctas);
    const auto kernel = attention_tiles_kernel<DIM, INT8, CAP>;
    cudaError_t e = allow_max_smem(reinterpret_cast<const void *>(kernel));
    if (e == cudaSuccess)
        e = launch_dependent(kernel, p.ctas, 64 * kWarps, kBytes, s, c, cut,
                             share, dtype);
    if (e != cudaSuccess) return e;
    return launch_dependent(attention_join_kernel<DIM, kTileColumns, 1>,
                            kJoinCtas * p.ctas, kJoin, 0, s, c, cut, share,
                            dtype, p.ctas);
}

template <bool INT8>
cudaError_t launch_tiles(const AttentionPlan &p, const mt_attention_call_t &c,
                         int dtype, void *workspace, cudaStream_t s) {
    const auto launch =
        c.dim == 128 ? c.cap > 0.f ? launch_tiles_as<128, INT8, true>
                                   : launch_tiles_as<128, INT8, false>
        : c.cap > 0.f ? launch_tiles_as<64, INT8, true>
                      : launch_tiles_as<64, INT8, false>;
    return launch(p, c, dtype, workspace, s);
}

}  // namespace

#define MT_DEFINE_ATTENTION_TILES(name, int8)                                \
    cudaError_t name(const AttentionPlan &p, const mt_attention_call_t &c,   \
                     int dtype, void *workspace, cudaStream_t s) {           \
        return launch_tiles<int8>(p, c, dtype, workspace, s);                \
    }

}  // namespace mt

// attention_rows.cuh -- attention over the quantised cache for many rows of a
// sequence (prompts): one translation unit per code format and number of parts.
//
// Here the queries are many enough to fill the instruction's 16 rows: a tile has
// 64 columns (rows of a sequence times the query heads of a key head), 16 to a
// warp, and all four warps go through the same chunks of 64 keys.  A chunk's
// codes are copied as they are while the one before is worked on, widened to
// FP16 once for all warps, and read from there as fragments by matrix loads
// (rows permuted so that those touch every bank once).  Scores, references,
// scales and roundings are as in attention_mma.cuh; what the scores give is the
// other product's first operand as it lies.  Units, cut tiles and their joining
// are the same too.
//
// Taken from 48 columns per sequence on, on average: 32 rows of two sequences 34
// us for 41 on tiles of 16 columns, 16 rows of 16 sequences (34 columns) 73 for
// 66; BF16 with one group a head only to 256 (attention_tiles.cuh).
//
// Bound: shared memory (73% of its throughput: every warp reads all of a chunk
// for its 16 columns) and the instructions around the products; those have 34%
// of the tensor pipe (with two parts, FP16, 58% and 51%).  Two
// sequences of up to 512 rows at 4096 keys, 32 + 8 heads of 128, causal: FP16 383
// us (capped 416), FP32 387; BF16 with two groups a head 318, four 392 (184 bytes
// spilled, FP32 312; one group 180); heads of 96 230.  BF16 with one group took
// 308 here, capped, and 372 on tiles of 16.
#pragma once

#include "attention_mma.cuh"

namespace mt {
namespace {

constexpr int kRowColumns = 64, kRowKeys = 64;

template <class H, int PARTS>
struct RowShared {
    // 16-byte units of FP16 of a key, and the room that a row of them takes
    // (a multiple of 8 units, so that they can be permuted by the key).
    static constexpr int UNITS = H::DIM / 8;
    static constexpr int ROOM = (UNITS + 7) / 8 * 8;
    struct Codes {
        uint8_t k[kRowKeys * H::DIM], v[kRowKeys * H::DIM];
        float ks[kRowKeys][H::GROUPS], vs[kRowKeys][H::GROUPS];
    };
    Codes codes;
    uint4 k[kRowKeys * ROOM], v[kRowKeys * ROOM];
    float ks[kRowKeys][H::GROUPS], vs[kRowKeys][H::GROUPS];
    uint4 q[kWarps][PARTS][H::STEPS][32];  // fragments
    unsigned there[kWarps];          // keys with a slot, 16 to a warp
    int32_t lo_any[2], hi_any[2], lo_all[2], hi_all[2];
    Deal deal;
    static __device__ __forceinline__ int place(int key, int unit) {
        return key * ROOM + (unit ^ (key & 7));
    }
};

__device__ __forceinline__ void load_matrices(unsigned (&r)[4],
                                              const void *p) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, "
                 "[%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(smem_addr(p)));
}
__device__ __forceinline__ void load_matrices_t(unsigned (&r)[4],
                                                const void *p) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, "
                 "%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(smem_addr(p)));
}
// Two values of a row of queries.
__device__ __forceinline__ float2 load2(int dtype, bool whole, const void *p,
                                        int64_t i) {
    if (!whole) return make_float2(load_as(dtype, p, i),
                                   load_as(dtype, p, i + 1));
    float v[2];
    if (dtype == DT_BF16)
        ld_vec<__nv_bfloat16, 2>(static_cast<const __nv_bfloat16 *>(p) + i, v);
    else if (dtype == DT_F16)
        ld_vec<__half, 2>(static_cast<const __half *>(p) + i, v);
    else
        ld_vec<float, 2>(static_cast<const float *>(p) + i, v);
    return make_float2(v[0], v[1]);
}
__device__ __forceinline__ void store2(int dtype, bool whole, void *p,
                                       int64_t i, float a, float b) {
    const float v[2] = {a, b};
    if (!whole) {
        store_as(dtype, p, i, a);
        store_as(dtype, p, i + 1, b);
    } else if (dtype == DT_BF16) {
        st_vec<__nv_bfloat16, 2>(static_cast<__nv_bfloat16 *>(p) + i, v);
    } else if (dtype == DT_F16) {
        st_vec<__half, 2>(static_cast<__half *>(p) + i, v);
    } else {
        st_vec<float, 2>(static_cast<float *>(p) + i, v);
    }
}

// A warp's 16 columns: lane (g, q) has columns g and g + 8 ("row" i = 0, 1 of
// the instruction's fragments), of a tile of keys 2 q and 2 q + 1.
template <class H, bool INT8, int PARTS>
struct RowWarp {
    static constexpr int N = kRowKeys / 8;      // tiles of 8 keys of a chunk
    static constexpr int TILES = H::DIM / 8;    // of the output
    using Sh = RowShared<H, PARTS>;
    float o[TILES][4];              // in units of 2^-(up of its group)
    float ref[2], l[2], f[2], slope[2];
    int lo[2], hi[2], p[2];
    unsigned most[2][(H::GROUPS + 3) / 4];

    __device__ __forceinline__ unsigned exponent(int i, int gr) const {
        return max(most[i][gr / 4] >> gr % 4 * 8 & 0xffu, 12u);
    }
    __device__ __forceinline__ void set(int i, int gr, unsigned e) {
        unsigned &w = most[i][gr / 4];
        w = (w & ~(0xffu << gr % 4 * 8)) | e << gr % 4 * 8;
    }
    static __device__ __forceinline__ float up(unsigned e) {
        return __uint_as_float((265u - e) << 23);
    }
    static __device__ __forceinline__ float down(unsigned e) {
        return __uint_as_float((e - 11u) << 23);
    }
    // A group's sums of column i times a factor.
    __device__ __forceinline__ void times(int i, int gr, float x) {
#pragma unroll
        for (int d = gr * (H::GROUP / 8); d < (gr + 1) * (H::GROUP / 8); ++d) {
            o[d][2 * i] *= x;
            o[d][2 * i + 1] *= x;
        }
    }
    // The tile's queries as fragments, its columns' factors and bounds.
    __device__ __forceinline__ void begin(const mt_attention_call_t &c,
                                          const Cut &cut, int dtype,
                                          const Tile &a, Sh &sh) {
        const int lane = threadIdx.x & 31, g = lane >> 2, q = lane & 3;
        const int from = begin_of(c, a.s);
        const int first = from + a.t * cut.per;
        const int rows = min(cut.per, a.tiles.rows - a.t * cut.per);
        const int dt = PARTS == 1 ? (int)DT_BF16 : dtype;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int col = (threadIdx.x >> 5) * 16 + g + 8 * i;
            const Place at = place_of<kRowColumns>(cut, first, rows, a.head,
                                                   a.part, col);
            const int64_t x0 =
                (int64_t)at.row * c.q_row + (int64_t)at.head * c.q_head;
            float2 x[H::STEPS][2];
            float largest = 0.f;
#pragma unroll
            for (int s = 0; s < H::STEPS; ++s)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    x[s][h] = make_float2(0.f, 0.f);
                    if (at.used)
                        x[s][h] = load2(dt, cut.whole & 1, c.q,
                                        x0 + 16 * s + 8 * h + 2 * q);
                }
#pragma unroll
            for (int s = 0; s < H::STEPS; ++s)
#pragma unroll
                for (int h = 0; h < 2; ++h)
                    largest = nanmax3(largest, fabsf(x[s][h].x),
                                      fabsf(x[s][h].y));
            largest = nanmax(largest, __shfl_xor_sync(kFull, largest, 1));
            largest = nanmax(largest, __shfl_xor_sync(kFull, largest, 2));
            const unsigned e = max(__float_as_uint(largest) >> 23, 15u);
            const bool bad = !(largest < INFINITY);
            const float by = bad ? 0.f : __uint_as_float((268u - e) << 23);
#pragma unroll
            for (int s = 0; s < H::STEPS; ++s)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const float u = bad ? 0.f : x[s][h].x * by;
                    const float v = bad ? 0.f : x[s][h].y * by;
                    const unsigned w = half_pair(u, v);
                    unsigned *to = &sh.q[threadIdx.x >> 5][0][s][lane].x;
                    to[2 * h + i] = w;
                    if constexpr (PARTS == 2) {
                        const float2 r = from_half_pair(w);
                        to[H::STEPS * 128 + 2 * h + i] =
                            half_pair(u - r.x, v - r.y);
                    }
                }
            f[i] = bad ? NAN
                       : c.scale * kLog2e * __uint_as_float((e - 14u) << 23);
            slope[i] = 0.f;
            lo[i] = INT32_MIN;
            hi[i] = INT32_MAX;
            p[i] = 0;
            if (at.used) {
                const int64_t n = (int64_t)begin_of(c, a.s + 1) - from;
                const int64_t start = c.starts[a.s];
                const int64_t pos = start + (at.row - from);
                int64_t b0, b1;
                row_sees(c, at.row, pos, start + n, b0, b1);
                if (c.slopes != nullptr) slope[i] = c.slopes[at.head] * kLog2e;
                lo[i] = (int)min(b0, (int64_t)INT32_MAX);
                hi[i] = (int)max(min(b1, (int64_t)INT32_MAX), (int64_t)-1);
                p[i] = (int)min(pos, (int64_t)INT32_MAX);
            }
            ref[i] = -INFINITY;
            l[i] = 0.f;
#pragma unroll
            for (int y = 0; y < (H::GROUPS + 3) / 4; ++y) most[i][y] = 0;
        }
#pragma unroll
        for (int d = 0; d < TILES; ++d)
#pragma unroll
            for (int e = 0; e < 4; ++e) o[d][e] = 0.f;
    }
    __device__ __forceinline__ void scores(const Sh &sh, float (&z)[N][4]) {
        const int lane = threadIdx.x & 31, q = lane & 3;
#pragma unroll
        for (int gr = 0; gr < H::GROUPS; ++gr) {
#pragma unroll
            for (int n0 = 0; n0 < N; n0 += 4) {
                // four tiles in turn, so that no product waits for the last
                float acc[4][4] = {};
#pragma unroll
                for (int s = gr * H::PER; s < (gr + 1) * H::PER; s += 2) {
                    // 8 keys, four units: two steps
                    unsigned b[4][4];
#pragma unroll
                    for (int y = 0; y < 4; ++y)
                        load_matrices(
                            b[y], &sh.k[Sh::place(8 * (n0 + y) + (lane & 7),
                                                  2 * s + (lane >> 3))]);
#pragma unroll
                    for (int part = 0; part < PARTS; ++part)
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            const uint4 f4 =
                                sh.q[threadIdx.x >> 5][part][s + h][lane];
                            const unsigned q4[4] = {f4.x, f4.y, f4.z, f4.w};
#pragma unroll
                            for (int y = 0; y < 4; ++y)
                                mma16816(acc[y], q4, b[y][2 * h],
                                         b[y][2 * h + 1]);
                        }
                }
#pragma unroll
                for (int y = 0; y < 4; ++y)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const int n = n0 + y;
                        const float k = sh.ks[8 * n + 2 * q + e][gr];
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            float &to = z[n][2 * i + e];
                            const float from = acc[y][2 * i + e];
                            to = gr == 0 ? from * k : fmaf(from, k, to);
                        }
                    }
            }
        }
    }
    // As in attention_mma.cuh; hidden: a bit for each of z's values.
    __device__ __forceinline__ bool bend(const mt_attention_call_t &c,
                                         bool whole, int j0, uint64_t there,
                                         unsigned &hidden, float (&z)[N][4]) {
        hidden = 0;
        const int q = threadIdx.x & 3;
#pragma unroll
        for (int n = 0; n < N; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) z[n][e] *= f[e >> 1];
        if (c.cap > 0.f) {
            const Cap cap(c.cap, kLog2e);
            cap_scores(cap, z);
        }
        if (c.slopes == nullptr && whole) return false;
#pragma unroll
        for (int n = 0; n < N; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int at = 8 * n + 2 * q + (e & 1), i = e >> 1;
                if (c.slopes != nullptr)
                    z[n][e] -= slope[i] * (float)abs(p[i] - (j0 + at));
                if (!whole && !(there >> at & 1u && j0 + at >= lo[i] &&
                                j0 + at <= hi[i])) {
                    z[n][e] = -INFINITY;
                    hidden |= 1u << (4 * n + e);
                }
            }
        return !whole;
    }
    __device__ __forceinline__ void weigh(float (&z)[N][4]) {
        float top[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            top[i] = nanmax(z[0][2 * i], z[0][2 * i + 1]);
#pragma unroll
            for (int n = 1; n < N; ++n)
                top[i] = nanmax3(top[i], z[n][2 * i], z[n][2 * i + 1]);
        }
        const bool ahead =
            !(top[0] <= ref[0] + 8.f) || !(top[1] <= ref[1] + 8.f);
        if (__any_sync(kFull, ahead)) {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                float t = nanmax(ref[i], top[i]);
                t = nanmax(t, __shfl_xor_sync(kFull, t, 1));
                t = nanmax(t, __shfl_xor_sync(kFull, t, 2));
                const float keep = pow2(ref[i] - (t == -INFINITY ? 0.f : t));
                ref[i] = t;
                l[i] *= keep;
                const unsigned less =
                    127u - min(__float_as_uint(keep) >> 23, 127u);
#pragma unroll
                for (int gr = 0; gr < H::GROUPS; ++gr) {
                    const unsigned old = exponent(i, gr);
                    const unsigned now = max(old > less ? old - less : 0u, 12u);
                    set(i, gr, now);
                    times(i, gr, keep * up(now) * down(old));
                }
            }
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const float about = ref[i] == -INFINITY ? 0.f : ref[i];
#pragma unroll
            for (int n = 0; n < N; ++n)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    float &w = z[n][2 * i + e];
                    w = pow2(w - about);
                    l[i] += w;
                }
        }
    }
    __device__ __forceinline__ void add(const float (&w)[N][4],
                                        unsigned hidden, bool masked,
                                        const Sh &sh) {
        const int lane = threadIdx.x & 31, q = lane & 3;
#pragma unroll
        for (int gr = 0; gr < H::GROUPS; ++gr) {
            float x[N][4];
#pragma unroll
            for (int n = 0; n < N; ++n)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    x[n][e] = w[n][e] * sh.vs[8 * n + 2 * q + (e & 1)][gr];
            if (masked) {
                // not seen: nothing, whatever stands in the scale
#pragma unroll
                for (int n = 0; n < N; ++n)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        if (hidden >> (4 * n + e) & 1u) x[n][e] = 0.f;
            }
            float top[2] = {0.f, 0.f};
#pragma unroll
            for (int n = 0; n < N; ++n)
#pragma unroll
                for (int i = 0; i < 2; ++i)
                    top[i] = nanmax3(top[i], fabsf(x[n][2 * i]),
                                     fabsf(x[n][2 * i + 1]));
            const bool out = !(top[0] * up(exponent(0, gr)) < 32768.f) ||
                             !(top[1] * up(exponent(1, gr)) < 32768.f);
            if (__any_sync(kFull, out)) {
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    unsigned e = __float_as_uint(top[i]) >> 23 & 0xffu;
                    e = max(e, __shfl_xor_sync(kFull, e, 1));
                    e = max(e, __shfl_xor_sync(kFull, e, 2));
                    const unsigned old = exponent(i, gr), now = max(old, e);
                    set(i, gr, now);
                    times(i, gr, up(now) * down(old));
                }
            }
            const float by[2] = {up(exponent(0, gr)), up(exponent(1, gr))};
            unsigned pf[PARTS][N / 2][4];
#pragma unroll
            for (int n = 0; n < N; ++n)
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const float u = x[n][2 * i] * by[i];
                    const float v = x[n][2 * i + 1] * by[i];
                    const unsigned h = half_pair(u, v);
                    pf[0][n / 2][2 * (n & 1) + i] = h;
                    if constexpr (PARTS == 2) {
                        const float2 r = from_half_pair(h);
                        pf[1][n / 2][2 * (n & 1) + i] =
                            half_pair(u - r.x, v - r.y);
                    }
                }
#pragma unroll
            for (int d = gr * (H::GROUP / 8); d < (gr + 1) * (H::GROUP / 8);
                 d += 4) {
                float acc[4][4];
#pragma unroll
                for (int y = 0; y < 4; ++y)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        acc[y][e] = PARTS == 1 ? o[d + y][e] : 0.f;
#pragma unroll
                for (int t = 0; t < N / 2; ++t) {
                    // 16 keys, two units each: four tiles of the output
                    unsigned b[2][4];
#pragma unroll
                    for (int y = 0; y < 2; ++y)
                        load_matrices_t(
                            b[y],
                            &sh.v[Sh::place(16 * t + (lane & 15),
                                            d + 2 * y + (lane >> 4))]);
#pragma unroll
                    for (int part = 0; part < PARTS; ++part)
#pragma unroll
                        for (int y = 0; y < 4; ++y)
                            mma16816(acc[y], pf[part][t], b[y / 2][2 * (y & 1)],
                                     b[y / 2][2 * (y & 1) + 1]);
                }
#pragma unroll
                for (int y = 0; y < 4; ++y)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        o[d + y][e] = PARTS == 1 ? acc[y][e]
                                                 : o[d + y][e] + acc[y][e];
            }
        }
    }
    __device__ __forceinline__ void end(const mt_attention_call_t &c,
                                        const Cut &cut, int dtype,
                                        const Tile &a, bool whole,
                                        float *sums) {
        const int lane = threadIdx.x & 31, g = lane >> 2, q = lane & 3;
        const int first = begin_of(c, a.s) + a.t * cut.per;
        const int rows = min(cut.per, a.tiles.rows - a.t * cut.per);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            float sum = l[i];
            sum += __shfl_xor_sync(kFull, sum, 1);
            sum += __shfl_xor_sync(kFull, sum, 2);
            const int col = (threadIdx.x >> 5) * 16 + g + 8 * i;
            const Place at = place_of<kRowColumns>(cut, first, rows, a.head,
                                                   a.part, col);
            if (!at.used) continue;
            const bool none = ref[i] == -INFINITY;
            if (!whole && q == 0) {
                sums[col] = ref[i];
                sums[kRowColumns + col] = sum;
            }
            if (whole && q == 0 && c.lse != nullptr)
                c.lse[(int64_t)at.row * c.q_heads + at.head] =
                    none ? ref[i]
                         : (ref[i] + log2f(sum)) * 0.6931471805599453f;
            const int64_t to =
                (int64_t)at.row * c.out_row + (int64_t)at.head * c.out_head;
#pragma unroll
            for (int d = 0; d < TILES; ++d) {
                const float by = down(exponent(i, d / (H::GROUP / 8)));
                const float x = o[d][2 * i] * by, y = o[d][2 * i + 1] * by;
                if (whole)
                    store2(PARTS == 1 ? (int)DT_BF16 : dtype,
                           (cut.whole & 2) != 0, c.out, to + 8 * d + 2 * q,
                           none ? 0.f : x / sum, none ? 0.f : y / sum);
                else
                    *reinterpret_cast<float2 *>(sums + 2 * kRowColumns +
                                                col * H::DIM + 8 * d + 2 * q) =
                        make_float2(x, y);
            }
        }
    }
};

template <class H, bool INT8, int PARTS>
__device__ __forceinline__ void rows_run(const mt_attention_call_t &c,
                                         const Cut &cut, int dtype,
                                         const Tile &a, int64_t u0, int64_t u1,
                                         RowShared<H, PARTS> &sh,
                                         RowWarp<H, INT8, PARTS> &w) {
    using Sh = RowShared<H, PARTS>;
    constexpr int N = kRowKeys / 8, kOwn = kRowKeys / kWarps;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    w.begin(c, cut, dtype, a, sh);
    // What the columns see: two warps look at 32 each.
    if (warp < 2) {
        const int from = begin_of(c, a.s);
        const Place at = place_of<kRowColumns>(
            cut, from + a.t * cut.per,
            min(cut.per, a.tiles.rows - a.t * cut.per), a.head, a.part, tid);
        int lo = INT32_MIN, hi = INT32_MAX;
        if (at.used) {
            const int64_t n = (int64_t)begin_of(c, a.s + 1) - from;
            const int64_t start = c.starts[a.s];
            int64_t b0, b1;
            row_sees(c, at.row, start + (at.row - from), start + n, b0, b1);
            lo = (int)min(b0, (int64_t)INT32_MAX);
            hi = (int)max(min(b1, (int64_t)INT32_MAX), (int64_t)-1);
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
    }
    __syncthreads();
    const int lo = min(sh.lo_any[0], sh.lo_any[1]);
    const int hi = max(sh.hi_any[0], sh.hi_any[1]);
    const int lo_all = max(sh.lo_all[0], sh.lo_all[1]);
    const int hi_all = min(sh.hi_all[0], sh.hi_all[1]);
    const int32_t *pages = c.table + a.s * c.table_stride;
    int64_t u = max(u0, (int64_t)(lo / kRowKeys));
    const int64_t end = lo > hi ? 0 : min(u1, (int64_t)(hi / kRowKeys) + 1);
    // A warp copies 16 keys of a chunk.
    const auto page_at = [&](int64_t v) {
        return v < end && lane < kOwn
                   ? page_of(c, pages, v * kRowKeys + warp * kOwn + lane, lo,
                             hi)
                   : Page{-1, 0};
    };
    const unsigned row = (unsigned)(c.k_heads * H::DIM);
    const unsigned scales = (unsigned)(c.k_heads * H::GROUPS);
    const uint8_t *kp = static_cast<const uint8_t *>(c.k_codes) +
                        a.head * H::DIM;
    const uint8_t *vp = static_cast<const uint8_t *>(c.v_codes) +
                        a.head * H::DIM;
    const auto load = [&](Page page) {
        constexpr int kPieces = H::DIM / 16;
        const int slot = slot_in(c, page);
        typename Sh::Codes &to = sh.codes;
#pragma unroll
        for (int i = 0; i < kOwn * kPieces / 32; ++i) {
            const int piece = lane + 32 * i;
            const int key = piece / kPieces, at = piece % kPieces * 16;
            const int s = __shfl_sync(kFull, slot, key);
            const uint64_t from = (uint64_t)(unsigned)max(s, 0) * row + at;
            const int place = (warp * kOwn + key) * H::DIM + at;
            copy16(to.k + place, kp + from, s >= 0);
            copy16(to.v + place, vp + from, s >= 0);
        }
        if (lane < kOwn) {
            const uint64_t from = (uint64_t)(unsigned)max(slot, 0) * scales;
            const int key = warp * kOwn + lane;
            copy_scales<4 * H::GROUPS>(
                to.ks[key], c.k_scales + a.head * H::GROUPS + from, slot >= 0);
            copy_scales<4 * H::GROUPS>(
                to.vs[key], c.v_scales + a.head * H::GROUPS + from, slot >= 0);
        }
        const unsigned there = __ballot_sync(kFull, slot >= 0);
        if (lane == 0) sh.there[warp] = there & 0xffffu;
    };
    const Page first = page_at(u);
    Page next = page_at(u + 1);
    if (u < end) load(first);
    asm volatile("cp.async.commit_group;" ::: "memory");
#pragma unroll 1
    for (; u < end; ++u) {
        asm volatile("cp.async.wait_group 0;" ::: "memory");
        __syncthreads();  // the chunk is there, the one before is done with
        const typename Sh::Codes &st = sh.codes;
        uint64_t there = 0;
#pragma unroll
        for (int x = 0; x < kWarps; ++x)
            there |= (uint64_t)sh.there[x] << (kOwn * x);
        for (int x = tid; x < kRowKeys * H::GROUPS; x += 32 * kWarps) {
            sh.ks[0][x] = st.ks[0][x];
            sh.vs[0][x] = st.vs[0][x];
        }
        // Widened once for all: 16 codes are two units.
        constexpr int kPieces = H::DIM / 16;
#pragma unroll
        for (int y = 0; y < 2 * kRowKeys * kPieces / (32 * kWarps); ++y) {
            const int half = kRowKeys * kPieces;
            const int at = tid + 32 * kWarps * y;
            const bool values = at >= half;
            const int piece = at - (values ? half : 0);
            const int key = piece / kPieces, unit = piece % kPieces;
            const uint4 w = reinterpret_cast<const uint4 *>(
                values ? st.v : st.k)[piece];
            uint4 x0, x1;
            widen4<INT8>(w.x, x0.x, x0.y);
            widen4<INT8>(w.y, x0.z, x0.w);
            widen4<INT8>(w.z, x1.x, x1.y);
            widen4<INT8>(w.w, x1.z, x1.w);
            uint4 *to = values ? sh.v : sh.k;
            to[Sh::place(key, 2 * unit)] = x0;
            to[Sh::place(key, 2 * unit + 1)] = x1;
        }
        __syncthreads();
        // The codes' place is free: the next chunk is on its way while this
        // one is worked on.
        const Page then = next;
        next = page_at(u + 2);
        if (u + 1 < end) load(then);
        asm volatile("cp.async.commit_group;" ::: "memory");
        if (there == 0) continue;
        const int j0 = (int)(u * kRowKeys);
        const bool whole = ~there == 0 && j0 >= lo_all &&
                           j0 + kRowKeys - 1 <= hi_all;
        float z[N][4];
        unsigned hidden;
        w.scores(sh, z);
        const bool masked = w.bend(c, whole, j0, there, hidden, z);
        w.weigh(z);
        w.add(z, hidden, masked, sh);
    }
    asm volatile("cp.async.wait_group 0;" ::: "memory");
}

template <class H, bool INT8, int PARTS>
__global__ void __launch_bounds__(32 * kWarps, attention_row_ctas(H::DIM, H::GROUPS, PARTS))
    attention_rows_kernel(const mt_attention_call_t c, const Cut cut,
                          const Share share, int dtype) {
    extern __shared__ __align__(16) uint8_t shared[];
    RowShared<H, PARTS> &sh =
        *reinterpret_cast<RowShared<H, PARTS> *>(shared);
    grid_wait_prerequisites();
    RowWarp<H, INT8, PARTS> w;
    deal_units(c, cut, share, sh.deal,
               [&](const Tile &a, int64_t u0, int64_t u1, bool whole,
                   int place) {
                   rows_run<H, INT8, PARTS>(c, cut, dtype, a, u0, u1, sh, w);
                   w.end(c, cut, dtype, a, whole,
                         share.sums + (2 * (int64_t)blockIdx.x + place) *
                                          place_floats(kRowColumns, H::DIM));
                   __syncthreads();  // shared memory is the next tile's
               });
}

template <class H, bool INT8, int PARTS>
cudaError_t launch_rows_as(const AttentionPlan &p,
                           const mt_attention_call_t &c, int dtype,
                           void *workspace, cudaStream_t s) {
    constexpr size_t kBytes = sizeof(RowShared<H, PARTS>);
    static_assert((kBytes + 1024) * attention_row_ctas(H::DIM, H::GROUPS, PARTS) <= 228 * 1024,
                  "the CTAs that share an SM fit its shared memory");
    const Cut cut = {p.times, p.per, p.parts, 1, 6, c.k_heads * p.parts,
                     p.whole};
    Share share;
    share.sums = static_cast<float *>(workspace);
    share.records = reinterpret_cast<Record *>(
        share.sums + 2 * (int64_t)p.ctas * place_floats(kRowColumns, H::DIM));
    share.cut = reinterpret_cast<int32_t *>(share.records + p.ctas);
    const auto kernel = attention_rows_kernel<H, INT8, PARTS>;
    cudaError_t e = cudaSuccess;
    if (kBytes > 40 * 1024)
        e = allow_max_smem(reinterpret_cast<const void *>(kernel));
    if (e == cudaSuccess)
        e = launch_dependent(kernel, p.ctas, 32 * kWarps, kBytes, s, c, cut,
                             share, dtype);
    if (e != cudaSuccess) return e;
    return launch_dependent(attention_join_kernel<H::DIM, kRowColumns, 1>,
                            kJoinCtas * p.ctas, kJoin, 0, s, c, cut, share,
                            dtype, p.ctas);
}

template <bool INT8, int PARTS>
cudaError_t launch_rows(const AttentionPlan &p, const mt_attention_call_t &c,
                        int dtype, void *workspace, cudaStream_t s) {
#define MT_ATTENTION_HEAD(d, g)                                              \
    if (c.dim == d && c.dim / c.group == g)                                  \
        return launch_rows_as<Head<d, g>, INT8, PARTS>(p, c, dtype,          \
                                                       workspace, s);
    MT_ATTENTION_HEAD(64, 1)
    MT_ATTENTION_HEAD(64, 2)
    MT_ATTENTION_HEAD(96, 1)
    MT_ATTENTION_HEAD(128, 1)
    MT_ATTENTION_HEAD(128, 2)
    MT_ATTENTION_HEAD(128, 4)
#undef MT_ATTENTION_HEAD
    return cudaErrorInvalidValue;
}

}  // namespace

#define MT_DEFINE_ATTENTION_ROWS(name, int8, parts)                          \
    cudaError_t name(const AttentionPlan &p, const mt_attention_call_t &c,   \
                     int dtype, void *workspace, cudaStream_t s) {           \
        return launch_rows<int8, parts>(p, c, dtype, workspace, s);          \
    }

}  // namespace mt

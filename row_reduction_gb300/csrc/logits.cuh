// logits.cuh -- a row of logits: penalties for tokens of its history, biases,
// temperature, grammar mask, and the row's softmax or log-softmax (one
// translation unit per storage type).
//
// A row is shared out between C CTAs (a power of two) so that a CTA's logits
// stay in registers: K packs of V values per thread, asked for before anything
// else.  While they arrive, the CTA counts, for its own logits only, the
// tokens of the row's history in shared memory; integer atomics, whose order
// changes nothing.  A bit per logit says whether its counter is in use, so
// the pass over the logits reads one byte per pack and the counters of
// touched tokens only.  Every CTA of a row reads the whole history, from L2
// after the first.
//
// Ownership.  Chunks of 32 packs (one access of a warp) go round robin to the
// CTAs: frequent tokens have low ids in most vocabularies, and contiguous
// slices would give one CTA most of a row's history.
//
// Softmax.  A thread takes its exponentials about its own largest value;
// warps, then CTAs, join their (max, sum) pairs, the CTAs of a row, a cluster,
// through distributed shared memory behind one cluster barrier; and each
// thread scales its exponentials once.
//
// Bound.  Without history 5.2 us for 64 x 131072 BF16 (33.5 MB, which L2
// holds) and 40 us for the softmax of 256 x 131072 (half the copy bandwidth).
// With history a CTA is a chain of short phases (count, touch, join, write),
// of which the two CTAs that 64 registers allow per SM do not hide all: 19 us
// with 8192 tokens and 300 biases per row, 65 us with 1024 tokens and a mask.
// Short rows are the farthest from their bytes' time: each still holds half an
// SM through the whole chain (459 x 2798 FP16 with 225 biases 17 us).  FP32
// with 32 values per thread does not fit 64 registers (132 to 256 bytes of
// spills): softmax of 256 x 65536 35 us, with 1024 tokens and a mask 63 us.
//
// Alignment.  Packs of V values start at 16-byte boundaries of x: pack p of
// a row holds columns p V - shift + e, shift being the row's address modulo
// 16 in elements, so only a row's first and last pack can be partial; such
// rows take guarded kernels (348 x 35405 BF16 25 us, 348 x 35408 18 us).  The
// ids of a history are read 16 bytes at a time where every row of them starts
// at a 16-byte boundary, else one by one (64 x 131072 with a history of 8191
// 23 us, of 8192 19 us; 17 x 50257 with 32767 27 us, with 32768 20 us).
#pragma once

#include "mt_decoder.cuh"

namespace mt {
namespace {

// Counter of a token: bit 31 "in the prompt", bits 20..30 the number of its
// bias + 1 (kSeveral: more than one), bits 0..19 how often it comes after
// the prompt.
constexpr unsigned kPrompt = 1u << 31;
constexpr int kBiasShift = 20;
constexpr unsigned kCountMask = (1u << kBiasShift) - 1;
constexpr unsigned kSeveral = 0x7ffu;
constexpr int kMaxThreads = 512;

// Reads a pair at the same shared-memory offset in the CTA of cluster rank
// `rank`.
__device__ __forceinline__ float2 ld_cluster2(const float2 *p, unsigned rank) {
    const unsigned local =
        static_cast<unsigned>(__cvta_generic_to_shared(p));
    unsigned remote;
    float2 v;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;"
                 : "=r"(remote)
                 : "r"(local), "r"(rank));
    asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];"
                 : "=f"(v.x), "=f"(v.y)
                 : "r"(remote)
                 : "memory");
    return v;
}

struct Params {
    mt_logits_call_t c;
    int32_t log2C;   // CTAs per row
    int32_t packs;   // packs per CTA, a multiple of 32
    int32_t wide_tokens;  // every row of tokens starts at a 16-byte boundary
};

// Which tokens are a CTA's own, and where it keeps their counters.
template <int V>
struct Place {
    static constexpr int kLog2Chunk = V == 8 ? 8 : 7;  // 32 V columns
    int shift, log2C, vocab;
    unsigned mine, mask;  // (id + shift) & mask == mine: a CTA's chunk
    __device__ __forceinline__ Place(int shift_, int log2C_, int rank,
                                     int vocab_)
        : shift(shift_), log2C(log2C_), vocab(vocab_),
          mine((unsigned)rank << kLog2Chunk),
          mask(((1u << log2C_) - 1u) << kLog2Chunk) {}
    __device__ __forceinline__ bool has(int id) const {
        return (unsigned)id < (unsigned)vocab &&
               ((unsigned)(id + shift) & mask) == mine;
    }
    __device__ __forceinline__ int element(int id) const {
        const int at = id + shift;
        return (at >> (kLog2Chunk + log2C) << kLog2Chunk) |
               (at & (32 * V - 1));
    }
};

// The bits of a pack's counters that are in use.
template <int V>
__device__ __forceinline__ unsigned in_use(const unsigned *used, int pack) {
    const unsigned byte = reinterpret_cast<const uint8_t *>(used)[
        V == 8 ? pack : pack >> 1];
    return V == 8 ? byte : byte >> (pack & 1) * 4 & 15u;
}

// Adds (or ORs) to a word of shared memory where `on`.
template <bool OR>
__device__ __forceinline__ void red_shared(bool on, unsigned at, unsigned v) {
    if (OR)
        asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %0, 0;\n\t"
                     "@p red.shared.or.b32 [%1], %2;\n\t}" ::"r"((unsigned)on),
                     "r"(at), "r"(v) : "memory");
    else
        asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %0, 0;\n\t"
                     "@p red.shared.add.u32 [%1], %2;\n\t}" ::"r"((unsigned)on),
                     "r"(at), "r"(v) : "memory");
}

// Tokens of this CTA that a lane has found and not counted yet.  Few of a
// history's tokens are a CTA's own, so the pass over the history only looks
// and puts them by, each lane in a column of shared memory of its own; they
// are counted when a lane may run out of room, most lanes at work.
constexpr int kRoom = 16;   // entries per lane
constexpr int kLooks = 8;   // ids that a lane looks at between two checks
template <int V>
struct Found {
    unsigned column, top;  // shared addresses: entry j at column + 128 j
    unsigned count, used;  // shared addresses
    Place<V> place;

    // Four ids; `left` of them are there, `prompt` of them the prompt's.  No
    // branches: a history is mostly others' tokens, and a warp's time is the
    // length of this chain.
    __device__ __forceinline__ void look(int4 v, int left, int prompt) {
        if (left < 4) {
            v.w = -1;
            if (left < 3) v.z = -1;
            if (left < 2) v.y = -1;
            if (left < 1) v.x = -1;
        }
        put(v.x, prompt > 0);
        put(v.y, prompt > 1);
        put(v.z, prompt > 2);
        put(v.w, prompt > 3);
    }
    __device__ __forceinline__ void put(int id, bool prompt) {
        asm volatile(
            "{\n\t.reg .pred p;\n\t.reg .b32 t;\n\t"
            "add.s32 t, %1, %2;\n\tand.b32 t, t, %3;\n\t"
            "setp.eq.u32 p, t, %4;\n\tsetp.lt.and.u32 p, %1, %5, p;\n\t"
            "@p st.shared.u32 [%0], %6;\n\t@p add.u32 %0, %0, 128;\n\t}"
            : "+r"(top)
            : "r"(id), "r"(place.shift), "r"(place.mask), "r"(place.mine),
              "r"(place.vocab), "r"((unsigned)id | (prompt ? kPrompt : 0u))
            : "memory");
    }
    // Counts what the lanes of a warp hold.  A counter that is not zero has
    // its bit set already and a prompt token that was seen needs nothing:
    // frequent tokens cost a read instead of atomics on one address.
    __device__ __forceinline__ void drain() {
#pragma unroll 1
        for (unsigned at = column; __any_sync(kFull, at < top); at += 256) {
            // two entries of the lane at a time
            unsigned entry[2], i[2], before[2];
            bool there[2];
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                there[j] = at + 128 * j < top;
                entry[j] = 0;
                if (there[j])
                    asm volatile("ld.shared.u32 %0, [%1];"
                                 : "=r"(entry[j]) : "r"(at + 128 * j)
                                 : "memory");
            }
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                i[j] = (unsigned)place.element((int)(entry[j] & ~kPrompt));
                before[j] = 0;
                if (there[j])
                    asm volatile("ld.volatile.shared.u32 %0, [%1];"
                                 : "=r"(before[j]) : "r"(count + 4 * i[j])
                                 : "memory");
            }
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const bool prompt = entry[j] & kPrompt;
                red_shared<true>(there[j] && before[j] == 0,
                                 used + (i[j] >> 5) * 4, 1u << (i[j] & 31));
                red_shared<true>(there[j] && prompt && !(before[j] & kPrompt),
                                 count + 4 * i[j], kPrompt);
                red_shared<false>(there[j] && !prompt, count + 4 * i[j], 1u);
            }
        }
        top = column;
    }
    // Called by whole warps after at most kLooks ids.
    __device__ __forceinline__ void keep_room() {
        if (__any_sync(kFull, top > column + 128 * (kRoom - kLooks))) drain();
    }
};

// Sum of a token's biases, in the order given (several for one token: rare).
__device__ __noinline__ float several(const float *bias, const int32_t *ids,
                                      int biases, int column) {
    float s = 0.f;
    for (int j = 0; j < biases; ++j)
        if (ids[j] == column) s += bias[j];
    return s;
}

// A touched logit: penalties, then biases.
__device__ __forceinline__ float touched(float z, unsigned m, float rep,
                                         float inv_rep, float freq,
                                         float pres) {
    const unsigned often = m & kCountMask;
    const float f = z > 0.f ? inv_rep : rep;
    z *= (m & (kCountMask | kPrompt)) ? f : 1.f;
    return often ? z - (freq * (float)often + pres) : z;
}

// 2^t: one MUFU operation (2^-inf = 0, NaN stays NaN, results below 2^-126
// flush to zero).
__device__ __forceinline__ float pow2(float t) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(t));
    return r;
}
__device__ __forceinline__ float nanmax3(float a, float b, float c) {
    float r;
    asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}

// AL: every row of x and y starts at a 16-byte boundary and has whole packs.
// Up to 32 values per thread leave registers for two CTAs per SM.
template <typename T, int MODE, int K, bool AL>
__global__ void __launch_bounds__(kMaxThreads,
                                  K * 16 / (int)sizeof(T) <= 32 ? 2 : 1)
    logits_kernel(const Params p) {
    constexpr int V = 16 / (int)sizeof(T);
    extern __shared__ __align__(16) unsigned count[];
    // (max, sum of exponentials about it) of each warp
    __shared__ float2 pairs[kMaxThreads / 32], joined;
    grid_launch_dependents();
    grid_wait_prerequisites();
    const mt_logits_call_t &c = p.c;
    const int C = 1 << p.log2C;
    const int64_t row = blockIdx.x >> p.log2C;
    const int rank = (int)(blockIdx.x & (unsigned)(C - 1));
    const T *x = static_cast<const T *>(c.x) + row * c.x_stride;
    T *y = static_cast<T *>(c.y) + row * c.y_stride;
    const int shift =
        AL ? 0 : (int)((reinterpret_cast<uintptr_t>(x) / sizeof(T)) & (V - 1));
    const int yshift =
        AL ? 0 : (int)((reinterpret_cast<uintptr_t>(y) / sizeof(T)) & (V - 1));
    const int T_ = (int)blockDim.x, tid = (int)threadIdx.x;
    // Local pack tid + k T_ holds the columns from first + k next on.
    const int first =
        ((((tid >> 5) << p.log2C) + rank) * 32 + (tid & 31)) * V - shift;
    const int next = (T_ << p.log2C) * V;

    // Everything that the row needs is asked for before any of it is waited
    // for, what is needed first before the rest: the row's parameters and
    // first tokens, the logits, the mask.  What is computed from them stands
    // behind the counting.
    const float rep = c.repetition ? c.repetition[row] : 1.f;
    const float freq = c.frequency ? c.frequency[row] : 0.f;
    const float pres = c.presence ? c.presence[row] : 0.f;
    const float temp = c.temperature ? c.temperature[row] : 1.f;
    const int length = c.lengths ? c.lengths[row] : c.history;
    const int given = c.prompt_lengths ? c.prompt_lengths[row] : 0;
    const bool marks = c.tokens != nullptr || c.biases > 0;
    const int32_t *ids = c.tokens + row * c.tokens_stride;
    const int quads = c.tokens && p.wide_tokens ? c.history >> 2 : 0;
    // 16-byte loads of tokens, four in flight per thread
    const auto quad = [ids, quads](int q) {
        return q < quads ? reinterpret_cast<const int4 *>(ids)[q]
                         : make_int4(-1, -1, -1, -1);
    };
    int4 v0 = quad(tid), v1 = quad(tid + T_);
    int4 w0 = quad(tid + 2 * T_), w1 = quad(tid + 3 * T_);
    const int32_t *row_bias_ids = c.bias_ids + row * c.biases;
    const float *row_bias = c.bias + row * c.biases;
    const int my_bias_id = tid < c.biases ? row_bias_ids[tid] : -1;
    const float my_bias = tid < c.biases ? row_bias[tid] : 0.f;
    // The CTA's logits; packs that are cut by an end of the row are read
    // value by value.
    Raw<T, V> raw[K];
#pragma unroll
    for (int k = 0; k < K; ++k) {
        const int col = first + k * next;
        if (AL) {
            if (col < c.vocab) raw[k].load(x + col);
            continue;
        }
        raw[k].zero();
        if (col >= 0 && col + V <= c.vocab) {
            raw[k].load(x + col);
        } else if (col + V > 0 && col < c.vocab) {
            for (int e = 0; e < V; ++e)
                if (col + e >= 0 && col + e < c.vocab) {
                    Raw<T, 1> one;
                    one.load(x + col + e);
                    raw[k].w[e * (int)sizeof(T) / 4] |=
                        one.w[0] << (e * (int)sizeof(T) % 4 * 8);
                }
        }
    }
    // The one or two mask bytes of a pack's columns (one where packs start
    // at a multiple of their width).
    const uint8_t *mask =
        c.mask ? reinterpret_cast<const uint8_t *>(c.mask +
                                                   row * c.mask_stride)
               : nullptr;
    unsigned bits0[K], bits1[K];
#pragma unroll
    for (int k = 0; k < K; ++k) {
        const int col = first + k * next;
        const int from = max(col, 0), last = min(col + V, c.vocab) - 1;
        bits0[k] = bits1[k] = ~0u;
        if (AL) {
            if (mask != nullptr && col < c.vocab)
                bits0[k] = __ldg(mask + (col >> 3));
            continue;
        }
        if (mask != nullptr && from <= last) {
            bits0[k] = __ldg(mask + (from >> 3));
            if (shift != 0 && last >> 3 > from >> 3)
                bits1[k] = __ldg(mask + (last >> 3));
        }
    }
    unsigned *used = count + p.packs * V;
    unsigned *found_at = used + p.packs * V / 32;
    float *bias = reinterpret_cast<float *>(found_at + T_ * kRoom);
    int32_t *bias_ids = reinterpret_cast<int32_t *>(bias + c.biases);
    if (marks) {
        for (int i = tid; i < p.packs * V / 4; i += T_)
            reinterpret_cast<uint4 *>(count)[i] = make_uint4(0, 0, 0, 0);
        for (int i = tid; i < p.packs * V / 32; i += T_) used[i] = 0;
        if (tid < c.biases) {
            bias_ids[tid] = my_bias_id;
            bias[tid] = my_bias;
        }
        for (int i = tid + T_; i < c.biases; i += T_) {
            bias_ids[i] = row_bias_ids[i];
            bias[i] = row_bias[i];
        }
        // Clamped, so that the differences below stay in range.
        const int len = min(max(length, 0), c.history);
        const int prompt = min(max(given, 0), c.history);
        // Whole warps go through the history together; what the first ids
        // give is put by before the counters are known to be zero.
        const int lane = tid & 31;
        const Place<V> place(shift, p.log2C, rank, c.vocab);
        const unsigned column = (unsigned)__cvta_generic_to_shared(
            found_at + (tid >> 5) * 32 * kRoom + lane);
        Found<V> found = {column, column,
                          (unsigned)__cvta_generic_to_shared(count),
                          (unsigned)__cvta_generic_to_shared(used), place};
        int q0 = tid - lane;
        if (q0 < quads && q0 * 4 < len) {
            const int at = (q0 + lane) * 4;
            found.look(v0, len - at, prompt - at);
            if (q0 + T_ < quads)
                found.look(v1, len - at - 4 * T_, prompt - at - 4 * T_);
        }
        __syncthreads();
#pragma unroll 1
        for (q0 += 2 * T_; q0 < quads && q0 * 4 < len; q0 += 2 * T_) {
            found.keep_room();
            const int at = (q0 + lane) * 4;
            v0 = w0;
            v1 = w1;
            w0 = quad(q0 + lane + 2 * T_);
            w1 = quad(q0 + lane + 3 * T_);
            found.look(v0, len - at, prompt - at);
            found.look(v1, len - at - 4 * T_, prompt - at - 4 * T_);
        }
#pragma unroll 1
        for (int i0 = quads * 4 + tid - lane; i0 < len; i0 += T_) {
            found.keep_room();
            const int at = i0 + lane;
            found.put(at < len ? ids[at] : -1, at < prompt);
        }
        found.drain();
        // A bias leaves its number in its token's counter; where another one
        // was there before (in any order), the field becomes kSeveral and
        // the pass below adds them up in the order given.
        for (int i = tid; i < c.biases; i += T_) {
            if (place.has(bias_ids[i])) {
                const int j = place.element(bias_ids[i]);
                atomicOr(used + (j >> 5), 1u << (j & 31));
                const unsigned before =
                    atomicOr(count + j, (unsigned)(i + 1) << kBiasShift);
                if ((before >> kBiasShift) & kSeveral)
                    atomicOr(count + j, kSeveral << kBiasShift);
            }
        }
        __syncthreads();
    }

    const float inv_rep = 1.f / rep;
    // 2^-126 .. 2^126: -infinity keeps its sign and is never multiplied by 0
    const float inv_temp =
        temp > 0.f
            ? 1.f / fminf(fmaxf(temp, 1.17549435e-38f), 8.5070592e+37f)
            : 1.f;
    // Bits of the values that lie in the row and that the mask leaves.
    constexpr unsigned kAll = (1u << V) - 1u;
    unsigned keep[K];
#pragma unroll
    for (int k = 0; k < K; ++k) {
        const int col = first + k * next;
        if (AL) {
            keep[k] = col < c.vocab ? bits0[k] >> (col & 7) & kAll : 0u;
            continue;
        }
        const int from = max(col, 0), to = min(col + V, c.vocab);
        keep[k] = ((bits0[k] & 0xffu) | bits1[k] << 8) >> (from & 7) & kAll;
        if (to - from < V)
            keep[k] = from < to
                          ? (keep[k] & ((1u << (to - from)) - 1u))
                                << (from - col)
                          : 0u;
    }
    // Touched logits of the thread's own packs: their new values, FP32, take
    // the place of their counters.  A compact loop: few of them, and code that
    // runs once per CTA costs its fetch.  It picks a pack's value by index
    // from shared memory, where the thread's entries of the history were.
    if (marks) {
        T *own = reinterpret_cast<T *>(found_at) + tid * V;
        constexpr bool kOwn = K * V * (int)sizeof(T) <= 4 * kRoom;
        if (kOwn) {
#pragma unroll
            for (int k = 0; k < K; ++k)
                if (tid + k * T_ < p.packs && in_use<V>(used, tid + k * T_))
                    raw[k].store(own + k * T_ * V);
        }
#pragma unroll 1
        for (int k = 0; k < K; ++k) {
            const int i = (tid + k * T_) * V;
            if (i >= p.packs * V) break;
            unsigned hit = in_use<V>(used, tid + k * T_);
#pragma unroll 1
            while (hit) {
                const int e = __ffs(hit) - 1, col = first + k * next + e;
                hit &= hit - 1;
                const unsigned m = count[i + e];
                float v = touched(to_f(kOwn ? own[k * T_ * V + e] : x[col]),
                                  m, rep, inv_rep, freq, pres);
                const unsigned b = m >> kBiasShift & kSeveral;
                if (b == kSeveral)
                    v += several(bias, bias_ids, c.biases, col);
                else if (b != 0)
                    v += bias[b - 1];
                count[i + e] = __float_as_uint(v);
            }
        }
    }
    // Values before temperature, -infinity where the mask (or the row's end)
    // leaves nothing; packs of which nothing is left are not looked at.
    float2 z[K][V / 2];
    float top = -INFINITY;
#pragma unroll
    for (int k = 0; k < K; ++k) {
        if (keep[k] == 0) continue;
        float *v = &z[k][0].x;
        raw[k].widen(v);
        if (marks) {
            const int i = (tid + k * T_) * V;
            const unsigned hit = in_use<V>(used, tid + k * T_);
            if (hit) {
#pragma unroll
                for (int e = 0; e < V; e += 4) {
                    const float4 n =
                        *reinterpret_cast<const float4 *>(count + i + e);
                    v[e] = hit >> e & 1u ? n.x : v[e];
                    v[e + 1] = hit >> (e + 1) & 1u ? n.y : v[e + 1];
                    v[e + 2] = hit >> (e + 2) & 1u ? n.z : v[e + 2];
                    v[e + 3] = hit >> (e + 3) & 1u ? n.w : v[e + 3];
                }
            }
        }
        if (keep[k] != kAll) {
#pragma unroll
            for (int e = 0; e < V; ++e)
                v[e] = keep[k] >> e & 1u ? v[e] : -INFINITY;
        }
        if (MODE != MT_LOGITS) {
#pragma unroll
            for (int h = 0; h < V / 2; ++h)
                top = nanmax3(top, z[k][h].x, z[k][h].y);
        }
    }
    float mul = inv_temp, sub = 0.f, log_total = 0.f;
    float nothing = -INFINITY;  // what a masked value gives
    if (MODE != MT_LOGITS) {
        // e^((v - w) / temperature) as 2^((v - w) a): the difference is
        // formed first (exact near w), so its error is 4 roundings of the
        // exponent.  The thread's exponentials are taken about its own
        // largest value (about 0 where it has none: all of them are 0).
        const float a = inv_temp * 1.4426950408889634f;
        const float ref = top == -INFINITY ? 0.f : top;
        float2 sums = make_float2(0.f, 0.f);
#pragma unroll
        for (int k = 0; k < K; ++k) {
            if (keep[k] == 0) continue;
#pragma unroll
            for (int h = 0; h < V / 2; ++h) {
                const float2 t = mul2(add2(z[k][h], both(-ref)), both(a));
                const float2 ex = make_float2(pow2(t.x), pow2(t.y));
                sums = add2(sums, ex);
                if (MODE == MT_LOGITS_SOFTMAX) z[k][h] = ex;
            }
        }
        const float sum = sums.x + sums.y;
        // The warp's pair.
        const int lane = tid & 31, warps = T_ >> 5;
        const float wtop = warp_nanmax(top);
        float wsum = top == -INFINITY ? 0.f : sum * pow2((top - wtop) * a);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1)
            wsum += __shfl_xor_sync(kFull, wsum, o);
        if (lane == 0) pairs[tid >> 5] = make_float2(wtop, wsum);
        __syncthreads();
        // The CTA's pair, by every warp in the same order, and then the
        // row's.
        float M, total;
        const auto join = [a, &M, &total](float2 v) {
            M = warp_nanmax(v.x);
            total = v.x == -INFINITY ? 0.f : v.y * pow2((v.x - M) * a);
#pragma unroll
            for (int o = 8; o > 0; o >>= 1)
                total += __shfl_xor_sync(kFull, total, o);
        };
        const float2 none = make_float2(-INFINITY, 0.f);
        join((lane & 15) < warps ? pairs[lane & 15] : none);
        if (C > 1) {
            if (tid == 0) joined = make_float2(M, total);
            cluster_sync();
            join((lane & 15) < C ? ld_cluster2(&joined, (unsigned)lane & 15u)
                                 : none);
        }
        // No CTA may end before all have read its pairs: arrive (with release
        // order behind the reads) here, wait at the end.
        if (C > 1)
            asm volatile("barrier.cluster.arrive.release.aligned;" ::
                             : "memory");
        // Softmax: e^(v - top) e^(top - M) / total; a row with nothing left
        // has total 0 and gives 0.  Log-softmax: (v - M) / temperature -
        // log(total); such a row keeps its -infinities.  A total that is NaN
        // makes the whole row NaN, masked values too.
        if (MODE == MT_LOGITS_SOFTMAX) {
            mul = 0.f;
            if (total != 0.f)
                mul = (top == -INFINITY ? 0.f : pow2((top - M) * a)) / total;
            nothing = 0.f * mul;
        }
        if (total != total) nothing = total;
        if (MODE == MT_LOGITS_LOG_SOFTMAX && total != 0.f) {
            sub = M;
            log_total = logf(total);
        }
    }
#pragma unroll
    for (int k = 0; k < K; ++k) {
        const int col = first + k * next;
        if ((!AL && col + V <= 0) || col >= c.vocab) continue;
        float *v = &z[k][0].x;
        if (keep[k] == 0) {
#pragma unroll
            for (int e = 0; e < V; ++e) v[e] = nothing;
        } else {
#pragma unroll
            for (int h = 0; h < V / 2; ++h) {
                if (MODE == MT_LOGITS_LOG_SOFTMAX)
                    z[k][h] = add2(z[k][h], both(-sub));
                z[k][h] = mul2(z[k][h], both(mul));
                if (MODE == MT_LOGITS_LOG_SOFTMAX)
                    z[k][h] = add2(z[k][h], both(-log_total));
            }
        }
        if (AL || (col >= 0 && col + V <= c.vocab && yshift == shift)) {
            st_vec<T, V>(y + col, v);
        } else {
#pragma unroll
            for (int e = 0; e < V; ++e)
                if (col + e >= 0 && col + e < c.vocab)
                    y[col + e] = from_f<T>(v[e]);
        }
    }
    if (MODE != MT_LOGITS && C > 1)
        asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

template <typename T, int MODE, int K, bool AL>
cudaError_t launch_packs(const Params &p, int threads, cudaStream_t s) {
    constexpr int V = 16 / (int)sizeof(T);
    const mt_logits_call_t &c = p.c;
    const void *k = reinterpret_cast<const void *>(logits_kernel<T, MODE, K, AL>);
    size_t smem = 0;  // a counter and a bit per logit of the slice, biases
    if (c.tokens != nullptr || c.biases > 0)
        smem = (size_t)p.packs * V * 4 + (size_t)p.packs * V / 8 +
               (size_t)c.biases * 8 + (size_t)threads * kRoom * 4;
    cudaError_t e = cudaSuccess;
    if (smem > 40 * 1024 && (e = allow_max_smem(k)) != cudaSuccess) return e;
    const bool cluster = MODE != MT_LOGITS && p.log2C > 0;
    if (cluster && p.log2C > 3 &&
        (e = allow_nonportable_cluster(k)) != cudaSuccess)
        return e;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = 1u << p.log2C;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(c.rows << p.log2C));
    cfg.blockDim = dim3((unsigned)threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = cluster ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, logits_kernel<T, MODE, K, AL>, p);
}

// Slices, packs per thread and threads.
template <typename T, int MODE>
cudaError_t launch_as(const mt_logits_call_t &c, cudaStream_t s) {
    constexpr int V = 16 / (int)sizeof(T);
    constexpr int kMost = 64 / V;  // packs per thread: at most 64 values
    int sms = 0;
    cudaError_t e = current_sm_count(&sms);
    if (e != cudaSuccess) return e;
    // The largest shift that a row of this call can have.
    const bool whole =
        (reinterpret_cast<uintptr_t>(c.x) & 15) == 0 &&
        (c.rows == 1 || c.x_stride * (int64_t)sizeof(T) % 16 == 0);
    const int all = (c.vocab + (whole ? 0 : V - 1) + V - 1) / V;
    const int chunks = (all + 31) / 32;
    const auto packs = [&](int l) {
        return (chunks + (1 << l) - 1) / (1 << l) * 32;
    };
    // Enough CTAs that 512 threads hold their part with 32 values each, and
    // more while the rows leave SMs idle and a CTA keeps 128 threads busy.
    // Softmax: clusters of up to 8; 16 only for rows that 8 CTAs cannot hold
    // with 64 values per thread (BF16 softmax 256x131072: 43 us on 8 CTAs per
    // row, 116 us on 16, of which the device places few at a time).
    const int most = MODE == MT_LOGITS ? 6 : 3;
    int l = 0;
    while (l < most && packs(l) * V > 32 * kMaxThreads) ++l;
    while (packs(l) * V > 64 * kMaxThreads) ++l;
    while (l < most && c.rows << l < 2 * sms && packs(l) > 256) ++l;
    Params p = {c, l, packs(l), 0};
    if (p.c.history == 0) p.c.tokens = nullptr;
    p.wide_tokens = (reinterpret_cast<uintptr_t>(c.tokens) & 15) == 0 &&
                    (c.rows == 1 || c.tokens_stride % 4 == 0);
    // Fewest packs per thread that 512 threads can do with, fewest threads
    // that do with that; more for a long history, which a CTA goes through
    // alone.
    int K = 1;
    while (K < kMost && (int64_t)K * kMaxThreads < p.packs) K *= 2;
    int threads = 64;
    while (threads < kMaxThreads &&
           (threads * K < p.packs || (p.c.tokens && threads * 8 < c.history)))
        threads *= 2;
    const bool aligned =
        whole && c.vocab % V == 0 &&
        (reinterpret_cast<uintptr_t>(c.y) & 15) == 0 &&
        (c.rows == 1 || c.y_stride * (int64_t)sizeof(T) % 16 == 0);
#define MT_LOGITS_CASE(k)                                                    \
    if (K == k)                                                              \
        return aligned ? launch_packs<T, MODE, k, true>(p, threads, s)       \
                       : launch_packs<T, MODE, k, false>(p, threads, s);
    MT_LOGITS_CASE(1)
    MT_LOGITS_CASE(2)
    MT_LOGITS_CASE(4)
    MT_LOGITS_CASE(8)
    if constexpr (kMost >= 16) {
        MT_LOGITS_CASE(16)
    }
#undef MT_LOGITS_CASE
    return cudaErrorInvalidValue;
}

template <typename T>
cudaError_t launch_mode(const mt_logits_call_t &c, cudaStream_t s) {
    switch (c.mode) {
        case MT_LOGITS: return launch_as<T, MT_LOGITS>(c, s);
        case MT_LOGITS_SOFTMAX: return launch_as<T, MT_LOGITS_SOFTMAX>(c, s);
        default: return launch_as<T, MT_LOGITS_LOG_SOFTMAX>(c, s);
    }
}

}  // namespace

#define MT_DEFINE_LOGITS(T, dt)                                              \
    cudaError_t launch_logits_##dt(const mt_logits_call_t &c,                \
                                   cudaStream_t s) {                         \
        return launch_mode<T>(c, s);                                         \
    }

}  // namespace mt

// logits.cu -- a row of logits: penalties for tokens of its history, biases,
// temperature, grammar mask, and the row's softmax or log-softmax.
//
// A row is cut into slices, one CTA each.  A CTA counts, for its own slice
// only, the tokens of the row's history in shared memory (integer atomics:
// their order changes nothing), then passes over the slice's logits once.
// Every CTA of a row reads the whole history, from L2 after the first.  For
// the softmax modes the CTAs of a row are a cluster: z stays in shared
// memory as FP32 in the place of the counters, and one exchange of (max,
// sum) through distributed shared memory joins the slices.
//
// Alignment.  Packs of V values start at 16-byte boundaries of x: pack p of
// a row holds columns p V - shift + e, shift being the row's address modulo
// 16 in elements, so only a row's first and last pack can be partial.
#include "mt_decoder.cuh"

namespace mt {
namespace {

// Counter of a token: bit 31 "in the prompt", bits 20..30 the number of its
// first bias + 1, bits 0..19 how often it comes after the prompt.
constexpr unsigned kPrompt = 1u << 31;
constexpr int kBiasShift = 20;
constexpr unsigned kCountMask = (1u << kBiasShift) - 1;
constexpr int kMaxThreads = 512;

struct Params {
    mt_logits_call_t c;
    int32_t slices;  // CTAs per row
    int32_t packs;   // packs per slice
};

template <typename T, int MODE>
__global__ void __launch_bounds__(kMaxThreads)
    logits_kernel(const Params p) {
    constexpr int V = 16 / (int)sizeof(T);
    extern __shared__ __align__(16) unsigned count[];
    __shared__ RedScratch red;
    grid_launch_dependents();
    grid_wait_prerequisites();
    const mt_logits_call_t &c = p.c;
    const int rank = (int)(blockIdx.x % (unsigned)p.slices);
    const int64_t row = blockIdx.x / (unsigned)p.slices;
    const T *x = static_cast<const T *>(c.x) + row * c.x_stride;
    T *y = static_cast<T *>(c.y) + row * c.y_stride;
    const int shift =
        (int)((reinterpret_cast<uintptr_t>(x) / sizeof(T)) & (V - 1));
    const int yshift =
        (int)((reinterpret_cast<uintptr_t>(y) / sizeof(T)) & (V - 1));
    const int all = (c.vocab + shift + V - 1) / V;  // packs of the row
    const int first = rank * p.packs;
    const int n = max(0, min(p.packs, all - first));  // packs of the slice
    const int base = first * V - shift;  // column of the slice's element 0
    const int T_ = (int)blockDim.x, tid = (int)threadIdx.x;
    float *zs = reinterpret_cast<float *>(count);
    float *bias_sum = zs + p.packs * V;
    int *bias_id = reinterpret_cast<int *>(bias_sum + c.biases);

    const bool history = c.tokens != nullptr && c.history > 0;
    const bool marks = history || c.biases > 0;
    if (marks) {
        for (int i = tid; i < n; i += T_) {
#pragma unroll
            for (int w = 0; w < V; w += 4)
                *reinterpret_cast<uint4 *>(count + i * V + w) =
                    make_uint4(0, 0, 0, 0);
        }
        for (int i = tid; i < c.biases; i += T_)
            bias_id[i] = c.bias_ids[row * c.biases + i];
        __syncthreads();
        const unsigned width = (unsigned)(n * V);
        if (history) {
            int len = c.history;
            if (c.lengths) len = min(len, max(0, c.lengths[row]));
            const int prompt = c.prompt_lengths ? c.prompt_lengths[row] : 0;
            const int32_t *ids = c.tokens + row * c.tokens_stride;
            for (int i = tid; i < len; i += T_) {
                const int id = ids[i];
                const unsigned at = (unsigned)id - (unsigned)base;
                if (id >= 0 && id < c.vocab && at < width) {
                    if (i < prompt)
                        atomicOr(count + at, kPrompt);
                    else
                        atomicAdd(count + at, 1u);
                }
            }
        }
        // The first bias of a token adds up all of its biases in order.
        for (int i = tid; i < c.biases; i += T_) {
            const int id = bias_id[i];
            const unsigned at = (unsigned)id - (unsigned)base;
            if (id < 0 || id >= c.vocab || at >= width) continue;
            bool mine = true;
            for (int j = 0; j < i && mine; ++j) mine = bias_id[j] != id;
            if (!mine) continue;
            float b = 0.f;
            for (int j = i; j < c.biases; ++j)
                if (bias_id[j] == id) b += c.bias[row * c.biases + j];
            bias_sum[i] = b;
            atomicOr(count + at, (unsigned)(i + 1) << kBiasShift);
        }
        __syncthreads();
    }
    const float rep = c.repetition ? c.repetition[row] : 1.f;
    const float freq = c.frequency ? c.frequency[row] : 0.f;
    const float pres = c.presence ? c.presence[row] : 0.f;
    const float temp = c.temperature ? c.temperature[row] : 1.f;
    const float inv_temp =
        temp > 0.f ? 1.f / fmaxf(temp, 1.17549435e-38f) : 1.f;
    const uint32_t *mask = c.mask ? c.mask + row * c.mask_stride : nullptr;

    float top = -INFINITY;
    for (int i = tid; i < n; i += T_) {
        const int col = base + i * V;
        const bool whole = col >= 0 && col + V <= c.vocab;
        float z[V];
        if (whole) {
            ld_vec<T, V>(x + col, z);
        } else {
#pragma unroll
            for (int e = 0; e < V; ++e)
                z[e] = col + e >= 0 && col + e < c.vocab ? to_f(x[col + e])
                                                         : -INFINITY;
        }
        if (marks) {
#pragma unroll
            for (int e = 0; e < V; ++e) {
                const unsigned m = count[i * V + e];
                if (m != 0) {
                    const unsigned often = m & kCountMask;
                    const unsigned b = (m >> kBiasShift) & 0x7ffu;
                    if (often != 0 || (m & kPrompt))
                        z[e] = z[e] > 0.f ? z[e] / rep : z[e] * rep;
                    if (often != 0) z[e] -= freq * (float)often + pres;
                    if (b != 0) z[e] += bias_sum[b - 1];
                }
            }
        }
        unsigned bits = ~0u;
        if (mask) {
            // Bits of columns col .. col+V-1 (of a partial pack, those that
            // exist; the row's first columns when col < 0).
            const int from = max(col, 0);
            const int word = from >> 5, last = min(col + V, c.vocab) - 1;
            const unsigned lo = __ldg(mask + word);
            const unsigned hi = last >> 5 > word ? __ldg(mask + word + 1) : 0u;
            bits = __funnelshift_r(lo, hi, from & 31) << (from - col);
        }
#pragma unroll
        for (int e = 0; e < V; ++e)
            z[e] = (bits >> e) & 1u ? z[e] * inv_temp : -INFINITY;
        if (MODE == MT_LOGITS) {
            if (whole && yshift == shift) {
                st_vec<T, V>(y + col, z);
            } else {
#pragma unroll
                for (int e = 0; e < V; ++e)
                    if (col + e >= 0 && col + e < c.vocab)
                        y[col + e] = from_f<T>(z[e]);
            }
        } else {
#pragma unroll
            for (int e = 0; e < V; ++e) {
                if (!whole && (col + e < 0 || col + e >= c.vocab))
                    z[e] = -INFINITY;
                top = nanmax(top, z[e]);
                zs[i * V + e] = z[e];
            }
        }
    }
    if (MODE == MT_LOGITS) return;

    int parity = 0;
    top = row_allreduce<MaxOp>(top, T_, red, parity);
    // A slice of which nothing is left: every e^z is 0.
    const float ref = top == -INFINITY ? 0.f : top;
    float sum = 0.f;
    for (int i = tid; i < n; i += T_) {
#pragma unroll
        for (int e = 0; e < V; ++e) {
            const float ex = exp_shifted(zs[i * V + e] - ref);
            sum += ex;
            if (MODE == MT_LOGITS_SOFTMAX) zs[i * V + e] = ex;
        }
    }
    sum = row_allreduce<SumOp>(sum, T_, red, parity);
    float M = top, total = sum;
    if (p.slices > 1) {
        if (tid == 0) {
            red.cl[0][0] = top;
            red.cl[0][1] = sum;
        }
        cluster_sync();
        M = -INFINITY;
        for (int r = 0; r < p.slices; ++r)
            M = nanmax(M, ld_cluster(&red.cl[0][0], (unsigned)r));
        total = 0.f;
        for (int r = 0; r < p.slices; ++r) {
            const float m = ld_cluster(&red.cl[0][0], (unsigned)r);
            const float s = ld_cluster(&red.cl[0][1], (unsigned)r);
            total += m == -INFINITY ? 0.f : s * exp_shifted(m - M);
        }
        // No CTA ends while another may still read its sums.
        cluster_sync();
    }
    // Softmax: e^(z - top) e^(top - M) / total; a row with nothing left has
    // total 0 and gives 0.  Log-softmax: (z - M) - log(total); such a row
    // keeps its -infinities.
    float mul = 0.f, sub = 0.f, log_total = 0.f;
    if (total != 0.f) {
        mul = (top == M ? 1.f : exp_shifted(top - M)) / total;
        sub = M;
        log_total = logf(total);
    }
    for (int i = tid; i < n; i += T_) {
        const int col = base + i * V;
        float z[V];
#pragma unroll
        for (int e = 0; e < V; ++e) {
            const float v = zs[i * V + e];
            z[e] = MODE == MT_LOGITS_SOFTMAX ? v * mul
                                             : (v - sub) - log_total;
        }
        if (col >= 0 && col + V <= c.vocab && yshift == shift) {
            st_vec<T, V>(y + col, z);
        } else {
#pragma unroll
            for (int e = 0; e < V; ++e)
                if (col + e >= 0 && col + e < c.vocab)
                    y[col + e] = from_f<T>(z[e]);
        }
    }
}

template <typename T, int MODE>
cudaError_t launch_as(const mt_logits_call_t &c, cudaStream_t s) {
    constexpr int V = 16 / (int)sizeof(T);
    int sms = 0;
    cudaError_t e = current_sm_count(&sms);
    if (e != cudaSuccess) return e;
    const int all = (c.vocab + 2 * V - 2) / V;  // with the largest shift
    // Slices: at most 16384 values each (64 KiB of counters, three CTAs per
    // SM), up to 16 CTAs, the largest cluster; more of them while the rows
    // leave SMs idle and a slice keeps 2048 values.
    int slices = 1;
    while (slices < 16 && (all + slices - 1) / slices * V > 16384) slices *= 2;
    while (slices < 16 && c.rows * slices < 2 * sms &&
           (all + slices - 1) / slices * V > 4096)
        slices *= 2;
    Params p = {c, slices, (all + slices - 1) / slices};
    int threads = 64;
    while (threads < kMaxThreads && threads < p.packs) threads *= 2;
    const bool marks = (c.tokens && c.history > 0) || c.biases > 0;
    size_t smem = 0;
    if (MODE != MT_LOGITS || marks)
        smem = (size_t)p.packs * V * 4 + (size_t)c.biases * 8;
    const void *k = reinterpret_cast<const void *>(logits_kernel<T, MODE>);
    if (smem > 48 * 1024)
        if ((e = allow_max_smem(k)) != cudaSuccess) return e;
    if (slices > 8 && MODE != MT_LOGITS)
        if ((e = allow_nonportable_cluster(k)) != cudaSuccess) return e;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)slices;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(c.rows * slices));
    cfg.blockDim = dim3((unsigned)threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = MODE != MT_LOGITS && slices > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, logits_kernel<T, MODE>, p);
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

cudaError_t launch_logits(int dtype, const mt_logits_call_t &c,
                          cudaStream_t s) {
    switch (dtype) {
        case DT_F32: return launch_mode<float>(c, s);
        case DT_F16: return launch_mode<__half>(c, s);
        default: return launch_mode<__nv_bfloat16>(c, s);
    }
}

}  // namespace mt

// mt_decoder_internal.h -- what decoder.cpp (argument checks, choice of
// variants) hands to the kernels of the decoder's row operators.
#pragma once

#include "../../include/mt_decoder.h"
#include "mt_internal.h"

namespace mt {

// SM count of the current device (queried once per device).
cudaError_t current_sm_count(int *out);
// Lets `kernel` take up to kDecoderSmemBytes of dynamic shared memory on the
// current device (set once per device and kernel).
constexpr int kDecoderSmemBytes = 208 * 1024;
cudaError_t allow_max_smem(const void *kernel);

// ---- rotary ----------------------------------------------------------------
struct RotHeads {
    const void *x, *dy;
    void *y;
    const void *w;
    int64_t xt, xh, dt, dh, yt, yh;  // strides in elements
    int32_t heads;
    int32_t groups;  // warps' worth of heads: ceil(heads / heads per warp)
};

// A head is served by L = 1 << log2L lanes; lane l owns the "double packs"
// (slots) l, l+L, ...: two packs of V values that hold V whole pairs.
struct RotArgs {
    RotHeads t[2];
    const void *pos;
    const uint64_t *turns;
    int64_t tokens;
    int32_t pos64;
    int32_t dim;
    int32_t pairs;      // rotary_dim / 2
    int32_t rot_slots;  // slots that are rotated
    int32_t slots;      // all slots of a head
    int32_t log2L;
    int32_t log2S;      // forward: warps that share one token
    float eps, inv_dim, scale;
    float sign;         // +1 forward, -1 backward (transposed rotation)
    // backward with norm: one row of dim partial sums per CTA, the first
    // blocks[0] CTAs serving t[0], the others t[1]
    float *partial;
    int32_t blocks[2];
    int32_t threads;    // per CTA: kRotThreads, or for FP32 kRotBackThreads
};
constexpr int kRotThreads = 256;
constexpr int kRotBackThreads = 384;
constexpr int kRotMaxDim = 512;
// Most CTAs of the backward pass with norm (rows of partial sums): two for
// each SM, as many as are resident at once, and no more than two for each of
// 152.
constexpr int kRotBackBlocks = 304;

// Whether each warp of a token has at most so many groups of heads.
inline bool rotary_fits(const RotArgs &a, int queries, int keys) {
    return a.t[0].groups <= queries << a.log2S &&
           a.t[1].groups <= keys << a.log2S;
}

#define MT_DECLARE_ROTARY(dt)                                                \
    cudaError_t launch_rotary_##dt(const RotArgs &a, int V, int K,           \
                                   bool interleaved, bool norm,              \
                                   cudaStream_t s);                          \
    cudaError_t launch_rotary_backward_##dt(const RotArgs &a, int V, int K,  \
                                            bool interleaved,                \
                                            cudaStream_t s);
MT_DECLARE_ROTARY(f32)
MT_DECLARE_ROTARY(f16)
MT_DECLARE_ROTARY(bf16)
#undef MT_DECLARE_ROTARY
// dweight[t][d] = sum over the tensor's blocks of partial[block][d].
cudaError_t launch_rotary_dweight(const float *partial, int dim,
                                  const int32_t blocks[2], float *dw0,
                                  float *dw1, cudaStream_t s);

// ---- cache -----------------------------------------------------------------
struct CacheArgs {
    uint8_t *codes[2];
    float *scales[2];
    void *rows[2];
    int64_t ts[2], hs[2];  // strides of rows
    const int64_t *slot;
    int64_t tokens, slots;
    int32_t tensors;       // 1 or 2
    int32_t heads, dim, group;
    int32_t int8;
};
// vec: values per lane, 16 or 8; 0: any sizes and addresses.
cudaError_t launch_cache_write(int dtype, const CacheArgs &a, int vec,
                               cudaStream_t s);
cudaError_t launch_cache_read(int dtype, const CacheArgs &a, int vec,
                              cudaStream_t s);
cudaError_t launch_cache_slots(const int32_t *table, int64_t stride,
                               int32_t width, const int32_t *offsets,
                               const int32_t *starts, int32_t sequences,
                               int32_t page, int64_t rows, int64_t *slot,
                               cudaStream_t s);

// ---- logits ----------------------------------------------------------------
// 16 CTAs of 512 threads with 64 values each, less a pack's shift.
constexpr int kLogitsMaxVocab = 524280;
constexpr int kLogitsMaxBias = 1024;
cudaError_t launch_logits_f32(const mt_logits_call_t &c, cudaStream_t s);
cudaError_t launch_logits_f16(const mt_logits_call_t &c, cudaStream_t s);
cudaError_t launch_logits_bf16(const mt_logits_call_t &c, cudaStream_t s);

}  // namespace mt

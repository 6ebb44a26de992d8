// step.cpp -- C entry points of the operators around a decoder's cache: pages
// of a step, attention over the cache, the norms around a block.  Argument
// checks and choice of kernel variants.
#include <math.h>
#include <stdint.h>

#include "mt_decoder_checks.h"
#include "mt_decoder_internal.h"

namespace mt {
namespace {

// ---- attention -------------------------------------------------------------
mt_status attention_setup(int dtype, const mt_attention_call_t *c,
                          bool *empty) {
    if (c == nullptr || !known_dtype(dtype)) return MT_ERR_INVALID_ARGUMENT;
    const int es = dtype_size(dtype);
    if (c->rows < 0 || c->slots < 0 || c->sequences < 0 || c->pages < 0 ||
        c->page_size < 1 || c->k_heads < 1 || c->q_heads < 1 ||
        c->q_heads % c->k_heads != 0 || c->dim < 1 || c->group < 1 ||
        c->dim % c->group != 0 || c->window < 0 || c->reserved != 0 ||
        (c->format != MT_CACHE_E4M3 && c->format != MT_CACHE_INT8) ||
        !isfinite(c->scale) || !(c->cap >= 0.f) || !isfinite(c->cap) ||
        (c->cap > 0.f && !isfinite(c->scale / c->cap * 4.f)) ||
        c->table_stride < 0)
        return MT_ERR_INVALID_ARGUMENT;
    if (c->dim > kAttentionMaxDim || c->q_heads > 65536 ||
        c->rows > INT32_MAX)
        return MT_ERR_UNSUPPORTED;
    if (misaligned(c->q, es) || misaligned(c->out, es) ||
        misaligned(c->lse, 4) || misaligned(c->k_scales, 4) ||
        misaligned(c->v_scales, 4) || misaligned(c->table, 4) ||
        misaligned(c->offsets, 4) || misaligned(c->starts, 4) ||
        misaligned(c->first, 4) || misaligned(c->last, 4) ||
        misaligned(c->slopes, 4))
        return MT_ERR_INVALID_ARGUMENT;
    const int64_t width = (int64_t)c->k_heads * c->dim;
    if (c->slots > kMaxOffset / width ||
        (c->sequences > 1 && c->table_stride > kMaxOffset / c->sequences))
        return MT_ERR_INVALID_ARGUMENT;
    if (!reachable(c->q_row, c->q_head, c->rows, c->q_heads) ||
        !reachable(c->out_row, c->out_head, c->rows, c->q_heads) ||
        (c->rows > 0 &&
         !disjoint(c->out_row, c->out_head, c->rows, c->q_heads, c->dim)))
        return MT_ERR_INVALID_ARGUMENT;
    *empty = c->rows == 0 || c->sequences == 0;
    if (*empty) return MT_OK;
    const bool keys = c->slots > 0 && c->pages > 0;
    // other tiles' rows of q may be read after a tile is written
    if (!c->q || !c->out || c->out == c->q || !c->offsets || !c->starts ||
        (keys && (!c->k_codes || !c->v_codes || !c->k_scales ||
                  !c->v_scales || !c->table)))
        return MT_ERR_INVALID_ARGUMENT;
    return MT_OK;
}

// The sizes that the matrix kernels take (on any device): those they are built
// for, each of which is a kernel of its own for either format and both numbers of
// parts.  Other sizes are right and slow (128 in one group, 64 sequences to 16384
// keys, 0.2 ms; 112 on the general kernel 60).
bool attention_head(const mt_attention_call_t &c) {
    const int groups = c.dim / c.group;
    switch (c.dim) {
        case 64: return groups <= 2;
        case 80: case 96: return groups == 1;
        case 128: return groups == 1 || groups == 2 || groups == 4;
        case 256: return groups == 1 || groups == 2 || groups == 8;
        default: return false;
    }
}
constexpr int64_t kManyColumns = 48, kTensorColumns = 256;
// Whether the call goes to the matrix kernels, and how: else a warp per row
// and query head.
mt_status attention_plan(int dtype, const mt_attention_call_t &c, bool *matrix,
                         AttentionPlan *p) {
    *matrix = attention_head(c) && c.slots > 0 && c.pages > 0 &&
              c.slots <= INT32_MAX &&
              !misaligned(c.k_codes, 32) && !misaligned(c.v_codes, 32) &&
              !misaligned(c.k_scales, 16) && !misaligned(c.v_scales, 16);
    if (!*matrix)
        return c.rows * c.q_heads <= (int64_t)INT32_MAX * kAttentionAnyWarps
                   ? MT_OK : MT_ERR_UNSUPPORTED;
    int sms = 0;
    if (cudaError_t e = current_sm_count(&sms)) return status_from_cuda(e);
    p->times = c.q_heads / c.k_heads;
    // Columns that a sequence has on average.  BF16 with one group a head from
    // 256 on: tiles of 128 on tensor memory (at 304 columns 61 us for 71, at 482
    // 75 for 97, at 1930 175 for 308; at 190 56 for 49).  From 48 on the kernel for many rows,
    // which fills tiles of 64 (34 us for 41 at 132 columns, 73 for 66 at 34);
    // else tiles of 16 where there are more than 8.  An average over all rows that
    // q has, since the host does not know the batch: a batch of unlike sequences
    // goes by the middle (a prompt of 2048 rows 221 us, 63 tokens 60, both 398),
    // and rows of q outside the batch count too (8 tokens 20 us, in a q of 256
    // rows 27, of 512 and more 35).
    const int64_t columns_all = (int64_t)p->times * c.rows;
    const bool many = c.dim <= 128 && c.dim % 32 == 0 &&
                      columns_all >= kManyColumns * (int64_t)c.sequences;
    const bool tensor = dtype == DT_BF16 && c.group == c.dim &&
                        (c.dim == 64 || c.dim == 128) &&
                        columns_all >= kTensorColumns * (int64_t)c.sequences;
    p->nt = tensor ? -1
            : many ? 0
            : c.dim <= 128 && columns_all > 8LL * c.sequences ? 2 : 1;
    const int columns = tensor ? 128 : many ? 64 : 8 * p->nt;
    p->per = p->times < columns ? columns / p->times : 1;
    p->parts = (p->times + columns - 1) / columns;
    p->heads = many ? 1 : c.k_heads % 4 == 0 ? 4 : c.k_heads % 2 == 0 ? 2 : 1;
    const int es = dtype_size(dtype);
    const auto fours = [&](const void *q, int64_t row, int64_t head) {
        const uint64_t bits =
            (uint64_t)(reinterpret_cast<uintptr_t>(q) / es) |
            (c.rows > 1 ? (uint64_t)row : 0) |
            (c.q_heads > 1 ? (uint64_t)head : 0);
        return (bits & 3) == 0;
    };
    p->whole = (fours(c.q, c.q_row, c.q_head) ? 1 : 0) |
               (fours(c.out, c.out_row, c.out_head) ? 2 : 0);
    // as many as are resident at once
    const int halves = dtype == DT_BF16 ? 1 : 2;
    p->ctas = sms * (tensor ? 2
                     : many ? attention_row_ctas(c.dim, c.dim / c.group, halves)
                          : attention_ctas(c.dim, c.dim / c.group, halves,
                                           p->nt));
    if (p->ctas > kAttentionMaxCtas) p->ctas = kAttentionMaxCtas;
    return MT_OK;
}
size_t attention_workspace(const mt_attention_call_t &c,
                           const AttentionPlan &p) {
    const size_t columns = p.nt < 0    ? 128
                           : p.nt == 0 ? 64 : 4 * 8 * (size_t)p.nt;
    return (size_t)p.ctas * (2 * columns * (c.dim + 2) * sizeof(float) +
                             kAttentionRecord);
}

// ---- norms around a block ----------------------------------------------------
// A matrix of a call: wanted or not, aligned, rows that are within reach and,
// for an output, do not overlap.
bool matrix_ok(const void *p, int64_t stride, int64_t rows, int64_t cols,
               int es, bool output) {
    int64_t extent = cols;
    return !misaligned(p, es) && add_extent(stride, rows, &extent) &&
           (!output || rows <= 1 || stride >= cols);
}
bool norm_sizes_ok(int dtype, int64_t rows, int64_t cols, int norms, float eps,
                   float scale) {
    return known_dtype(dtype) && rows >= 0 && cols >= 1 && norms >= 1 &&
           norms <= (MT_NORM_AFTER | MT_NORM_BEFORE) && eps >= 0.f &&
           isfinite(scale);
}

// Values of a row that every access can take at once: the widest pack that
// fits all rows' addresses and divides the row.
struct Widest {
    int es;
    int64_t rows;
    uint64_t bits;
    void add(const void *p, int64_t stride) {
        bits |= (uint64_t)(reinterpret_cast<uintptr_t>(p) / es);
        if (p && rows > 1) bits |= (uint64_t)stride;
    }
    int values() const { return widest(bits, 16 / es); }
};

// A row of partial sums for each CTA, of which there are no more than rows.
size_t norm_workspace(const mt_block_norm_back_t &c) {
    if (!c.dgate_sum && !c.dweight && !c.dnext_weight) return 0;
    const int64_t most = norm_back_blocks(c.cols);
    return (size_t)(c.rows < most ? c.rows : most) * 3 * (size_t)c.cols *
           sizeof(float);
}

// Whether no output of the call is one of its inputs or another output (those
// without a value are no matter).
bool apart(const mt_cache_extend_call_t &c) {
    const void *in[] = {c.sequences > 0 ? c.lengths : nullptr,
                        c.sequences > 0 ? c.counts : nullptr,
                        c.free_size > 0 ? c.free_pages : nullptr,
                        c.free_count};
    const void *out[] = {c.offsets, c.new_free_count,
                         c.sequences > 0 ? c.new_lengths : nullptr,
                         c.rows > 0 ? c.slots : nullptr,
                         c.rows > 0 ? c.positions : nullptr,
                         c.sequences > 0 && c.pages > 0 ? c.table : nullptr};
    constexpr int kOut = sizeof(out) / sizeof(out[0]);
    for (int i = 0; i < kOut; ++i) {
        if (out[i] == nullptr) continue;
        for (const void *p : in)
            if (p == out[i]) return false;
        for (int j = 0; j < i; ++j)
            if (out[j] == out[i]) return false;
    }
    return true;
}

}  // namespace
}  // namespace mt

using namespace mt;

extern "C" {

mt_status mt_cache_extend(const mt_cache_extend_call_t *call,
                          mt_stream_t stream) {
    if (call == nullptr) return MT_ERR_INVALID_ARGUMENT;
    const mt_cache_extend_call_t &c = *call;
    if (c.rows < 0 || c.pages < 0 || c.sequences < 0 || c.free_size < 0 ||
        c.page_size < 1 || c.table_stride < 0 ||
        (c.sequences > 1 && (c.table_stride < c.pages ||
                             c.table_stride > kMaxOffset / c.sequences)) ||
        misaligned(c.table, 4) || misaligned(c.lengths, 4) ||
        misaligned(c.counts, 4) || misaligned(c.free_pages, 4) ||
        misaligned(c.free_count, 4) || misaligned(c.offsets, 4) ||
        misaligned(c.slots, 8) || misaligned(c.positions, 4) ||
        misaligned(c.new_lengths, 4) || misaligned(c.new_free_count, 4))
        return MT_ERR_INVALID_ARGUMENT;
    if (!c.free_count || !c.offsets || !c.new_free_count ||
        (c.free_size > 0 && !c.free_pages) ||
        (c.rows > 0 && (!c.slots || !c.positions)) ||
        (c.sequences > 0 && (!c.lengths || !c.counts || !c.new_lengths ||
                             (c.pages > 0 && !c.table))) ||
        !apart(c))
        return MT_ERR_INVALID_ARGUMENT;
    if (c.rows > INT32_MAX || c.sequences == INT32_MAX ||
        c.free_size == INT32_MAX)
        return MT_ERR_UNSUPPORTED;
    return status_from_cuda(launch_cache_extend(c, (cudaStream_t)stream));
}

mt_status mt_cache_attention_workspace(int dtype,
                                       const mt_attention_call_t *call,
                                       size_t *bytes) {
    bool empty = false;
    if (bytes == nullptr) return MT_ERR_INVALID_ARGUMENT;
    if (mt_status st = attention_setup(dtype, call, &empty)) return st;
    *bytes = 0;
    bool matrix = false;
    AttentionPlan p = {};
    if (empty) return MT_OK;
    if (mt_status st = attention_plan(dtype, *call, &matrix, &p)) return st;
    if (matrix) *bytes = attention_workspace(*call, p);
    return MT_OK;
}

mt_status mt_cache_attention(int dtype, const mt_attention_call_t *call,
                             void *workspace, size_t workspace_bytes,
                             mt_stream_t stream) {
    bool empty = false;
    if (mt_status st = attention_setup(dtype, call, &empty)) return st;
    if (empty) return MT_OK;
    bool matrix = false;
    AttentionPlan p = {};
    if (mt_status st = attention_plan(dtype, *call, &matrix, &p)) return st;
    cudaStream_t s = (cudaStream_t)stream;
    if (!matrix)
        return status_from_cuda(launch_attention_any(dtype, *call, s));
    if (workspace_bytes < attention_workspace(*call, p))
        return MT_ERR_OUT_OF_RESOURCES;
    if (workspace == nullptr || misaligned(workspace, 16))
        return MT_ERR_INVALID_ARGUMENT;
    const bool int8 = call->format == MT_CACHE_INT8;
    const auto launch =
        p.nt < 0 ? (int8 ? launch_attention_tiles_int8
                         : launch_attention_tiles_e4m3)
        : p.nt == 0
            ? (dtype == DT_BF16 ? int8 ? launch_attention_rows_int8_p1
                                       : launch_attention_rows_e4m3_p1
                                : int8 ? launch_attention_rows_int8_p2
                                       : launch_attention_rows_e4m3_p2)
        : dtype == DT_BF16
            ? (int8 ? p.nt == 2 ? launch_attention_int8_p1n2
                                : launch_attention_int8_p1n1
                    : p.nt == 2 ? launch_attention_e4m3_p1n2
                                : launch_attention_e4m3_p1n1)
            : (int8 ? p.nt == 2 ? launch_attention_int8_p2n2
                                : launch_attention_int8_p2n1
                    : p.nt == 2 ? launch_attention_e4m3_p2n2
                                : launch_attention_e4m3_p2n1);
    return status_from_cuda(launch(p, *call, dtype, workspace, s));
}

mt_status mt_block_norm(int dtype, const mt_block_norm_call_t *call,
                        mt_stream_t stream) {
    if (call == nullptr) return MT_ERR_INVALID_ARGUMENT;
    const mt_block_norm_call_t &c = *call;
    if (!norm_sizes_ok(dtype, c.rows, c.cols, c.norms, c.eps,
                       c.residual_scale))
        return MT_ERR_INVALID_ARGUMENT;
    if (c.cols > kNormMaxCols || c.rows > INT32_MAX)
        return MT_ERR_UNSUPPORTED;
    const int es = dtype_size(dtype);
    const bool before = c.norms & MT_NORM_BEFORE;
    if (!matrix_ok(c.x, c.x_stride, c.rows, c.cols, es, false) ||
        !matrix_ok(c.residual, c.residual_stride, c.rows, c.cols, es, false) ||
        !matrix_ok(c.gate, c.gate_stride, c.rows, c.cols, es, false) ||
        !matrix_ok(c.h, c.h_stride, c.rows, c.cols, es, true) ||
        (before && !matrix_ok(c.y, c.y_stride, c.rows, c.cols, es, true)) ||
        misaligned(c.weight, es) || misaligned(c.next_weight, es) ||
        (!(c.norms & MT_NORM_AFTER) && c.weight) ||
        (!before && (c.next_weight || c.y)))
        return MT_ERR_INVALID_ARGUMENT;
    if (c.rows == 0) return MT_OK;
    if (!c.x || !c.residual || !c.h || (before && !c.y) || c.h == c.y)
        return MT_ERR_INVALID_ARGUMENT;
    cudaStream_t s = (cudaStream_t)stream;
    Widest w{es, c.rows, (uint64_t)c.cols};
    w.add(c.x, c.x_stride);
    w.add(c.residual, c.residual_stride);
    w.add(c.gate, c.gate_stride);
    w.add(c.h, c.h_stride);
    w.add(c.y, c.y_stride);
    w.add(c.weight, 0);
    w.add(c.next_weight, 0);
    return status_from_cuda(
        dtype == DT_F32   ? launch_block_norm_f32(c, w.values(), s)
        : dtype == DT_F16 ? launch_block_norm_f16(c, w.values(), s)
                          : launch_block_norm_bf16(c, w.values(), s));
}

mt_status mt_block_norm_backward_workspace(int dtype,
                                           const mt_block_norm_back_t *call,
                                           size_t *bytes) {
    if (call == nullptr || bytes == nullptr ||
        !norm_sizes_ok(dtype, call->rows, call->cols, call->norms, call->eps,
                       call->residual_scale))
        return MT_ERR_INVALID_ARGUMENT;
    if (call->cols > kNormMaxCols || call->rows > INT32_MAX)
        return MT_ERR_UNSUPPORTED;
    *bytes = norm_workspace(*call);
    return MT_OK;
}

mt_status mt_block_norm_backward(int dtype, const mt_block_norm_back_t *call,
                                 void *workspace, size_t workspace_bytes,
                                 mt_stream_t stream) {
    if (call == nullptr) return MT_ERR_INVALID_ARGUMENT;
    const mt_block_norm_back_t &c = *call;
    if (!norm_sizes_ok(dtype, c.rows, c.cols, c.norms, c.eps,
                       c.residual_scale))
        return MT_ERR_INVALID_ARGUMENT;
    if (c.cols > kNormMaxCols || c.rows > INT32_MAX)
        return MT_ERR_UNSUPPORTED;
    const int es = dtype_size(dtype);
    const bool before = c.norms & MT_NORM_BEFORE;
    const bool after = c.norms & MT_NORM_AFTER;
    const auto in = [&](const void *p, int64_t stride) {
        return matrix_ok(p, stride, c.rows, c.cols, es, false);
    };
    const auto out = [&](const void *p, int64_t stride) {
        return p == nullptr || matrix_ok(p, stride, c.rows, c.cols, es, true);
    };
    if (!in(c.dy, c.dy_stride) || !in(c.dh, c.dh_stride) ||
        !in(c.x, c.x_stride) || !in(c.h, c.h_stride) ||
        !in(c.gate, c.gate_stride) || !out(c.dx, c.dx_stride) ||
        !out(c.dresidual, c.dresidual_stride) ||
        !out(c.dgate, c.dgate_stride) || misaligned(c.weight, es) ||
        misaligned(c.next_weight, es) || misaligned(c.dgate_sum, 4) ||
        misaligned(c.dweight, 4) || misaligned(c.dnext_weight, 4))
        return MT_ERR_INVALID_ARGUMENT;
    // What a call without a norm, or without a gate, does not take.
    if ((!before && (c.dy || c.h || c.next_weight || c.dnext_weight)) ||
        (!after && (c.weight || c.dweight)) ||
        (!c.gate && (c.dgate || c.dgate_sum)) || (c.dgate && c.dgate_sum))
        return MT_ERR_INVALID_ARGUMENT;
    cudaStream_t s = (cudaStream_t)stream;
    float *sums[3] = {c.dgate_sum, c.dweight, c.dnext_weight};
    const size_t need = norm_workspace(c);
    if (c.rows == 0) {  // sums over no rows
        for (float *d : sums)
            if (d) {
                cudaError_t e =
                    cudaMemsetAsync(d, 0, c.cols * sizeof(float), s);
                if (e != cudaSuccess) return status_from_cuda(e);
            }
        return MT_OK;
    }
    if (!c.dx || !c.dresidual || c.dx == c.dresidual ||
        (c.dgate && (c.dgate == c.dx || c.dgate == c.dresidual)) ||
        (before && (!c.dy || !c.h)) || (!before && !c.dh) ||
        ((after || c.dgate || c.dgate_sum) && !c.x))
        return MT_ERR_INVALID_ARGUMENT;
    if (workspace_bytes < need) return MT_ERR_OUT_OF_RESOURCES;
    if (need > 0 && (workspace == nullptr || misaligned(workspace, 16)))
        return MT_ERR_INVALID_ARGUMENT;
    float *partial = need > 0 ? static_cast<float *>(workspace) : nullptr;
    int blocks = 0;
    Widest w{es, c.rows, (uint64_t)c.cols};
    w.add(c.dy, c.dy_stride);
    w.add(c.dh, c.dh_stride);
    w.add(c.x, c.x_stride);
    w.add(c.h, c.h_stride);
    w.add(c.gate, c.gate_stride);
    w.add(c.dx, c.dx_stride);
    w.add(c.dresidual, c.dresidual_stride);
    w.add(c.dgate, c.dgate_stride);
    w.add(c.weight, 0);
    w.add(c.next_weight, 0);
    const int V = w.values();
    cudaError_t e =
        dtype == DT_F32
            ? launch_block_norm_back_f32(c, V, partial, &blocks, s)
        : dtype == DT_F16
            ? launch_block_norm_back_f16(c, V, partial, &blocks, s)
            : launch_block_norm_back_bf16(c, V, partial, &blocks, s);
    if (e == cudaSuccess && need > 0)
        e = launch_norm_sums(partial, c.cols, blocks, sums[0], sums[1],
                             sums[2], s);
    return status_from_cuda(e);
}

}  // extern "C"

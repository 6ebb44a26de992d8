/*
 * mt_decoder.h -- C ABI of the row operators that stand between the matrix
 * products of a decoder's step, next to the per-row reductions of
 * mt_rowreduce.h: rotary positions of query and key heads with the per-head
 * RMSNorm in front of them (forward and backward), the quantised cache
 * (rows of heads reduced to one scale per group and stored as 8-bit codes,
 * and read back), and the logits (penalties, biases, grammar mask and
 * temperature, then the row's softmax or log-softmax in the same pass); and
 * what stands around that cache: the pages of a step's tokens, attention over
 * the cached codes, and the norms behind a block and before the next one with
 * the block's gate and the residual's scale (forward and backward).
 * Plain C; implemented in the same library.
 *
 * Conventions, where they differ from mt_rowreduce.h
 * --------------------------------------------------
 * Layout     heads: value d of head h of token t is at element
 *            t*token_stride + h*head_stride + d of the pointer, so a view
 *            into a fused projection needs no copy.  Strides are in elements
 *            and may be anything for inputs (0 repeats a row); the rows of an
 *            output must not overlap: with more than one token (head), the
 *            absolute token (head) stride must be at least dim, and one of
 *            the two must span the other's rows.
 * Memory     as in mt_rowreduce.h: caller-owned device memory on the current
 *            device, no allocation, no synchronisation, work enqueued on
 *            `stream`.  Calls can be captured into a CUDA graph.
 * Aliasing   an output may be an input exactly (same pointer, same strides).
 *            Any other overlap is undefined.
 * Errors     arguments are checked before anything is enqueued; a violated
 *            rule gives MT_ERR_INVALID_ARGUMENT, a size beyond a stated limit
 *            MT_ERR_UNSUPPORTED, a workspace that is too small
 *            MT_ERR_OUT_OF_RESOURCES.  Calls with nothing to do (no tokens,
 *            no rows, a cache without slots) return MT_OK without a launch
 *            and outputs untouched, except weight gradients, which are set to
 *            zero.
 * Numerics   FP32 arithmetic with one rounding at each output store (half
 *            step, to nearest even); sums run in a fixed order, so the same
 *            call gives the same bits.  No float atomics.  That order goes by
 *            the call's sizes and alignment and the device's SM count: in
 *            another batch, a row's norm or softmax may differ in its last
 *            bits.
 */
#ifndef MT_DECODER_H
#define MT_DECODER_H

#include "mt_rowreduce.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ---- rotary positions ----------------------------------------------------
 * Pair i of a head (of rotary_dim/2 pairs) is turned by the angle
 * p * f_i, p the token's position and f_i the pair's frequency in radians
 * per position:
 *     y_a = s (a cos - b sin),   y_b = s (a sin + b cos).
 * Pair i is (i, i + rotary_dim/2) in the half layout, (2i, 2i+1) in the
 * interleaved one; the values from rotary_dim on pass unrotated (and not
 * scaled by s).  With norm, each head is first normalised,
 * x <- x / sqrt(mean over dim of x^2 + eps) * weight.
 *
 * Angles are exact for positions of any size: a frequency is held as the
 * fraction of a turn that one position adds, in units of 2^-64 turns, and
 * position times that, modulo 2^64, is the angle.  mt_rotary_turns() makes
 * that form from radians. */

/* How frequencies are stretched for contexts longer than the ones that were
 * trained on.  `factor` s >= 1 is the ratio of the lengths. */
typedef enum mt_rotary_scaling_type {
    MT_ROTARY_PLAIN = 0,  /* f_i = base^(-2i/rotary_dim) */
    MT_ROTARY_LINEAR = 1, /* f_i / s */
    /* base replaced by base * s^(rotary_dim/(rotary_dim-2)): the fastest
     * pair keeps its frequency, the slowest is divided by s */
    MT_ROTARY_NTK = 2,
    /* Pairs that make more than `high` turns over original_length positions
     * keep f_i, pairs that make less than `low` turns get f_i / s, with a
     * linear ramp over the pair index between (bounds rounded outwards to
     * whole pairs); values are scaled by 0.1 ln(s) + 1. */
    MT_ROTARY_YARN = 3,
    /* As above with a ramp that is linear in the number of turns
     * n = original_length f_i / 2 pi:
     * f_i (m + (1-m)/s), m = clamp((n - low)/(high - low), 0, 1). */
    MT_ROTARY_BANDS = 4
} mt_rotary_scaling_type;

typedef struct mt_rotary_scaling {
    int32_t type;           /* mt_rotary_scaling_type */
    int32_t reserved;       /* 0 */
    double factor;          /* s >= 1 (ignored by PLAIN) */
    double original_length; /* > 0 (YARN, BANDS) */
    double low, high;       /* turns, 0 < low < high (YARN, BANDS) */
} mt_rotary_scaling_t;

/* Host only.  Writes rotary_dim/2 frequencies (radians per position) and the
 * factor on rotated values.  scaling may be NULL (PLAIN).  rotary_dim even,
 * 2..512 (NTK: at least 4); base > 1. */
MT_API mt_status mt_rotary_frequencies(int32_t rotary_dim, double base,
                                       const mt_rotary_scaling_t *scaling,
                                       double *freqs, double *factor);

/* Host only.  turns[i] = freqs[i] / 2 pi in units of 2^-64 turns, modulo one
 * turn.  freqs of any sign, below 1e6 in magnitude. */
MT_API mt_status mt_rotary_turns(const double *freqs, int32_t n,
                                 uint64_t *turns);

/* The heads of one tensor (queries or keys) in a rotary call. */
typedef struct mt_rotary_heads {
    const void *x;      /* forward: input.  backward with norm: the forward
                           call's input; without norm: NULL */
    const void *dy;     /* backward: gradient of the output.  forward: NULL */
    void *y;            /* forward: output.  backward: gradient of x */
    const void *weight; /* dim values, NULL = ones; without norm NULL */
    float *dweight;     /* backward with norm: dim FP32 values, or NULL (not
                           wanted).  Otherwise NULL */
    int64_t x_token, x_head, dy_token, dy_head, y_token, y_head; /* strides */
    int32_t heads;      /* 0..65536; 0 = the tensor is absent */
    int32_t reserved;   /* 0 */
} mt_rotary_heads_t;

typedef struct mt_rotary_call {
    mt_rotary_heads_t q, k;
    const void *positions;  /* tokens int32 or int64 values, of any sign */
    const uint64_t *turns;  /* DEVICE pointer, rotary_dim/2 values */
    int64_t tokens;         /* 0..2^33 */
    int32_t position_bytes; /* 4 or 8 */
    int32_t dim;            /* values per head, 1..512 */
    int32_t rotary_dim;     /* even, 2..dim */
    int32_t interleaved;    /* 0 half layout, 1 interleaved */
    int32_t norm;           /* 1 = RMSNorm each head first */
    float eps;
    float scale;            /* s: factor on rotated values */
    int32_t reserved;       /* 0 */
} mt_rotary_call_t;

/* Queries and keys in one launch.  dtype: mt_dtype of x, y and weight. */
MT_API mt_status mt_rotary(int dtype, const mt_rotary_call_t *call,
                           mt_stream_t stream);

/* Gradients.  g = s R^T dy on the rotated values.  Without norm dx = g.  With
 * norm, r = 1/sqrt(mean(x^2)+eps):
 *     dx = r (g w - x r^2 mean(g w x)),   dweight = sum over rows of g x r,
 * with r recomputed from x.  dweight needs a workspace of
 * mt_rotary_backward_workspace() bytes (16-byte aligned device memory that
 * nothing else uses until the call's work is done; two captured graphs that
 * may run at the same time need one each); without dweight it may be
 * NULL. */
MT_API mt_status mt_rotary_backward(int dtype, const mt_rotary_call_t *call,
                                    void *workspace, size_t workspace_bytes,
                                    mt_stream_t stream);
MT_API mt_status mt_rotary_backward_workspace(const mt_rotary_call_t *call,
                                              size_t *bytes);

/* ---- quantised cache -------------------------------------------------------
 * A cache tensor holds, for each of `slots` slots, heads x dim codes of one
 * byte (contiguous) and heads x dim/group FP32 scales (contiguous).  A group
 * of `group` consecutive values of a head shares one scale:
 *     scale = max(amax * (1/q), 2^-126),   code = round(x * (1/scale)),
 * amax the group's largest absolute value, q the format's largest code; the
 * value read back is code * scale, within half a step of the format.  A group
 * that holds a NaN or an infinity gets scale NaN and codes 0, and reads back
 * as NaN. */
typedef enum mt_cache_format {
    MT_CACHE_E4M3 = 0, /* 4 exponent, 3 fraction bits, q = 448 */
    MT_CACHE_INT8 = 1  /* two's complement, q = 127 (-128 is not used) */
} mt_cache_format;

typedef struct mt_cache_rows {
    void *codes;    /* slots x heads x dim bytes */
    float *scales;  /* slots x heads x dim/group */
    void *rows;     /* write: the values (read only); read: the output */
    int64_t token_stride, head_stride; /* of rows */
} mt_cache_rows_t;

typedef struct mt_cache_call {
    mt_cache_rows_t k, v;  /* v.codes, v.scales and v.rows NULL: k alone */
    const int64_t *slot;   /* DEVICE: tokens slots.  A token whose slot is
                              negative or >= slots takes no part: nothing is
                              stored for it, and a read leaves its output row
                              as it was. */
    int64_t tokens, slots; /* tokens*heads*dim <= 2^40, or 2^32 where group
                              is not a multiple of 8 */
    int32_t heads;         /* >= 1 */
    int32_t dim;           /* >= 1; heads*dim <= 2^20 */
    int32_t group;         /* divides dim */
    int32_t format;        /* mt_cache_format */
} mt_cache_call_t;

/* Stores the rows of keys and values in one launch.  The slots of a call
 * that lie inside the cache must differ from one another: where two tokens
 * name the same slot, what stands in that slot afterwards is undefined (a
 * mixture of the two; no other slot is touched). */
MT_API mt_status mt_cache_write(int dtype, const mt_cache_call_t *call,
                                mt_stream_t stream);
/* Reads rows back, rounded once to dtype.  Slots may repeat. */
MT_API mt_status mt_cache_read(int dtype, const mt_cache_call_t *call,
                               mt_stream_t stream);

/* Slots of the rows of a packed batch from its page tables.  Rows
 * offsets[s] .. offsets[s+1]-1 belong to sequence s and stand at positions
 * starts[s], starts[s]+1, ... of it; position p is in slot
 * table[s*table_stride + p/page_size] * page_size + p % page_size.  A row
 * behind offsets[sequences], before offsets[0], at a negative position, past
 * the table's width or in a negative page gets slot -1.  offsets (sequences+1
 * values, not decreasing), starts and table are int32 DEVICE arrays; rows at
 * most 2^38. */
MT_API mt_status mt_cache_slots(const int32_t *table, int64_t table_stride,
                                int32_t pages_per_sequence,
                                const int32_t *offsets, const int32_t *starts,
                                int32_t sequences, int32_t page_size,
                                int64_t rows, int64_t *slot,
                                mt_stream_t stream);

/* ---- logits ------------------------------------------------------------------
 * For each row, with every part optional (NULL pointers), in this order:
 *   z = x
 *   token in the row's history:  z = z > 0 ? z / repetition
 *                                          : z * repetition
 *   token c > 0 times in the history after the prompt:
 *                                z -= frequency * c + presence
 *   each of the row's biases:    z += value
 *   z /= temperature             (a temperature that is not > 0 counts as 1,
 *                                one beyond 2^-126 .. 2^126 as the bound)
 *   bit of the mask is 0:        z = -infinity, whatever stood there
 * and y = z, softmax(z) or log_softmax(z).  A row of which nothing is left
 * (every z is -infinity) gives probabilities 0 and log-probabilities
 * -infinity; a NaN that the mask leaves gives a NaN row. */
typedef enum mt_logits_mode {
    MT_LOGITS = 0,
    MT_LOGITS_SOFTMAX = 1,
    MT_LOGITS_LOG_SOFTMAX = 2
} mt_logits_mode;

typedef struct mt_logits_call {
    const void *x;             /* rows x vocab, row stride x_stride */
    void *y;                   /* same type, row stride y_stride >= vocab */
    int64_t rows, x_stride, y_stride; /* rows 0..2^24 */
    int32_t vocab;             /* 1..524280 */
    int32_t mode;              /* mt_logits_mode */
    const int32_t *tokens;     /* rows x history token ids, row stride
                                  tokens_stride; ids outside [0, vocab) are
                                  passed over */
    int64_t tokens_stride;
    int32_t history;           /* ids per row, 0..1048575 */
    int32_t biases;            /* biases per row, 0..1024 */
    const int32_t *lengths;    /* rows: ids of the row that count (NULL: all;
                                  values are clamped to 0..history) */
    const int32_t *prompt_lengths; /* rows: how many of them, from the start,
                                  are the prompt (NULL: none; values are
                                  clamped to 0..history) */
    const float *repetition, *frequency, *presence; /* rows each; repetition
                                  at least 2^-126 */
    const int32_t *bias_ids;   /* rows x biases, contiguous; ids outside
                                  [0, vocab) are passed over; the same id may
                                  come several times: its biases add up in
                                  the order given */
    const float *bias;         /* rows x biases, contiguous */
    const uint32_t *mask;      /* bit v%32 of word v/32 of a row: 1 = allowed;
                                  row stride mask_stride >= (vocab+31)/32
                                  words, or 0 for one mask for all rows */
    int64_t mask_stride;
    const float *temperature;  /* rows */
} mt_logits_call_t;

MT_API mt_status mt_process_logits(int dtype, const mt_logits_call_t *call,
                                   mt_stream_t stream);

/* ---- pages of a step ---------------------------------------------------------
 * A cache of pages of page_size slots is shared by sequences.  Sequence s
 * holds lengths[s] tokens, in the pages that its row of the table names, and
 * is to hold counts[s] more.  It needs
 *     n_s = ceil((lengths + counts) / page_size) - ceil(lengths / page_size)
 * new pages, which are taken from the end of the list of free pages, in the
 * order of the sequences: with e_s = n_0 + .. + n_(s-1), its i-th new page is
 * free_pages[*free_count - 1 - e_s - i], and its row of the table takes them
 * behind the pages that it has.  A sequence whose pages run past the table's
 * width or whose length passes 2^31 - 1 gets none, and counts as n_s = 0; one
 * that needs pages of which not all are left, e_s + n_s > *free_count, gets
 * none either (nor does any after it that needs some).  A sequence that got no
 * pages but needs some keeps its table and length, and its rows get slot -1.
 *
 * Rows offsets[s] .. offsets[s+1]-1 of the step's packed batch are sequence
 * s's new tokens: slots[r] is the slot of row r and positions[r] its position
 * in its sequence (lengths[s], lengths[s]+1, ...); behind the batch -1 and 0.
 * A row whose page is a negative entry gets slot -1.  The table's entries of
 * pages that are not new are read only, and only for the rows that stand in
 * them.  Negative lengths and counts count as 0, *free_count is clamped to
 * 0 .. free_size, and offsets end at 2^31 - 1.  Called again with the same
 * arguments (lengths, free_count), it does the same again. */
typedef struct mt_cache_extend_call {
    int32_t *table;            /* sequences x pages, row stride table_stride;
                                  takes the new pages */
    int64_t table_stride;      /* >= pages with more than one sequence */
    const int32_t *lengths, *counts; /* sequences each */
    const int32_t *free_pages; /* free_size page numbers, >= 0 and different */
    const int32_t *free_count; /* DEVICE: how many of them are free, from the
                                  start of the list */
    int32_t *offsets;          /* sequences + 1 */
    int64_t *slots;            /* rows */
    int32_t *positions;        /* rows */
    int32_t *new_lengths;      /* sequences: lengths + counts, or lengths */
    int32_t *new_free_count;   /* 1 */
    int64_t rows;              /* 0..2^31 - 1 */
    int32_t pages;             /* the table's width, >= 0 */
    int32_t sequences;         /* 0..2^31 - 2 */
    int32_t free_size;         /* 0..2^31 - 2 */
    int32_t page_size;         /* >= 1 */
} mt_cache_extend_call_t;

/* The outputs, and the table, must not be inputs or each other.  With fewer
 * rows than the counts add up to, only so many are written out; the lengths
 * and pages are those of all. */
MT_API mt_status mt_cache_extend(const mt_cache_extend_call_t *call,
                                 mt_stream_t stream);

/* ---- attention over the cache --------------------------------------------------
 * Queries against the keys and values of the quantised cache, where they
 * stand.  Rows offsets[s] .. offsets[s+1]-1 of q belong to sequence s and
 * stand at positions p = starts[s], starts[s]+1, ...; key j of a sequence is
 * in slot table[s*table_stride + j/page_size] * page_size + j % page_size, as
 * in mt_cache_slots.  Query head h reads key head h / (q_heads / k_heads).
 *     z_j = scale (q . k_j)
 *     z_j = cap tanh(z_j / cap)             (cap > 0)
 *     z_j -= slopes[h] |p - j|              (slopes)
 *     o = sum_j softmax(z)_j v_j,   lse = log sum_j exp(z_j)
 * over the keys that the row sees: from 0, or first[row], to p, or last[row],
 * and of those with a window the keys from p - window + 1 on.  Bounds are
 * clamped to the keys that the sequence holds, 0 .. starts[s] + its rows - 1,
 * so first makes a document's mask and last a prefix's; a key without a page
 * (a negative entry, past the table's width or the cache's slots) is not
 * seen.  A row that sees nothing gives zeros, and lse -infinity.  Rows before
 * offsets[0] and from offsets[sequences] on are left as they were.  A query
 * head that holds a NaN or an infinity, and a row that sees a group that reads
 * back as NaN in the values, or in the keys, gives NaN (from a value: in that
 * group alone); what a row does not see has no effect on it.  (The codes of
 * e4m3 that are NaN themselves, which mt_cache_write never stores, must not
 * stand in slots that a row of the sequence sees.) */
typedef struct mt_attention_call {
    const void *q;             /* rows x q_heads x dim */
    void *out;                 /* the same type and shape; not q */
    float *lse;                /* rows x q_heads, contiguous, or NULL */
    int64_t q_row, q_head, out_row, out_head; /* strides in elements */
    const void *k_codes, *v_codes;    /* as in mt_cache_rows_t */
    const float *k_scales, *v_scales;
    const int32_t *table;      /* sequences x pages */
    int64_t table_stride;
    const int32_t *offsets;    /* sequences + 1, not decreasing; clamped to
                                  0 .. rows */
    const int32_t *starts;     /* sequences; a row at a negative position sees
                                  nothing */
    const int32_t *first, *last; /* rows each, or NULL */
    const float *slopes;       /* q_heads, or NULL */
    int64_t rows;              /* 0..2^31 - 1; rows x q_heads to 2^33 - 4 for
                                  heads that no matrix kernel takes */
    int64_t slots;
    int32_t sequences, pages, page_size;
    int32_t q_heads;           /* a multiple of k_heads, at most 65536 */
    int32_t k_heads;           /* >= 1 */
    int32_t dim;               /* 1..512 */
    int32_t group;             /* divides dim */
    int32_t format;            /* mt_cache_format */
    int32_t window;            /* >= 1, or 0: none */
    float scale;               /* finite */
    float cap;                 /* > 0 and finite, as is 4 scale / cap; or 0:
                                  none */
    int32_t reserved;          /* 0 */
} mt_attention_call_t;

/* dtype: mt_dtype of q and out.  The workspace is as in mt_rotary_backward
 * (mt_cache_attention_workspace() bytes, 16-byte aligned; NULL where those
 * are 0); its size goes by the call's sizes and the current device. */
MT_API mt_status mt_cache_attention(int dtype, const mt_attention_call_t *call,
                                    void *workspace, size_t workspace_bytes,
                                    mt_stream_t stream);
MT_API mt_status mt_cache_attention_workspace(int dtype,
                                              const mt_attention_call_t *call,
                                              size_t *bytes);

/* ---- norms around a block ------------------------------------------------------
 * A block's output x joins the residual stream, through a norm of its own and
 * a gate, and the stream goes through the norm before the next block, in one
 * pass over each row:
 *     u = x / sqrt(mean(x^2) + eps) * weight     (MT_NORM_AFTER; else u = x)
 *     h = residual_scale * residual + gate * u
 *     y = h / sqrt(mean(h^2) + eps) * next_weight   (MT_NORM_BEFORE)
 * y is made from h before its rounding.  gate may be NULL (ones). */
enum {
    MT_NORM_AFTER = 1,  /* the norm behind the block */
    MT_NORM_BEFORE = 2  /* the norm before the next one */
};

typedef struct mt_block_norm_call {
    const void *x, *residual;      /* rows x cols */
    const void *gate;              /* rows x cols, row stride 0: one for all
                                      rows; or NULL */
    const void *weight;            /* cols, NULL = ones (MT_NORM_AFTER) */
    const void *next_weight;       /* cols, NULL = ones (MT_NORM_BEFORE) */
    void *h, *y;                   /* rows x cols; y with MT_NORM_BEFORE only */
    int64_t x_stride, residual_stride, gate_stride, h_stride, y_stride;
    int64_t rows;                  /* 0..2^31 - 1 */
    int32_t cols;                  /* 1..2^20 */
    int32_t norms;                 /* MT_NORM_AFTER, MT_NORM_BEFORE or both */
    float eps, residual_scale;
} mt_block_norm_call_t;

/* h and y may be x or residual. */
MT_API mt_status mt_block_norm(int dtype, const mt_block_norm_call_t *call,
                               mt_stream_t stream);

/* Gradients.  dy and dh are those of y and h, h the forward call's output.
 * r1 = 1/sqrt(mean(x^2)+eps), r2 = 1/sqrt(mean(h^2)+eps):
 *     g  = dh + r2 (dy next_weight - h r2^2 mean(dy next_weight h))
 *     dresidual = residual_scale g,   dgate = g u,   e = g gate
 *     dx = r1 (e weight - x r1^2 mean(e weight x))
 *     dweight = sum over rows of e x r1,  dnext_weight = of dy h r2;
 * without a norm g = dh, or dx = e.  A gate of one row for all has its
 * gradient summed over rows in FP32 (dgate_sum); else dgate has the gate's
 * type. */
typedef struct mt_block_norm_back {
    const void *dy;                /* with MT_NORM_BEFORE only */
    const void *dh;                /* NULL: zeros (MT_NORM_BEFORE) */
    const void *x;                 /* MT_NORM_AFTER, or a gate's gradient */
    const void *h;                 /* with MT_NORM_BEFORE only */
    const void *gate, *weight, *next_weight;   /* as in the forward call */
    void *dx, *dresidual;          /* rows x cols */
    void *dgate;                   /* rows x cols, or NULL */
    float *dgate_sum, *dweight, *dnext_weight; /* cols each, or NULL */
    int64_t dy_stride, dh_stride, x_stride, h_stride, gate_stride, dx_stride,
        dresidual_stride, dgate_stride;
    int64_t rows;
    int32_t cols, norms;
    float eps, residual_scale;
} mt_block_norm_back_t;

/* dx, dresidual and dgate may be dy, dh, x, h or gate exactly (each at most
 * one of them).  The workspace is as in mt_rotary_backward: needed for
 * dgate_sum, dweight and dnext_weight. */
MT_API mt_status mt_block_norm_backward(int dtype,
                                        const mt_block_norm_back_t *call,
                                        void *workspace,
                                        size_t workspace_bytes,
                                        mt_stream_t stream);
MT_API mt_status mt_block_norm_backward_workspace(
    int dtype, const mt_block_norm_back_t *call, size_t *bytes);

#ifdef __cplusplus
}
#endif

#endif /* MT_DECODER_H */

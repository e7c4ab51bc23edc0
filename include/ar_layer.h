/*
 * ar_layer.h -- C ABI of libar's operators around the collectives of a
 * tensor-parallel step: the sum of n ranks' partial results with the residual
 * and an RMS norm (ar_reduce_norm), the embedding lookup from a table split by
 * vocabulary entries over the ranks (ar_embedding), each with its gradient,
 * and the global gradient norm with clipping (ar_grad_norm, ar_clip_grads).
 * Every rank is a buffer in one MI355X's HBM; what every rank would hold alike
 * (the residual stream, a norm's result, looked-up rows) is held once.
 *
 * Reduction, residual, norm (ar_reduce_norm), per row of `width` columns:
 *   s     = residual + sum_r partial_r          (rank after rank, fp32)
 *   rstd  = 1 / sqrt(mean(s^2) + eps)
 *   y_c   = s_c * rstd * (offset + weight_c)
 *   out, summed   y and s rounded to the storage type (y from the unrounded s)
 *   out8, scales  e4m3 (OCP: largest value 448) of y / scale, y and the quotient
 *                 being fp32 numbers, rounded to nearest even, with
 *                 scale = max |y| / 448, but 2^-100 at least, over
 *                 the row (group 0) or over every `group` columns (the last
 *                 group may be short); where some |y| is not finite, scale and
 *                 the group's values are NaN
 * Its gradient (ar_reduce_norm_backward): with x the stored s, h = x * rstd, u = grad_out * (offset + weight),
 *   grad_x      = rstd * (u - h * mean(u h)) + grad_summed   (of the residual and of every partial)
 *   grad_weight = sum over the rows of grad_out * h          (fp32; 0 without rows)
 * Squares that leave the range of fp32 are added up in 64 bits; a rstd past it (eps
 * 0, rows of subnormal numbers) is stored as an infinity, y is finite all the same.
 *
 * Embedding (ar_embedding): out[t] = scale * table[token_t], zeros for a token
 * outside [0, V), V = sum of entries ("no token", e.g. -1).  Rank r holds
 * `entries[r]` rows of the table, the ranks' entries following one another in
 * rank order.  Its gradient (ar_embedding_backward), for every entry v of
 * every rank: grad[v] = scale * sum of grad_out[t] over token_t = v, in the
 * order of t within fixed pieces; written for all entries, zeros where there
 * is no token, or, with `accumulate`, added to what the buffer holds (entries
 * without a token are not touched).
 *
 * Gradient norm: norm = scale * sqrt(sum g^2) over all elements of all buffers,
 * added up in 64 bits.  ar_clip_grads also writes out = g * scale * f,
 * f = max_norm / (norm + eps) where that is below 1, else 1, with the norm in 64
 * bits (`norm` may be past fp32, an infinity, where it is not).  Where the norm
 * is NaN, everything is; where a gradient is infinite and max_norm is not, f is
 * 0; an infinite max_norm never clips (f = 1).
 *
 * Arithmetic: fp32 (rstd's root to within a step) and 64 bits as stated; results
 * are rounded once, to nearest even, to the type they are stored in.  Sums are
 * taken in an order fixed by the shape (for the gradient norm: by the list and by
 * which of its buffers adjoin), so equal calls give equal bits.
 *
 * Buffers: arrays of pointers are HOST arrays of DEVICE pointers, read during
 * the call only.  Everything else is a device pointer to contiguous row-major
 * data unless a pitch is given, aligned to its element; the padding between
 * rows is neither read nor written.  Outputs may not overlap one another or an
 * input, except, element for element: `summed` and `out` may each be the
 * residual or a partial whose pitch is the width; `grad_x` may be grad_out,
 * grad_summed, or x at the pitch `width`; `outs[i]` may be the list's buffer i.
 * Buffers at any element alignment and rows of any length run vector kernels.
 * `workspace`: 16-byte aligned, at least the bytes of the matching function;
 * needs no initialisation, means nothing afterwards; calls that may run at the
 * same time need one each.  It may be NULL when the size is 0.
 *
 * Ordering, errors: as ar.h: asynchronous on `stream`, arguments validated
 * before any launch, no device allocation, capturable in HIP graphs.
 * rows == 0 and tokens == 0 return AR_OK without a launch unless there is a
 * gradient to be written as zeros.
 */
#ifndef AR_LAYER_H
#define AR_LAYER_H

#include <stdint.h>

#include "ar.h"

#ifdef __cplusplus
extern "C" {
#endif

#define AR_NORM_WIDTH_MAX 16384      /* most columns of a normalised row */
#define AR_EMBED_WIDTH_MAX 65536     /* most columns of a table */
#define AR_EMBED_ENTRIES_MAX (1 << 20)
#define AR_EMBED_TOKENS_MAX (1 << 28)
#define AR_GRADS_MAX (1 << 20)       /* most buffers of a list */

typedef struct {
    int n;                         /* ranks, 1..AR_MAX_RANKS */
    ar_dtype_t dtype;              /* of partials, residual, summed, out and their gradients: fp32, bf16 or fp16 */
    ar_dtype_t weight_dtype;       /* of the weight: dtype or fp32 */
    long long rows;                /* >= 0, < 2^31 */
    long long width;               /* 1..AR_NORM_WIDTH_MAX */
    const long long *pitches;      /* HOST, n entries >= width, < 2^31: elements between a partial's rows; NULL: the width */
    float eps;                     /* finite, >= 0 */
    float offset;                  /* finite */
    int group;                     /* columns of a scale: 0 (the row), 32, 64, 128, 256 or 512 */
} ar_norm_t;

/* `weight` [width]; optional: `residual` [rows, width], `summed`, `out`
 * [rows, width], `rstd` [rows] fp32, `out8` [rows, width] bytes with `scales`
 * [rows, groups of a row] fp32 (both or neither).  At least one output. */
ar_status_t ar_reduce_norm(const void *const *partials, const ar_norm_t *shape, const void *weight,
                           const void *residual, void *summed, void *out, float *rstd, void *out8, float *scales,
                           hipStream_t stream);

/* Workspace bytes of ar_reduce_norm_backward with `grad_weight`.  Host only. */
ar_status_t ar_norm_workspace(const ar_norm_t *shape, size_t *bytes);

/* `x` [rows, width] (ar_reduce_norm's `summed`, or the one partial), rows
 * `x_pitch` elements apart (0: the width); `rstd` [rows] from ar_reduce_norm;
 * `grad_out`, `grad_x` [rows, width]; optional: `grad_summed` [rows, width],
 * the gradient that reaches `summed` from elsewhere, and `grad_weight` [width]
 * fp32, which alone needs the workspace.  The shape's n and pitches are not used. */
ar_status_t ar_reduce_norm_backward(const void *x, long long x_pitch, const ar_norm_t *shape, const void *weight,
                                    const float *rstd, const void *grad_out, const void *grad_summed, void *grad_x,
                                    float *grad_weight, void *workspace, size_t workspace_bytes, hipStream_t stream);

typedef struct {
    int n;                         /* ranks, 1..AR_MAX_RANKS */
    ar_dtype_t dtype;              /* of the table and its gradient: fp32, bf16 or fp16 */
    ar_dtype_t out_dtype;          /* of the looked-up rows and their gradient: the same choice */
    long long tokens;              /* 0..AR_EMBED_TOKENS_MAX */
    long long width;               /* columns, 1..AR_EMBED_WIDTH_MAX */
    const long long *entries;      /* HOST, n entries >= 0, 1 <= sum <= AR_EMBED_ENTRIES_MAX */
    const long long *pitches;      /* HOST, n entries >= width, < 2^31: elements between a table's rows; NULL: the width */
    const long long *grad_pitches; /* the same for gradient buffers; NULL: the pitches */
    float scale;                   /* finite */
} ar_embed_t;

/* `tables`: n pointers (NULL where entries[r] is 0); `token_ids` [tokens] int64;
 * `out` [tokens, width] of out_dtype. */
ar_status_t ar_embedding(const void *const *tables, const ar_embed_t *shape, const int64_t *token_ids, void *out,
                         hipStream_t stream);

/* Workspace bytes of ar_embedding_backward.  Host only. */
ar_status_t ar_embedding_workspace(const ar_embed_t *shape, size_t *bytes);

/* `grad_out` [tokens, width] of out_dtype; `grads`: n pointers (NULL where entries[r] is 0). */
ar_status_t ar_embedding_backward(const void *grad_out, const ar_embed_t *shape, const int64_t *token_ids,
                                  void *const *grads, int accumulate, void *workspace, size_t workspace_bytes,
                                  hipStream_t stream);

typedef struct {
    long long count;               /* buffers, 0..AR_GRADS_MAX */
    const void *const *bufs;       /* HOST, `count` device pointers (NULL where sizes[i] is 0) */
    const long long *sizes;        /* HOST, elements of each, >= 0, <= 2^40 in all */
    const int *dtypes;             /* HOST, ar_dtype_t of each: fp32, bf16 or fp16 */
} ar_grads_t;

/* Workspace bytes of the two calls below.  Host only. */
ar_status_t ar_grad_workspace(const ar_grads_t *grads, size_t *bytes);

/* `norm` [1] fp32; `scale` finite, > 0. */
ar_status_t ar_grad_norm(const ar_grads_t *grads, float scale, float *norm, void *workspace, size_t workspace_bytes,
                         hipStream_t stream);

/* `outs`: HOST, a device pointer for each buffer, of its size and type;
 * `max_norm` >= 0 or infinite, `eps` finite and >= 0; `norm` [1] fp32. */
ar_status_t ar_clip_grads(const ar_grads_t *grads, void *const *outs, float max_norm, float scale, float eps,
                          float *norm, void *workspace, size_t workspace_bytes, hipStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* AR_LAYER_H */

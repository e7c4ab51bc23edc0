/*
 * ar_vocab.h -- C ABI of libar's reductions over a vocabulary axis that is
 * split over n logical ranks: the log probabilities of given tokens (with
 * entropy and top alternatives) and distillation from a teacher's top logits,
 * each with its gradient.  Every rank is a buffer in one MI355X's HBM.
 *
 * Logits.  Rank r holds, for every row (token position), the logits of
 * widths[r] consecutive vocabulary entries; the ranks' columns follow one
 * another in rank order, V = sum of widths entries in all (the split of a
 * tensor-parallel output layer; ar_layout_shard's bounds for
 * Layout((rows, V), (n,), (1,)) are one such set of widths).  A row of rank r
 * starts pitches[r] elements after the previous one.  Below, x is a logit,
 * T the temperature, z = x / T, p = softmax(z) over all V entries.
 *
 * Log probabilities (ar_logprobs), per row:
 *   logprobs      ln p[target]; 0 for a target outside [0, V) ("no token", e.g. -100)
 *   entropy       -sum_v p_v ln p_v
 *   top_logprobs, top_ids   the top_k largest logits' ln p and ids, largest
 *                 first, equal logits by lowest id; a NaN is ordered as -inf;
 *                 past V entries: -inf and -1
 * Gradient, for upstream gradients gl of logprobs and gh of entropy:
 *   dx_v = 1/T * (gl * ([v = target] - p_v) - gh * p_v * (ln p_v + entropy))
 * (gl counts as 0 in a row without a token).
 *
 * Distillation (ar_distill), per row, from K teacher entries (id i_k, value
 * t_k); entries whose id is outside [0, V) are padding:
 *   AR_TEACHER_RENORM  q = softmax(t / T) over the entries, q_t = 0;
 *   AR_TEACHER_TAIL    the values are log probabilities (at temperature T) out
 *                 of the whole vocabulary: q_k = exp(t_k), and the remaining
 *                 mass q_t = 1 - sum q (0 when below 2^-20, where it is only
 *                 the rounding of the values) is compared with the student's
 *                 mass p_t on all entries that are not listed.
 *   A repeated id adds its entries' probabilities: Q_v = sum of q_k over i_k = v.
 *   loss  sum_v Q_v (ln Q_v - ln p_v) + q_t (ln q_t - ln p_t) over the listed v
 *                 (the Kullback-Leibler divergence; terms with Q_v = 0 are 0)
 *   dx_v  g/T * (Q p_v - Q_v - [v not listed] q_t p_v / p_t),
 *                 Q = sum q + q_t, g the upstream gradient of the row's loss
 *   A row with no entry in [0, V) (renormalised: none above -inf) has loss 0
 *   and gradient 0.
 *
 * Special rows.  Logits of -inf are masked entries (p = 0).  A row of -inf
 * only has no distribution: ln p = -inf, entropy 0, distillation loss +inf,
 * gradients 0.  The lowest finite value is an ordinary number: a row of it is
 * uniform.  A NaN or +inf logit makes the row's results NaN.  A row whose
 * upstream gradients are all 0 gets a zero gradient, whatever its logits.
 *
 * Arithmetic: fp32 throughout (maxima, sums, entropies, gradients); gradients
 * are rounded once, to nearest even, to the logits' type.  Sums are taken in
 * an order fixed by the shape, so equal calls give equal bits.
 *
 * Buffers: ``logits`` and ``grads`` are HOST arrays of n DEVICE pointers
 * (rank r's may be NULL when widths[r] is 0), read during the call only.
 * Everything else is a device pointer to contiguous row-major data, aligned
 * to its element; outputs marked optional may be NULL.  ``grads`` may be the
 * logits themselves (same pointers and pitches, in place); any other overlap
 * of a gradient buffer with logits or another gradient buffer is rejected
 * (buffers that interleave at one pitch, as columns of one wider buffer, do
 * not overlap).  Outputs may not overlap one another or any input.
 * The padding between rows is neither read nor written.
 * ``workspace`` holds partial results of calls with few rows, at least
 * ar_vocab_workspace() bytes, 16-byte aligned; its contents need no
 * initialisation and mean nothing afterwards; calls that may run at the same
 * time need one each.  It may be NULL when the size is 0.
 *
 * Ordering, errors: as ar.h: asynchronous on ``stream``, arguments validated
 * before any launch, no device allocation, capturable in HIP graphs.
 * rows == 0 returns AR_OK without a launch.
 */
#ifndef AR_VOCAB_H
#define AR_VOCAB_H

#include <stdint.h>

#include "ar.h"

#ifdef __cplusplus
extern "C" {
#endif

#define AR_VOCAB_MAX (1 << 20)   /* most vocabulary entries */
#define AR_TOP_MAX 64            /* most top alternatives */
#define AR_TEACHER_MAX 256       /* most teacher entries per row */

typedef enum { AR_TEACHER_RENORM = 0, AR_TEACHER_TAIL = 1 } ar_teacher_t;

typedef struct {
    int n;                         /* ranks, 1..AR_MAX_RANKS */
    ar_dtype_t dtype;              /* fp32, bf16 or fp16 */
    long long rows;                /* >= 0 */
    const long long *widths;       /* HOST, n entries >= 0, 1 <= sum <= AR_VOCAB_MAX */
    const long long *pitches;      /* HOST, n entries >= widths[r], < 2^31; NULL: the widths */
    const long long *grad_pitches; /* the same for gradient buffers; NULL: the pitches */
    float temperature;             /* finite, > 0 */
} ar_vocab_t;

/* Workspace bytes of any call below on ``shape`` with up to ``top_k`` alternatives.  Host only. */
ar_status_t ar_vocab_workspace(const ar_vocab_t *shape, int top_k, size_t *bytes);

/* ``targets`` [rows] int64, ``logprobs`` [rows] fp32; optional: ``entropy``
 * [rows] fp32; with 1 <= top_k <= AR_TOP_MAX ``top_logprobs`` [rows, top_k]
 * fp32 and ``top_ids`` [rows, top_k] int64 (both or neither NULL; NULL with
 * top_k == 0); ``saved`` [rows, 4] fp32 for ar_logprobs_backward: a reference
 * logit m, sum_v exp((x_v - m) / T), the entropy, and 0. */
ar_status_t ar_logprobs(const void *const *logits, const ar_vocab_t *shape, const int64_t *targets, float *logprobs,
                        float *entropy, int top_k, float *top_logprobs, int64_t *top_ids, float *saved,
                        void *workspace, size_t workspace_bytes, hipStream_t stream);

/* ``saved`` from ar_logprobs on the same logits; ``grad_logprobs`` and
 * ``grad_entropy`` [rows] fp32, either NULL for zeros. */
ar_status_t ar_logprobs_backward(const void *const *logits, void *const *grads, const ar_vocab_t *shape,
                                 const int64_t *targets, const float *saved, const float *grad_logprobs,
                                 const float *grad_entropy, hipStream_t stream);

/* ar_logprobs (without alternatives) and ar_logprobs_backward in one call,
 * for upstream gradients known beforehand (cross-entropy with per-row
 * weights).  ``logprobs``, ``entropy`` and ``saved`` are optional. */
ar_status_t ar_logprobs_grad(const void *const *logits, void *const *grads, const ar_vocab_t *shape,
                             const int64_t *targets, const float *grad_logprobs, const float *grad_entropy,
                             float *logprobs, float *entropy, float *saved, void *workspace, size_t workspace_bytes,
                             hipStream_t stream);

/* ``teacher_ids`` [rows, k] int64, ``teacher_values`` [rows, k] fp32,
 * 1 <= k <= AR_TEACHER_MAX; ``loss`` [rows] fp32; optional ``saved``
 * [rows, 4] fp32 for ar_distill_backward: m and the sum as above, and the same
 * two of the unlisted entries alone (AR_TEACHER_RENORM: of all entries again);
 * -inf and 0 in a row without a teacher, whose logits are not summed. */
ar_status_t ar_distill(const void *const *logits, const ar_vocab_t *shape, const int64_t *teacher_ids,
                       const float *teacher_values, int k, ar_teacher_t mode, float *loss, float *saved,
                       void *workspace, size_t workspace_bytes, hipStream_t stream);

/* ``saved`` from ar_distill with the same logits, teacher and mode;
 * ``grad_loss`` [rows] fp32, NULL for ones. */
ar_status_t ar_distill_backward(const void *const *logits, void *const *grads, const ar_vocab_t *shape,
                                const int64_t *teacher_ids, const float *teacher_values, int k, ar_teacher_t mode,
                                const float *saved, const float *grad_loss, hipStream_t stream);

/* ar_distill and ar_distill_backward in one call; ``loss`` and ``saved`` are optional. */
ar_status_t ar_distill_grad(const void *const *logits, void *const *grads, const ar_vocab_t *shape,
                            const int64_t *teacher_ids, const float *teacher_values, int k, ar_teacher_t mode,
                            const float *grad_loss, float *loss, float *saved, void *workspace,
                            size_t workspace_bytes, hipStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* AR_VOCAB_H */

/*
 * dploss.h -- a loss at the end of a model, with the gradient that its backward
 * pass starts from: distillation from a teacher's top logits, beside the cross
 * entropy of the labels.
 *
 * Conventions are those of dpstep.h and dplayer.h: device pointers are the
 * caller's, calls are asynchronous on the caller's stream, never synchronise
 * and never allocate, and return a dp_status.  The same call on the same inputs
 * gives the same bits.
 */
#ifndef DPLOSS_H
#define DPLOSS_H

#include <stddef.h>
#include <stdint.h>
#include <hip/hip_runtime_api.h>

#include "dpstep.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Most rows of a call, and the largest vocabulary. */
#define DPD_MAX_TOKENS (INT64_C(1) << 21)
#define DPD_MAX_VOCAB (INT64_C(1) << 18)
/* Longest list of a teacher's logits. */
#define DPD_MAX_TOP 1024

/* The loss of one row z of `vocab` logits, with the teacher's logits y_k of the
 * tokens id_k, k < top, at the temperature tau:
 *   loss = soft tau^2 KL + hard CE
 *   KL = sum_k p_k (log p_k - log q[id_k])  +  p' (log p' - log q')
 *   q = softmax(z / tau) over the vocabulary
 *   CE = log(sum_v exp(z_v)) - z_label
 * Without totals (total null) the teacher's probabilities are those of its list
 * alone, p_k = exp(y_k / tau) / sum_j exp(y_j / tau), and there is no p'.  With them,
 * total = log(sum of exp(y / tau) over the teacher's whole vocabulary),
 * p_k = exp(y_k / tau - total), and the remaining probability p' = max(0, 1 -
 * sum_k p_k) is compared with what the student gives to all tokens outside the list,
 * q' = sum of q over them (no such term where p' or q' is 0).  Entries whose id lies
 * outside [0, vocab) are padding and not part of the list; an id may occur more than once
 * (each occurrence is a term).  A row whose list is empty has KL = 0, and so, without
 * totals, has one that holds nothing but -infinity (with them its tokens have p_k = 0, and
 * KL = -log q').  A NaN among the teacher's logits of a row makes its loss and its gradient
 * NaN.  A label outside [0, vocab), or labels null, leave CE out.  Statistics and sums are
 * binary32; z and z / tau lie within 2^24 of 0, where its numbers are one apart. */
typedef struct dpd_distill_desc {
    double temperature; /* > 0 */
    double soft, hard;  /* finite */
    double scale;       /* factor of the gradient alone (a loss scale), finite */
    int64_t vocab;      /* 1 .. DPD_MAX_VOCAB */
    int32_t top;        /* 0 .. DPD_MAX_TOP */
    int32_t id_bytes;   /* 4 or 8: ids and labels are int32_t or int64_t */
} dpd_distill_desc;

/* loss[t] for `tokens` rows (binary32; null: not wanted) and, unless dlogits is
 * null,
 *   dlogits[t] = scale * weight[t] * d loss[t] / d z[t]
 * in one reading of the logits (rows longer than the registers hold, and those whose
 * remainder lies far below their greatest logit, are read again).  weight: binary32 factors of the rows (a mask,
 * 1 / rows), null for 1; a row of weight 0 is not read and gets loss 0 and zeros.
 * logits and dlogits: rows of vocab elements of dtype (DP_F32, DP_F16, DP_BF16), ld
 * apart; dlogits may be logits itself with its stride, in place.  teacher: rows
 * of `top` logits of teacher_dtype, ld_teacher apart, and ids beside them, ld_ids
 * apart.  total, labels: one a row, or null. */
dp_status dpd_distill(const dpd_distill_desc* distill, int64_t tokens, dp_dtype dtype, const void* logits, int64_t ld,
                      dp_dtype teacher_dtype, const void* teacher, int64_t ld_teacher, const void* ids, int64_t ld_ids,
                      const float* total, const void* labels, const float* weight, float* loss, void* dlogits,
                      int64_t ld_dlogits, hipStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* DPLOSS_H */

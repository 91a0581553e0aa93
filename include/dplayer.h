/*
 * dplayer.h -- operators of a model's layers around the step of dpstep.h:
 * forwards that read a plan's parameters (DP_ROLE_PARAM), and backwards that
 * write a tensor's gradient straight into the binary32 accumulators
 * (DP_ROLE_ACC) of every replica, as that tensor's part of a micro-step.
 *
 * A gradient that arrives as a dense low-precision buffer costs a buffer, a
 * rounding and a pass of dp_accumulate_all.  The calls here take what the
 * backward pass has in hand instead (token ids and the gradient of the looked
 * up rows, the inputs of a norm, the 8-bit input of a linear layer) and leave
 *   ACC[r] = G_r            (first != 0)
 *   ACC[r] = ACC[r] + G_r   (first == 0)
 * with G_r summed in binary32 in an order that depends on the sizes and the
 * token ids alone, never on timing: the same call on the same inputs gives the
 * same bits.
 *
 * Micro-steps.  The dpl_accumulate_* calls are buckets of one micro-step of
 * every replica, as those of dp_accumulate_all_range are, each covering its
 * tensors whole: they come in any order and on several streams beside that
 * call's buckets, take the same first flag (DP_ERR_INVALID_ARG) and do not
 * overlap them (DP_ERR_STATE); the micro-step is complete once all together
 * cover [0, P).  A tensor whose gradient is a sum of several calls (a table
 * looked up twice, or tied to a linear layer whose input is packed) takes more
 * != 0 in all of them but the last: such a call writes or adds its term and
 * leaves the tensor uncovered, and the next call on it adds.  Every term is a
 * dpl_accumulate_* call: a dense gradient buffer (dp_accumulate_all_range) covers
 * its tensors alone and is refused on one with terms still to come
 * (DP_ERR_STATE).  The caller orders the calls on one tensor.  After the
 * last micro-step the accumulators go on to dp_reduce_replicas(DP_ROLE_ACC)
 * (with one replica and g_bar its accumulator, to dp_grad_stats(scan = 1)).
 *
 * Conventions are those of dpstep.h: device pointers are the caller's, calls
 * are asynchronous on the caller's stream, never synchronise and never
 * allocate (but for the plan's one-time set-up at its first GPU call, which
 * has to come before any graph capture), and return a dp_status.  Plan
 * pointers are read when the call is made: a captured call keeps those bound
 * at capture.  Memory that a call names as workspace is scratch for the length
 * of that call on its stream: calls that may run at the same time, and graphs
 * that may replay at the same time, need a workspace each.  Outputs must not
 * overlap inputs or each other unless a call says so.
 *
 * Rows.  An activation tensor is `tokens` rows of `dim` elements of a dtype
 * (DP_F32, DP_F16, DP_BF16); consecutive rows are `ld` elements apart (ld >=
 * dim; elements between the rows are never written and never change a result).
 * Any size, stride and element-aligned address works.
 */
#ifndef DPLAYER_H
#define DPLAYER_H

#include <stddef.h>
#include <stdint.h>
#include <hip/hip_runtime_api.h>

#include "dpstep.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Most tokens of one call (each replica's). */
#define DPL_MAX_TOKENS (INT64_C(1) << 24)
/* Widest row of the block norms. */
#define DPL_MAX_NORM_DIM 8192
/* Channels that share one scale in the 8-bit activation format. */
#define DPL_GROUP 32

/* ---- embedding ------------------------------------------------------------ */

/* A plan tensor as a table of rows x dim parameters, row-major (its numel is a
 * multiple of dim and has fewer than 2^31 - 1 rows). */
typedef struct dpl_table {
    int32_t tensor;   /* plan tensor */
    int32_t id_bytes; /* 4 or 8: token ids are int32_t or int64_t */
    int64_t dim;      /* elements of a row, >= 1 */
    double scale;     /* factor of every looked-up value, rounded to binary32; finite */
} dpl_table;

/* out[t] = scale * W[ids[t]], t < tokens, with W the tensor's low-precision
 * parameters (DP_ROLE_PARAM), multiplied in binary32 and rounded once to
 * dtype.  An id outside [0, rows) (padding) gives a row of zeros. */
dp_status dpl_embed(dp_plan* plan, const dpl_table* table, int64_t tokens, const void* ids, dp_dtype dtype, void* out,
                    int64_t ld, hipStream_t stream);

/* Bytes of workspace for dpl_accumulate_embed with up to `tokens` tokens a
 * replica (host work only). */
dp_status dpl_embed_workspace(const dp_plan* plan, const dpl_table* table, int64_t tokens, size_t* bytes);

/* The lookup's gradient: G_r[v] = scale * (sum of dy[r][t] over the tokens t
 * with ids[r][t] == v), summed in binary32 and multiplied at the end.  Ids
 * outside [0, rows) are skipped, and with first == 0 the rows without a token
 * are not touched.  ids, dy: host arrays [n_replicas] of device pointers.  The
 * tokens are sorted by id (stably, so the sums have a fixed order), and rows
 * with many tokens are summed in pieces by several workgroups. */
dp_status dpl_accumulate_embed(dp_plan* plan, const dpl_table* table, int64_t tokens, const void* const* ids,
                               dp_dtype dtype, const void* const* dy, int64_t ld, int32_t first, int32_t more,
                               void* workspace, size_t workspace_bytes, hipStream_t stream);

/* ---- norms around a block --------------------------------------------------- */

/* The norms after one block and before the next, with the gate and the scaled
 * residual between them:
 *   u  = N(y) * w_post + b_post        (u = y where post_w < 0)
 *   s  = residual_scale * h + gate * u  (gate = 1 where gate < 0)
 *   x  = N(s) * w_pre + b_pre           (no x where pre_w < 0)
 *   N(v) = (v - mean(v)) / sqrt(mean((v - mean(v))^2) + eps)   centered != 0
 *   N(v) = v / sqrt(mean(v^2) + eps)                           centered == 0
 * over the dim elements of a row, in binary32.  Weights, biases and the gate
 * are plan tensors of dim elements each (a bias only beside its weight); -1
 * where there is none, and no tensor twice. */
typedef struct dpl_norms {
    int32_t post_w, post_b, gate, pre_w, pre_b;
    int32_t centered;
    int64_t dim;           /* 1 .. DPL_MAX_NORM_DIM */
    double eps;            /* > 0 */
    double residual_scale; /* finite */
} dpl_norms;

/* The forward, on `tokens` rows.  s may be h or y themselves (each row is read
 * whole before it is written); x is null exactly where pre_w < 0.  x is
 * computed from s before s is rounded to dtype. */
dp_status dpl_block_norm(dp_plan* plan, const dpl_norms* norms, int64_t tokens, dp_dtype dtype, const void* h,
                         int64_t ld_h, const void* y, int64_t ld_y, void* s, int64_t ld_s, void* x, int64_t ld_x,
                         hipStream_t stream);

/* Bytes of workspace for dpl_accumulate_block_norm with up to `tokens` tokens a
 * replica (host work only). */
dp_status dpl_block_norm_workspace(const dp_plan* plan, const dpl_norms* norms, int64_t tokens, size_t* bytes);

/* One replica's rows for the backward.  ds is the gradient that reaches s
 * along the residual (null: none); x's gradient dx is null exactly where
 * pre_w < 0, and then ds is not null.  dh or dy may be null (not wanted).  y
 * may be null where nothing needs it: no gate, no post norm. */
typedef struct dpl_norm_rows {
    const void* s;
    const void* y;
    const void* dx;
    const void* ds;
    void* dh;
    void* dy;
} dpl_norm_rows;

/* The backward: dh, dy and, for every tensor of norms, its gradient into
 * ACC[r].  The statistics are computed again from s and y as stored.  rows:
 * host array [n_replicas]; all of them have the same pointers null.  ld is the
 * row stride of every one of them. dh may be ds or dx, and dy any of y, dx, ds
 * that is not dh. */
dp_status dpl_accumulate_block_norm(dp_plan* plan, const dpl_norms* norms, int64_t tokens, dp_dtype dtype,
                                    const dpl_norm_rows* rows, int64_t ld, int32_t first, int32_t more,
                                    void* workspace, size_t workspace_bytes, hipStream_t stream);

/* ---- activations in 8 bits --------------------------------------------------- */

/* The format: codes[t][c], one e4m3 byte (OCP FP8: 448 the largest, 0x7f NaN,
 * no infinity) for each element, and scales[t][c / 32], one byte e + 127 for
 * 32 consecutive channels of a row (the last group may be short).  The value
 * is code * 2^e with e the smallest power in [-117, 119] under which the
 * group's largest finite magnitude is at most 448, so that a bf16 holds every
 * value exactly.  Codes are rounded to nearest even: a relative error of at
 * most 2^-4 for magnitudes from 2^-6 * 2^e, and an absolute one of 2^-10 * 2^e
 * below.  Magnitudes beyond 448 * 2^119, which DP_F32 and DP_BF16 rows may hold, are
 * limited to it, an eighth below the largest of them.  An infinity or NaN
 * becomes NaN, so the step's check still finds it.
 * DP_F16 sources are first limited to +-61440, so that an f16 holds the
 * decoded value exactly too.
 *
 * codes: rows of dim bytes, ld_codes apart; scales: rows of ceil(dim / 32)
 * bytes, ld_scales apart. */
dp_status dpl_pack_activations(int64_t tokens, int64_t dim, dp_dtype dtype, const void* x, int64_t ld, void* codes,
                               int64_t ld_codes, void* scales, int64_t ld_scales, hipStream_t stream);
dp_status dpl_unpack_activations(int64_t tokens, int64_t dim, dp_dtype dtype, const void* codes, int64_t ld_codes,
                                 const void* scales, int64_t ld_scales, void* x, int64_t ld, hipStream_t stream);

/* A linear layer's weight as a plan tensor of outputs x inputs elements,
 * row-major, or inputs x outputs with transposed != 0. */
typedef struct dpl_linear {
    int32_t tensor;
    int32_t transposed;
    int64_t inputs, outputs;
} dpl_linear;

/* One replica's operands: the packed input of the layer, [tokens][inputs], and
 * the gradient of its output, [tokens][outputs]. */
typedef struct dpl_linear_rows {
    const void* codes;
    const void* scales;
    const void* dy;
} dpl_linear_rows;

/* Bytes of workspace for dpl_accumulate_linear with up to `tokens` tokens a
 * replica (host work only; may be 0, at most 64 MiB). */
dp_status dpl_linear_workspace(const dp_plan* plan, const dpl_linear* linear, int64_t tokens, size_t* bytes);

/* The weight gradient from the packed input:
 *   G_r[o][i] = sum_t dy[r][t][o] * x[r][t][i]
 * with x decoded to dtype (DP_BF16 or DP_F16, dy's), products exact and sums in
 * binary32.  DP_BF16 holds every decoded value; DP_F16 holds those of rows packed
 * from DP_F16, and others are rounded to it, to nearest even, beyond its range to
 * an infinity.  rows: host array [n_replicas]. */
dp_status dpl_accumulate_linear(dp_plan* plan, const dpl_linear* linear, int64_t tokens, dp_dtype dtype,
                                const dpl_linear_rows* rows, int64_t ld_codes, int64_t ld_scales, int64_t ld_dy,
                                int32_t first, int32_t more, void* workspace, size_t workspace_bytes,
                                hipStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* DPLAYER_H */

/*
 * dpattn.h -- attention of a model's layers beside the operators of dplayer.h:
 * the positions of queries and keys, the attention itself, and its backward
 * pass.  They have no parameters, so no plan: a call takes the rows of any
 * number of sequences, those of every replica among them if they lie in one
 * tensor.
 *
 * Conventions are those of dpstep.h and dplayer.h: device pointers are the
 * caller's, calls are asynchronous on the caller's stream, never synchronise
 * and never allocate, and return a dp_status.  Memory that a call names as
 * workspace is scratch for the length of that call on its stream: calls that
 * may run at the same time, and graphs that may replay at the same time, need a
 * workspace each.  Outputs must not overlap inputs or each other unless a call
 * says so.  The same call on the same inputs gives the same bits; how a sum is
 * split among waves, and so its last bits, depends on the rows and heads of the
 * call.
 *
 * Rows of heads.  A tensor has `tokens` rows of heads of `dim` elements of a
 * dtype.  Element d of head h in row t is p[t * ld + h * head + d]: the rows of
 * one projection (queries, keys and values side by side), a tensor of its own, or
 * one with the heads outside.  Any element-aligned address and any stride from
 * 0 works for an input (0 repeats a head or a row); rows and heads of an output
 * must not overlap.  Elements between the heads are never read or written.
 */
#ifndef DPATTN_H
#define DPATTN_H

#include <stddef.h>
#include <stdint.h>
#include <hip/hip_runtime_api.h>

#include "dpstep.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Most rows of a tensor, and most sequences. */
#define DPA_MAX_TOKENS (INT64_C(1) << 24)
/* Most heads. */
#define DPA_MAX_HEADS 1024
/* Largest head of the attention. */
#define DPA_MAX_DIM 128
/* Most axes of a position, most pairs of elements that turn, and most tensors
 * of a call of dpa_rotary. */
#define DPA_MAX_AXES 4
#define DPA_MAX_PAIRS 256
#define DPA_MAX_TENSORS 4

typedef struct dpa_rows {
    void* p;      /* an input's memory is only read */
    int64_t ld;   /* elements from a row to the next */
    int64_t head; /* elements from a head to the next */
} dpa_rows;

/* ---- positions ----------------------------------------------------------------- */

/* Rotary positions on several axes.  The first 2 * (sections[0] + ... +
 * sections[axes - 1]) = rot elements of a head are pairs, elements (i, i + rot / 2), or
 * (2 i, 2 i + 1) with interleaved != 0.  The first sections[0] pairs turn with
 * the position on axis 0, the next sections[1] with axis 1, and so on.  Pair i
 * turns by position * base^(-2 i / rot), or with own_ladder != 0, being the
 * j-th of its section, by position * base^(-j / sections[axis]):
 *   y_lo = x_lo cos - x_hi sin
 *   y_hi = x_lo sin + x_hi cos
 * The remaining elements are copied.  Angles are computed and reduced in
 * binary64, so that far positions (to 2^31 and beyond) keep their phase; the
 * products are binary32, rounded once. */
typedef struct dpa_rotary_desc {
    int32_t axes;                   /* 1 .. DPA_MAX_AXES */
    int32_t sections[DPA_MAX_AXES]; /* pairs of each axis, >= 0 */
    int32_t interleaved, own_ladder;
    int32_t reserved; /* 0 */
    double base;      /* > 0 */
} dpa_rotary_desc;

/* One tensor of the call: x and y of `heads` heads each.  y may be x itself (the
 * same address and strides), in place. */
typedef struct dpa_rotary_rows {
    dpa_rows x, y;
    int32_t heads;
    int32_t reserved; /* 0 */
} dpa_rotary_rows;

/* Turns `count` tensors (1 .. DPA_MAX_TENSORS; the queries and the keys, say) of
 * `tokens` rows of heads of dim elements (rot <= dim) by the positions of their
 * rows; inverse != 0 turns them back, which is the backward pass (of dy into
 * dx).  positions: int32_t or int64_t (position_bytes 4 or 8), that of row t on
 * axis a at [t * position_ld + a * position_axis]. */
dp_status dpa_rotary(const dpa_rotary_desc* rotary, int64_t tokens, int32_t dim, const void* positions,
                     int32_t position_bytes, int64_t position_ld, int64_t position_axis, int32_t count,
                     const dpa_rotary_rows* rows, dp_dtype dtype, int32_t inverse, hipStream_t stream);

/* ---- attention --------------------------------------------------------------------- */

/* Which queries see which keys.  Sequence s has the query rows [q_s, q_s + L)
 * and the key rows [k_s, k_s + M).
 *  - offsets null: every sequence has tokens / sequences query rows, one behind
 *    the other (sequences divides tokens; 0 sequences have no rows).
 *    Otherwise they are rows [offsets[s * step], offsets[s * step + 1]) : step
 *    1 for sequences one behind the other (sequences + 1 numbers), 2 for a
 *    begin and an end each (a padded batch).  Device memory, int32_t or int64_t
 *    (offset_bytes 4 or 8).  Begins must not fall, and sequences must not
 *    overlap.  Numbers outside [0, tokens] are limited to it, so that no row
 *    outside the tensors is ever touched; sequences against these rules give
 *    unspecified rows.
 *  - offsets_k the same for the keys.  Null: with offsets the same rows as the
 *    queries' (tokens_k == tokens), without them tokens_k / sequences rows each.
 * Query i of a sequence, i < L, has the place i + M - L among the keys (the last
 * query is at the last key).  It sees key j if
 *   j <= place           with causal != 0
 *   j >  place - window  with window > 0 (0: no window)
 * Rows of no sequence (padding between or behind them) are neither read nor
 * written, in any tensor.  An infinity or NaN in a row may reach the results of
 * other rows of its sequence, those that the mask keeps from it among them: a
 * masked score counts 0 times the value, as in the product by a matrix of
 * probabilities.
 * A call has fewer than 2^23 tiles: (rows / 128 + sequences) times heads. */
typedef struct dpa_attention_desc {
    int32_t heads;    /* of the queries, 1 .. DPA_MAX_HEADS, a multiple of kv_heads */
    int32_t kv_heads; /* query head h reads key head h / (heads / kv_heads) */
    int32_t dim;      /* a multiple of 8 up to DPA_MAX_DIM */
    int32_t causal;
    int64_t window;
    double scale; /* factor of the products, 2^-100 .. 2^100, taken as binary32 */
    int64_t tokens, tokens_k, sequences;
    const void* offsets;
    const void* offsets_k;
    int32_t offset_bytes, step;
} dpa_attention_desc;

/* out_i = sum_j p_ij v_j, p_ij = exp(scale q_i k_j - lse_i), over the keys j that
 * query i sees; lse[h * tokens + i] = log(sum_j exp(scale q_i k_j)), binary32.  A
 * query that sees no key gets a row of zeros and lse = -infinity.  dtype is
 * DP_BF16 or DP_F16, of all four tensors; products are exact and summed in
 * binary32, and p is rounded to dtype before its product with v.  Scores scale q_i k_j lie
 * within 2^24 of 0, where binary32 numbers are one apart: beyond, rows are unspecified (in
 * dpa_attention_backward p is off by some 2^-22 |lse| of itself). */
dp_status dpa_attention(const dpa_attention_desc* attention, dp_dtype dtype, const dpa_rows* q, const dpa_rows* k,
                        const dpa_rows* v, const dpa_rows* out, float* lse, hipStream_t stream);

/* Bytes of workspace for dpa_attention_backward (host work only). */
dp_status dpa_attention_workspace(int64_t tokens, int32_t heads, size_t* bytes);

/* The gradients of q, k and v from that of out, with the out and lse that
 * dpa_attention left:
 *   dv_j = sum_i p_ij dout_i
 *   ds_ij = p_ij (dout_i v_j - dout_i out_i)
 *   dq_i = scale sum_j ds_ij k_j,  dk_j = scale sum_i ds_ij q_i
 * with p computed again from lse; p and ds are rounded to dtype before their
 * products.  In f16 ds keeps its bits only from 2^-14 (6e-5) on, is 0 below 2^-25 and
 * infinite from 65520 on, and it falls with the length of a row: dout wants the loss scale
 * that f16 gradients take anyway.  (p keeps its bits down to 2^-24; in dpa_attention to
 * 2^-20 of the row's greatest.)  dk and dv of a key head are sums over the query heads
 * that read it.  A key that no query sees, and a query that sees no key, get zeros.
 * (Inputs that repeat a head or a row by a stride of 0 get the gradient of each
 * repetition; dq, dk and dv are tensors of their own, as is every output.) */
dp_status dpa_attention_backward(const dpa_attention_desc* attention, dp_dtype dtype, const dpa_rows* q,
                                 const dpa_rows* k, const dpa_rows* v, const dpa_rows* out, const float* lse,
                                 const dpa_rows* dout, const dpa_rows* dq, const dpa_rows* dk, const dpa_rows* dv,
                                 void* workspace, size_t workspace_bytes, hipStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* DPATTN_H */

// Internal interface between the attention's C ABI (attention.cpp) and its
// gfx950 kernels.  Not installed; not part of the ABI.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "dpattn.h"
#include "dploss.h"

namespace dpk {

// Where the sequences lie, and their mask, as the kernels see them.
struct Sequences {
    const void* offsets[2];  // of the queries and the keys; null: equal lengths
    int64_t rows[2];         // of the tensors
    int64_t length[2];       // of a sequence, without offsets
    int32_t offset_bytes, step;
    int32_t count;
    int32_t heads, kv_heads, dim;
    int32_t causal, window;  // window 0: none
    float scale;
};

struct AttentionArgs {
    Sequences s;
    dpa_rows q, k, v, out, dout, dq, dk, dv;
    float* lse;
    float* delta;  // [heads][rows of the queries]
};

// Workgroups of a launch for tiles of `tile` rows of the queries (side 0) or the keys (1).
int64_t attention_slots(const Sequences& s, int side, int64_t tile);
// How the waves of a workgroup share the rows of the queries (side 0) or the keys (1).
enum class AttentionShape { kPlain, kWide, kPairs, kSplit };
AttentionShape attention_shape(const Sequences& s, int side);
int64_t attention_groups(const Sequences& s);  // most workgroups of any launch
hipError_t launch_attention(dp_dtype dt, const AttentionArgs& a, hipStream_t stream);
hipError_t launch_attention_grad(dp_dtype dt, const AttentionArgs& a, hipStream_t stream);

struct RotaryArgs {
    double frequency[DPA_MAX_PAIRS];
    unsigned char axis[DPA_MAX_PAIRS];
    dpa_rotary_rows rows[DPA_MAX_TENSORS];
    const void* positions;
    int64_t position_ld, position_axis, tokens;
    int32_t position_bytes, count, dim, pairs;
    bool interleaved, inverse;
    bool once;  // what is written passes the caches
};
hipError_t launch_rotary(dp_dtype dt, const RotaryArgs& a, hipStream_t stream);

struct DistillArgs {
    const void* logits;
    const void* teacher;
    const void* ids;
    const float* total;
    const void* labels;
    const float* weight;
    float* loss;
    void* dlogits;
    int64_t tokens, vocab, ld, ld_teacher, ld_ids, ld_dlogits;
    int32_t top, id_bytes;
    float temperature, soft, hard, scale;
};
hipError_t launch_distill(dp_dtype dt, dp_dtype teacher_dt, const DistillArgs& a, hipStream_t stream);

}  // namespace dpk

// Internal interface between the layer operators' C ABI (layers.cpp) and
// their gfx950 kernels.  Not installed; not part of the ABI.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "dplayer.h"
#include "dpstep.h"

namespace dpk {

// ---- embedding (embed.hip) -------------------------------------------------
hipError_t launch_embed(dp_dtype pdt, dp_dtype odt, const void* table, int64_t rows, int64_t dim, float scale,
                        int64_t tokens, const void* ids, int id_bytes, void* out, int64_t ld,
                        hipStream_t stream);

struct EmbedGrad {
    const void* ids[DP_MAX_REPLICAS];
    const void* dy[DP_MAX_REPLICAS];
    float* acc[DP_MAX_REPLICAS];
    int64_t rows, dim, tokens, ld;
    float scale;
    int32_t n, id_bytes;
    bool overwrite;  // ACC = G, else ACC += G
};
size_t embed_workspace(int64_t dim, int64_t tokens, int n);
int64_t embed_waves(const EmbedGrad& a);   // workgroups of the sums, of four waves, for one replica
int64_t embed_groups(const EmbedGrad& a);  // workgroups of the first launch: the sort's and the zeros'
hipError_t launch_embed_grad(dp_dtype dt, const EmbedGrad& a, void* workspace, hipStream_t stream);

// ---- norms around a block (block_norm.hip) -----------------------------------
struct BlockNorm {
    const void* weight[5];  // post_w, post_b, gate, pre_w, pre_b in the parameter dtype; null: none
    int64_t dim;
    float eps, alpha;
    bool centered;
    bool bias;  // post_b or pre_b is there
};
hipError_t launch_block_norm(dp_dtype dt, dp_dtype pdt, const BlockNorm& b, int64_t tokens, const void* h,
                             int64_t ld_h, const void* y, int64_t ld_y, void* s, int64_t ld_s, void* x, int64_t ld_x,
                             hipStream_t stream);
size_t block_norm_workspace(const BlockNorm& b, int64_t tokens, int n);  // reads dim, centered and bias
// at[i]: which accumulator (acc[at * n + r], overwrite[at]) takes the gradient
// of weight i, -1 for none.
hipError_t launch_block_grad(dp_dtype dt, dp_dtype pdt, const BlockNorm& b, int64_t tokens, int n,
                             const dpl_norm_rows* rows, int64_t ld, float* const* acc, const int* at,
                             const bool* overwrite, void* workspace, hipStream_t stream);

// ---- activations in 8 bits (act8.hip) ------------------------------------------
hipError_t launch_pack(dp_dtype dt, int64_t tokens, int64_t dim, const void* x, int64_t ld, void* codes,
                       int64_t ld_codes, void* scales, int64_t ld_scales, hipStream_t stream);
hipError_t launch_unpack(dp_dtype dt, int64_t tokens, int64_t dim, const void* codes, int64_t ld_codes,
                         const void* scales, int64_t ld_scales, void* x, int64_t ld, hipStream_t stream);

// ---- weight gradient of a linear layer (linear.hip) -----------------------------
struct LinearGrad {
    dpl_linear_rows rows[DP_MAX_REPLICAS];
    float* acc[DP_MAX_REPLICAS];
    int64_t tokens, outputs, inputs, ld_dy, ld_codes, ld_scales;
    int32_t n;
    bool transposed, overwrite;
    bool pieces;  // rows of at least one 16-byte piece, tiles within 32-bit offsets
};
int64_t linear_jobs(int64_t outputs, int64_t inputs, int64_t tokens, int n);  // workgroups of its launch
size_t linear_workspace(int64_t outputs, int64_t inputs, int64_t tokens, int n);
hipError_t launch_linear(dp_dtype dt, const LinearGrad& g, void* workspace, hipStream_t stream);

}  // namespace dpk

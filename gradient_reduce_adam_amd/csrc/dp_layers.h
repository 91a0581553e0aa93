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
// `vec` flags say that rows can be moved in whole vectors: base addresses and
// row strides are multiples of what one lane moves.
hipError_t launch_embed(dp_dtype pdt, dp_dtype odt, const void* table, int64_t rows, int64_t dim, float scale,
                        int64_t tokens, const void* ids, int id_bytes, void* out, int64_t ld, bool vec,
                        hipStream_t stream);

struct EmbedGrad {
    const void* ids[DP_MAX_REPLICAS];
    const void* dy[DP_MAX_REPLICAS];
    float* acc[DP_MAX_REPLICAS];
    int64_t rows, dim, tokens, ld;
    float scale;
    int32_t n, id_bytes;
    bool overwrite;       // ACC = G, else ACC += G
    bool vec_dy, vec_acc;
};
size_t embed_workspace(int64_t dim, int64_t tokens, int n);
int64_t embed_waves(const EmbedGrad& a);  // workgroups of its largest launch, for one replica
hipError_t launch_embed_grad(dp_dtype dt, const EmbedGrad& a, void* workspace, hipStream_t stream);

}  // namespace dpk

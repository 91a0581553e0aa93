// C ABI of the layer operators (dplayer.h): argument checks, the plan's part
// in each call, and the launches.  The kernels live in embed.hip,
// block_norm.hip, act8.hip and linear.hip.
#include <hip/hip_runtime.h>

#include <cmath>
#include <initializer_list>

#include "dp_layers.h"
#include "dplayer.h"
#include "plan.h"

using dpapi::fail;
using dpapi::hip_fail;

namespace {

constexpr int64_t kMaxWaves = (int64_t{1} << 26) - 1;  // one-wave workgroups of one dispatch

int64_t esize(dp_dtype d) { return d == DP_F32 ? 4 : 2; }
bool dtype_ok(dp_dtype d) { return d == DP_F32 || d == DP_F16 || d == DP_BF16; }
long long ll(int64_t x) { return static_cast<long long>(x); }

dp_status launched(hipError_t e, const char* what) { return e == hipSuccess ? DP_OK : hip_fail(e, what); }

bool multiple(const void* p, int64_t bytes) { return reinterpret_cast<uintptr_t>(p) % static_cast<uintptr_t>(bytes) == 0; }

// Rows that can be moved `bytes` at a time.
bool vec_rows(const void* p, int64_t ld, int64_t elem, int64_t bytes) {
    return multiple(p, bytes) && ld * elem % bytes == 0;
}

dp_status check_rows(const char* where, const char* what, const void* p, int64_t tokens, int64_t dim, int64_t ld,
                     int64_t elem) {
    if (tokens > 0 && !p) return fail(DP_ERR_INVALID_ARG, "%s: %s is null", where, what);
    if (ld < dim) return fail(DP_ERR_INVALID_ARG, "%s: %s: row stride %lld below the row's %lld", where, what, ll(ld), ll(dim));
    if (ld > (int64_t{1} << 40)) return fail(DP_ERR_INVALID_ARG, "%s: %s: row stride %lld", where, what, ll(ld));
    if (!multiple(p, elem)) return fail(DP_ERR_INVALID_ARG, "%s: %s is not aligned to its elements", where, what);
    return DP_OK;
}

dp_status check_tokens(const char* where, int64_t tokens) {
    if (tokens < 0 || tokens > DPL_MAX_TOKENS)
        return fail(DP_ERR_INVALID_ARG, "%s: %lld tokens outside [0, %lld]", where, ll(tokens), ll(DPL_MAX_TOKENS));
    return DP_OK;
}

dp_status check_tensor(const char* where, const dp_plan* plan, int32_t tensor) {
    if (tensor < 0 || tensor >= plan->T)
        return fail(DP_ERR_INVALID_ARG, "%s: tensor %d outside [0, %d)", where, tensor, plan->T);
    if (plan->numel[static_cast<size_t>(tensor)] == 0)
        return fail(DP_ERR_INVALID_ARG, "%s: tensor %d has no elements", where, tensor);
    return DP_OK;
}

dp_status check_workspace(const char* where, const void* workspace, size_t have, size_t want) {
    if (have < want)
        return fail(DP_ERR_INVALID_ARG, "%s: workspace of %zu bytes, %zu are needed", where, have, want);
    if (want > 0 && (!workspace || !multiple(workspace, 256)))
        return fail(DP_ERR_INVALID_ARG, "%s: the workspace must be aligned to 256 bytes", where);
    return DP_OK;
}

// The accumulators of a whole-tensor call are binary32 at element alignment.
dp_status check_acc(const char* where, float* const* acc, int count) {
    for (int i = 0; i < count; ++i)
        if (!acc[i] || !multiple(acc[i], 4)) return fail(DP_ERR_INVALID_ARG, "%s: an accumulator is not aligned to its elements", where);
    return DP_OK;
}

// ---- embedding ---------------------------------------------------------------
dp_status check_table(const char* where, const dp_plan* plan, const dpl_table* t, int64_t* rows) {
    if (!plan || !t) return fail(DP_ERR_INVALID_ARG, "%s: null argument", where);
    dp_status s = check_tensor(where, plan, t->tensor);
    if (s != DP_OK) return s;
    const int64_t numel = plan->numel[static_cast<size_t>(t->tensor)];
    if (t->dim < 1 || t->dim > (int64_t{1} << 26) || numel % t->dim != 0)
        return fail(DP_ERR_INVALID_ARG, "%s: tensor %d of %lld elements has no rows of %lld", where, t->tensor, ll(numel), ll(t->dim));
    *rows = numel / t->dim;
    if (*rows >= INT32_MAX) return fail(DP_ERR_INVALID_ARG, "%s: %lld rows (below 2^31 - 1 are supported)", where, ll(*rows));
    if (t->id_bytes != 4 && t->id_bytes != 8) return fail(DP_ERR_INVALID_ARG, "%s: ids of %d bytes (4 or 8)", where, t->id_bytes);
    if (!std::isfinite(static_cast<float>(t->scale))) return fail(DP_ERR_INVALID_ARG, "%s: the scale is not finite", where);
    return DP_OK;
}

dp_status check_ids(const char* where, const void* ids, int64_t tokens, int32_t id_bytes) {
    if (tokens > 0 && (!ids || !multiple(ids, id_bytes)))
        return fail(DP_ERR_INVALID_ARG, "%s: ids are null or not aligned to their elements", where);
    return DP_OK;
}

}  // namespace

extern "C" {

dp_status dpl_embed(dp_plan* plan, const dpl_table* table, int64_t tokens, const void* ids, dp_dtype dtype, void* out,
                    int64_t ld, hipStream_t stream) {
    const char* where = "dpl_embed";
    int64_t rows = 0;
    dp_status s = check_table(where, plan, table, &rows);
    if (s == DP_OK) s = check_tokens(where, tokens);
    if (s == DP_OK && !dtype_ok(dtype)) s = fail(DP_ERR_INVALID_ARG, "%s: unknown dtype %d", where, static_cast<int>(dtype));
    if (s == DP_OK) s = check_ids(where, ids, tokens, table->id_bytes);
    if (s == DP_OK) s = check_rows(where, "out", out, tokens, table->dim, ld, esize(dtype));
    const void* w = nullptr;
    if (s == DP_OK) s = dpapi::param_of(plan, table->tensor, &w);
    if (s != DP_OK) return s;
    const bool vec = vec_rows(w, table->dim, 2, 16) && vec_rows(out, ld, esize(dtype), 16);
    return launched(dpk::launch_embed(plan->pdt, dtype, w, rows, table->dim, static_cast<float>(table->scale), tokens,
                                      ids, table->id_bytes, out, ld, vec, stream),
                    "embedding launch");
}

dp_status dpl_embed_workspace(const dp_plan* plan, const dpl_table* table, int64_t tokens, size_t* bytes) {
    int64_t rows = 0;
    dp_status s = check_table("dpl_embed_workspace", plan, table, &rows);
    if (s == DP_OK) s = check_tokens("dpl_embed_workspace", tokens);
    if (s == DP_OK && !bytes) s = fail(DP_ERR_INVALID_ARG, "dpl_embed_workspace: null argument");
    if (s != DP_OK) return s;
    *bytes = dpk::embed_workspace(table->dim, tokens, plan->n);
    return DP_OK;
}

dp_status dpl_accumulate_embed(dp_plan* plan, const dpl_table* table, int64_t tokens, const void* const* ids,
                               dp_dtype dtype, const void* const* dy, int64_t ld, int32_t first, int32_t more,
                               void* workspace, size_t workspace_bytes, hipStream_t stream) {
    const char* where = "dpl_accumulate_embed";
    dpk::EmbedGrad a{};
    dp_status s = check_table(where, plan, table, &a.rows);
    if (s == DP_OK) s = check_tokens(where, tokens);
    if (s != DP_OK) return s;
    if (!dtype_ok(dtype)) return fail(DP_ERR_INVALID_ARG, "%s: unknown dtype %d", where, static_cast<int>(dtype));
    if (!ids || !dy) return fail(DP_ERR_INVALID_ARG, "%s: null argument", where);
    a.n = plan->n;
    a.vec_dy = a.vec_acc = true;
    for (int32_t r = 0; r < plan->n; ++r) {
        s = check_ids(where, ids[r], tokens, table->id_bytes);
        if (s == DP_OK) s = check_rows(where, "dy", dy[r], tokens, table->dim, ld, esize(dtype));
        if (s != DP_OK) return s;
        a.ids[r] = ids[r];
        a.dy[r] = dy[r];
        a.vec_dy = a.vec_dy && vec_rows(dy[r], ld, esize(dtype), 4 * esize(dtype));
    }
    s = check_workspace(where, workspace, workspace_bytes, dpk::embed_workspace(table->dim, tokens, plan->n));
    if (s != DP_OK) return s;
    bool overwrite = false;
    s = dpapi::part_begin(plan, &table->tensor, 1, first != 0, where, a.acc, &overwrite);
    if (s == DP_OK) s = check_acc(where, a.acc, plan->n);
    if (s != DP_OK) return s;
    for (int32_t r = 0; r < plan->n; ++r) a.vec_acc = a.vec_acc && vec_rows(a.acc[r], table->dim, 4, 16);
    a.dim = table->dim;
    a.tokens = tokens;
    a.ld = ld;
    a.scale = static_cast<float>(table->scale);
    a.id_bytes = table->id_bytes;
    a.overwrite = overwrite;
    if (dpk::embed_waves(a) > kMaxWaves)
        return fail(DP_ERR_INVALID_ARG, "%s: %lld tokens of %lld elements are too many for one call", where, ll(tokens), ll(a.dim));
    s = launched(dpk::launch_embed_grad(dtype, a, workspace, stream), "embedding gradient launch");
    if (s != DP_OK) return s;
    dpapi::part_end(plan, &table->tensor, 1, first != 0, more != 0);
    return DP_OK;
}

}  // extern "C"

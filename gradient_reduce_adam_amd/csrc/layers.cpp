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

// one dispatch has fewer than 2^32 threads: workgroups of one wave, and of 1024 threads
constexpr int64_t kMaxWaves = (int64_t{1} << 26) - 1;
constexpr int64_t kMaxGroups = (int64_t{1} << 22) - 1;

int64_t esize(dp_dtype d) { return d == DP_F32 ? 4 : 2; }
bool dtype_ok(dp_dtype d) { return d == DP_F32 || d == DP_F16 || d == DP_BF16; }
long long ll(int64_t x) { return static_cast<long long>(x); }

dp_status launched(hipError_t e, const char* what) { return e == hipSuccess ? DP_OK : hip_fail(e, what); }

bool multiple(const void* p, int64_t bytes) { return reinterpret_cast<uintptr_t>(p) % static_cast<uintptr_t>(bytes) == 0; }

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

// ---- norms around a block ----------------------------------------------------
// The tensors of a dpl_norms in the kernels' order, and their parameters.
struct Norms {
    dpk::BlockNorm b{};
    int32_t tensors[5];  // those that are there
    int at[5];           // weight i is tensors[at[i]], -1: none
    int count = 0;
};

dp_status check_norms(const char* where, const dp_plan* plan, const dpl_norms* d, Norms* out) {
    if (!plan || !d) return fail(DP_ERR_INVALID_ARG, "%s: null argument", where);
    if (d->dim < 1 || d->dim > DPL_MAX_NORM_DIM)
        return fail(DP_ERR_INVALID_ARG, "%s: rows of %lld elements outside [1, %d]", where, ll(d->dim), DPL_MAX_NORM_DIM);
    const float eps = static_cast<float>(d->eps), alpha = static_cast<float>(d->residual_scale);
    if (!(eps > 0.0f) || !std::isfinite(eps)) return fail(DP_ERR_INVALID_ARG, "%s: eps must be a positive binary32 number", where);
    if (!std::isfinite(alpha)) return fail(DP_ERR_INVALID_ARG, "%s: the residual scale is not finite", where);
    const int32_t t[5] = {d->post_w, d->post_b, d->gate, d->pre_w, d->pre_b};
    const char* names[5] = {"post_w", "post_b", "gate", "pre_w", "pre_b"};
    for (int i = 0; i < 5; ++i) {
        out->at[i] = -1;
        if (t[i] < 0) continue;
        dp_status s = check_tensor(where, plan, t[i]);
        if (s != DP_OK) return s;
        if (plan->numel[static_cast<size_t>(t[i])] != d->dim)
            return fail(DP_ERR_INVALID_ARG, "%s: %s is tensor %d of %lld elements, rows have %lld", where, names[i], t[i],
                        ll(plan->numel[static_cast<size_t>(t[i])]), ll(d->dim));
        for (int k = 0; k < out->count; ++k)
            if (out->tensors[k] == t[i]) return fail(DP_ERR_INVALID_ARG, "%s: tensor %d is named twice", where, t[i]);
        out->at[i] = out->count;
        out->tensors[out->count++] = t[i];
    }
    if ((d->post_b >= 0 && d->post_w < 0) || (d->pre_b >= 0 && d->pre_w < 0))
        return fail(DP_ERR_INVALID_ARG, "%s: a bias without its weight", where);
    out->b.dim = d->dim;
    out->b.eps = eps;
    out->b.alpha = alpha;
    out->b.centered = d->centered != 0;
    out->b.bias = d->post_b >= 0 || d->pre_b >= 0;
    return DP_OK;
}

// The weights' addresses, once everything else is checked.
dp_status norm_weights(const char* where, dp_plan* plan, Norms* n) {
    if (n->count == 0) return dpapi::ensure_device(plan);
    for (int i = 0; i < 5; ++i) {
        if (n->at[i] < 0) continue;
        dp_status s = dpapi::param_of(plan, n->tensors[n->at[i]], &n->b.weight[i]);
        if (s != DP_OK) return s;
        if (!multiple(n->b.weight[i], 2)) return fail(DP_ERR_INVALID_ARG, "%s: a weight is not aligned to its elements", where);
    }
    return DP_OK;
}

// Rows of 16-bit elements go with parameters of the same type.
dp_status check_norm_dtype(const char* where, const dp_plan* plan, dp_dtype dtype) {
    if (!dtype_ok(dtype)) return fail(DP_ERR_INVALID_ARG, "%s: unknown dtype %d", where, static_cast<int>(dtype));
    if (dtype != DP_F32 && dtype != plan->pdt)
        return fail(DP_ERR_INVALID_ARG, "%s: 16-bit rows must have the parameters' dtype", where);
    return DP_OK;
}

// ---- activations in 8 bits -----------------------------------------------------
dp_status check_packed(const char* where, int64_t tokens, int64_t dim, dp_dtype dtype, const void* codes,
                       int64_t ld_codes, const void* scales, int64_t ld_scales) {
    dp_status s = check_tokens(where, tokens);
    if (s != DP_OK) return s;
    if (dim < 1 || dim > (int64_t{1} << 24)) return fail(DP_ERR_INVALID_ARG, "%s: rows of %lld elements outside [1, 2^24]", where, ll(dim));
    if (!dtype_ok(dtype)) return fail(DP_ERR_INVALID_ARG, "%s: unknown dtype %d", where, static_cast<int>(dtype));
    s = check_rows(where, "codes", codes, tokens, dim, ld_codes, 1);
    if (s == DP_OK) s = check_rows(where, "scales", scales, tokens, (dim + DPL_GROUP - 1) / DPL_GROUP, ld_scales, 1);
    if (s != DP_OK) return s;
    if ((dim + DPL_GROUP - 1) / DPL_GROUP * tokens > (int64_t{1} << 30))
        return fail(DP_ERR_INVALID_ARG, "%s: %lld rows of %lld elements are too many for one call", where, ll(tokens), ll(dim));
    return DP_OK;
}

// ---- weight gradient of a linear layer -------------------------------------------
dp_status check_linear(const char* where, const dp_plan* plan, const dpl_linear* d, int64_t tokens) {
    if (!plan || !d) return fail(DP_ERR_INVALID_ARG, "%s: null argument", where);
    dp_status s = check_tensor(where, plan, d->tensor);
    if (s == DP_OK) s = check_tokens(where, tokens);
    if (s != DP_OK) return s;
    const int64_t most = int64_t{1} << 24, numel = plan->numel[static_cast<size_t>(d->tensor)];
    if (d->inputs < 1 || d->outputs < 1 || d->inputs > most || d->outputs > most || d->inputs * d->outputs != numel)
        return fail(DP_ERR_INVALID_ARG, "%s: tensor %d of %lld elements is no %lld x %lld matrix", where, d->tensor,
                    ll(numel), ll(d->outputs), ll(d->inputs));
    if (dpk::linear_jobs(d->outputs, d->inputs, tokens, plan->n) > kMaxGroups)
        return fail(DP_ERR_INVALID_ARG, "%s: a %lld x %lld matrix is too large for one call", where, ll(d->outputs),
                    ll(d->inputs));
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
    if (!multiple(w, 2)) return fail(DP_ERR_INVALID_ARG, "%s: the table is not aligned to its elements", where);
    return launched(dpk::launch_embed(plan->pdt, dtype, w, rows, table->dim, static_cast<float>(table->scale), tokens,
                                      ids, table->id_bytes, out, ld, stream),
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
    for (int32_t r = 0; r < plan->n; ++r) {
        s = check_ids(where, ids[r], tokens, table->id_bytes);
        if (s == DP_OK) s = check_rows(where, "dy", dy[r], tokens, table->dim, ld, esize(dtype));
        if (s != DP_OK) return s;
        a.ids[r] = ids[r];
        a.dy[r] = dy[r];
    }
    s = check_workspace(where, workspace, workspace_bytes, dpk::embed_workspace(table->dim, tokens, plan->n));
    if (s != DP_OK) return s;
    bool overwrite = false;
    s = dpapi::part_begin(plan, &table->tensor, 1, first != 0, where, a.acc, &overwrite);
    if (s == DP_OK) s = check_acc(where, a.acc, plan->n);
    if (s != DP_OK) return s;
    a.dim = table->dim;
    a.tokens = tokens;
    a.ld = ld;
    a.scale = static_cast<float>(table->scale);
    a.id_bytes = table->id_bytes;
    a.overwrite = overwrite;
    if (dpk::embed_waves(a) > kMaxWaves / 4 || dpk::embed_groups(a) > kMaxGroups)
        return fail(DP_ERR_INVALID_ARG, "%s: %lld tokens of %lld elements and %lld rows are too many for one call", where,
                    ll(tokens), ll(a.dim), ll(a.rows));
    s = launched(dpk::launch_embed_grad(dtype, a, workspace, stream), "embedding gradient launch");
    if (s != DP_OK) return s;
    dpapi::part_end(plan, &table->tensor, 1, first != 0, more != 0);
    return DP_OK;
}

dp_status dpl_block_norm(dp_plan* plan, const dpl_norms* norms, int64_t tokens, dp_dtype dtype, const void* h,
                         int64_t ld_h, const void* y, int64_t ld_y, void* s_out, int64_t ld_s, void* x, int64_t ld_x,
                         hipStream_t stream) {
    const char* where = "dpl_block_norm";
    Norms n;
    dp_status s = check_norms(where, plan, norms, &n);
    if (s == DP_OK) s = check_tokens(where, tokens);
    if (s == DP_OK) s = check_norm_dtype(where, plan, dtype);
    if (s != DP_OK) return s;
    const int64_t e = esize(dtype);
    const bool has_x = n.at[3] >= 0;
    s = check_rows(where, "h", h, tokens, n.b.dim, ld_h, e);
    if (s == DP_OK) s = check_rows(where, "y", y, tokens, n.b.dim, ld_y, e);
    if (s == DP_OK) s = check_rows(where, "s", s_out, tokens, n.b.dim, ld_s, e);
    if (s == DP_OK && has_x) s = check_rows(where, "x", x, tokens, n.b.dim, ld_x, e);
    if (s != DP_OK) return s;
    if (!has_x && x) return fail(DP_ERR_INVALID_ARG, "%s: x without a norm before the next block", where);
    if (tokens > 1 && ((s_out == h && ld_s != ld_h) || (s_out == y && ld_s != ld_y)))
        return fail(DP_ERR_INVALID_ARG, "%s: s in place of an input needs its row stride", where);
    if (tokens > 0 && x && (x == h || x == y || x == s_out))
        return fail(DP_ERR_INVALID_ARG, "%s: x must not overlap another tensor", where);
    s = norm_weights(where, plan, &n);
    if (s != DP_OK) return s;
    return launched(dpk::launch_block_norm(dtype, plan->pdt, n.b, tokens, h, ld_h, y, ld_y, s_out, ld_s,
                                           has_x ? x : nullptr, ld_x, stream),
                    "block norm launch");
}

dp_status dpl_block_norm_workspace(const dp_plan* plan, const dpl_norms* norms, int64_t tokens, size_t* bytes) {
    Norms n;
    dp_status s = check_norms("dpl_block_norm_workspace", plan, norms, &n);
    if (s == DP_OK) s = check_tokens("dpl_block_norm_workspace", tokens);
    if (s == DP_OK && !bytes) s = fail(DP_ERR_INVALID_ARG, "dpl_block_norm_workspace: null argument");
    if (s != DP_OK) return s;
    *bytes = dpk::block_norm_workspace(n.b, tokens, plan->n);
    return DP_OK;
}

dp_status dpl_accumulate_block_norm(dp_plan* plan, const dpl_norms* norms, int64_t tokens, dp_dtype dtype,
                                    const dpl_norm_rows* rows, int64_t ld, int32_t first, int32_t more,
                                    void* workspace, size_t workspace_bytes, hipStream_t stream) {
    const char* where = "dpl_accumulate_block_norm";
    Norms n;
    dp_status s = check_norms(where, plan, norms, &n);
    if (s == DP_OK) s = check_tokens(where, tokens);
    if (s == DP_OK) s = check_norm_dtype(where, plan, dtype);
    if (s != DP_OK) return s;
    if (!rows) return fail(DP_ERR_INVALID_ARG, "%s: null argument", where);
    if (n.count == 0) return fail(DP_ERR_INVALID_ARG, "%s: no norm and no gate", where);
    const int64_t e = esize(dtype);
    const bool has_x = n.at[3] >= 0, has_y = n.at[0] >= 0 || n.at[2] >= 0;
    for (int32_t r = 0; r < plan->n; ++r) {
        const dpl_norm_rows& p = rows[r];
        const void* all[6] = {p.s, p.y, p.dx, p.ds, p.dh, p.dy};
        const char* names[6] = {"s", "y", "dx", "ds", "dh", "dy"};
        const void* zero[6] = {rows[0].s, rows[0].y, rows[0].dx, rows[0].ds, rows[0].dh, rows[0].dy};
        for (int i = 0; i < 6; ++i) {
            if (tokens > 0 && !all[i] != !zero[i])
                return fail(DP_ERR_INVALID_ARG, "%s: %s is null for some replicas only", where, names[i]);
            s = check_rows(where, names[i], all[i], 0, n.b.dim, ld, e);
            if (s != DP_OK) return s;
        }
        if (tokens > 0 && !p.dx != !has_x)
            return fail(DP_ERR_INVALID_ARG, "%s: dx is given exactly with a norm before the next block", where);
        if (tokens > 0 && has_x && !p.s) return fail(DP_ERR_INVALID_ARG, "%s: s is null", where);
        if (tokens > 0 && has_y && !p.y) return fail(DP_ERR_INVALID_ARG, "%s: y is null", where);
        if (tokens > 0 && !has_x && !p.ds) return fail(DP_ERR_INVALID_ARG, "%s: no gradient: dx and ds are null", where);
        if (tokens > 0 && ((p.dh && (p.dh == p.dy || p.dh == p.s || p.dh == p.y)) || (p.dy && p.dy == p.s)))
            return fail(DP_ERR_INVALID_ARG, "%s: outputs overlap each other, s or y", where);
    }
    s = check_workspace(where, workspace, workspace_bytes, dpk::block_norm_workspace(n.b, tokens, plan->n));
    if (s != DP_OK) return s;
    float* acc[5 * DP_MAX_REPLICAS];
    bool overwrite[5];
    s = dpapi::part_begin(plan, n.tensors, n.count, first != 0, where, acc, overwrite);
    if (s == DP_OK) s = norm_weights(where, plan, &n);
    if (s == DP_OK) s = check_acc(where, acc, n.count * plan->n);
    if (s != DP_OK) return s;
    s = launched(dpk::launch_block_grad(dtype, plan->pdt, n.b, tokens, plan->n, rows, ld, acc, n.at, overwrite,
                                        workspace, stream),
                 "block norm gradient launch");
    if (s != DP_OK) return s;
    dpapi::part_end(plan, n.tensors, n.count, first != 0, more != 0);
    return DP_OK;
}

dp_status dpl_pack_activations(int64_t tokens, int64_t dim, dp_dtype dtype, const void* x, int64_t ld, void* codes,
                               int64_t ld_codes, void* scales, int64_t ld_scales, hipStream_t stream) {
    const char* where = "dpl_pack_activations";
    dp_status s = check_packed(where, tokens, dim, dtype, codes, ld_codes, scales, ld_scales);
    if (s == DP_OK) s = check_rows(where, "x", x, tokens, dim, ld, esize(dtype));
    if (s != DP_OK) return s;
    return launched(dpk::launch_pack(dtype, tokens, dim, x, ld, codes, ld_codes, scales, ld_scales, stream),
                    "activation packing launch");
}

dp_status dpl_unpack_activations(int64_t tokens, int64_t dim, dp_dtype dtype, const void* codes, int64_t ld_codes,
                                 const void* scales, int64_t ld_scales, void* x, int64_t ld, hipStream_t stream) {
    const char* where = "dpl_unpack_activations";
    dp_status s = check_packed(where, tokens, dim, dtype, codes, ld_codes, scales, ld_scales);
    if (s == DP_OK) s = check_rows(where, "x", x, tokens, dim, ld, esize(dtype));
    if (s != DP_OK) return s;
    return launched(dpk::launch_unpack(dtype, tokens, dim, codes, ld_codes, scales, ld_scales, x, ld, stream),
                    "activation unpacking launch");
}

dp_status dpl_linear_workspace(const dp_plan* plan, const dpl_linear* linear, int64_t tokens, size_t* bytes) {
    dp_status s = check_linear("dpl_linear_workspace", plan, linear, tokens);
    if (s == DP_OK && !bytes) s = fail(DP_ERR_INVALID_ARG, "dpl_linear_workspace: null argument");
    if (s != DP_OK) return s;
    *bytes = dpk::linear_workspace(linear->outputs, linear->inputs, tokens, plan->n);
    return DP_OK;
}

dp_status dpl_accumulate_linear(dp_plan* plan, const dpl_linear* linear, int64_t tokens, dp_dtype dtype,
                                const dpl_linear_rows* rows, int64_t ld_codes, int64_t ld_scales, int64_t ld_dy,
                                int32_t first, int32_t more, void* workspace, size_t workspace_bytes,
                                hipStream_t stream) {
    const char* where = "dpl_accumulate_linear";
    dp_status s = check_linear(where, plan, linear, tokens);
    if (s != DP_OK) return s;
    if (dtype != DP_BF16 && dtype != DP_F16) return fail(DP_ERR_INVALID_ARG, "%s: dtype must be DP_BF16 or DP_F16", where);
    if (!rows) return fail(DP_ERR_INVALID_ARG, "%s: null argument", where);
    dpk::LinearGrad g{};
    g.pieces = linear->inputs >= 16 && linear->outputs >= 8 && ld_dy < (int64_t{1} << 24) &&
               ld_codes < (int64_t{1} << 24) && ld_scales < (int64_t{1} << 24);
    for (int32_t r = 0; r < plan->n; ++r) {
        s = check_rows(where, "codes", rows[r].codes, tokens, linear->inputs, ld_codes, 1);
        if (s == DP_OK)
            s = check_rows(where, "scales", rows[r].scales, tokens, (linear->inputs + DPL_GROUP - 1) / DPL_GROUP, ld_scales, 1);
        if (s == DP_OK) s = check_rows(where, "dy", rows[r].dy, tokens, linear->outputs, ld_dy, 2);
        if (s != DP_OK) return s;
        g.rows[r] = rows[r];
    }
    s = check_workspace(where, workspace, workspace_bytes,
                        dpk::linear_workspace(linear->outputs, linear->inputs, tokens, plan->n));
    if (s != DP_OK) return s;
    bool overwrite = false;
    s = dpapi::part_begin(plan, &linear->tensor, 1, first != 0, where, g.acc, &overwrite);
    if (s == DP_OK) s = check_acc(where, g.acc, plan->n);
    if (s != DP_OK) return s;
    g.tokens = tokens;
    g.outputs = linear->outputs;
    g.inputs = linear->inputs;
    g.ld_dy = ld_dy;
    g.ld_codes = ld_codes;
    g.ld_scales = ld_scales;
    g.n = plan->n;
    g.transposed = linear->transposed != 0;
    g.overwrite = overwrite;
    s = launched(dpk::launch_linear(dtype, g, workspace, stream), "linear gradient launch");
    if (s != DP_OK) return s;
    dpapi::part_end(plan, &linear->tensor, 1, first != 0, more != 0);
    return DP_OK;
}

}  // extern "C"

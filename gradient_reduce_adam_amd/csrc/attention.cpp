// C ABI of the attention and its positions (dpattn.h): argument checks and the
// launches.  The kernels live in rotary.hip, attention.hip and attention_grad.hip.
#include <hip/hip_runtime.h>

#include <cmath>

#include "dp_attention.h"
#include "dpattn.h"
#include "plan.h"

using dpapi::fail;
using dpapi::hip_fail;

namespace {

constexpr int64_t kMaxGroups = (int64_t{1} << 23) - 1;  // of up to 512 threads, fewer than 2^32 in a launch
constexpr int64_t kMaxStride = int64_t{1} << 36;        // 2^24 rows stay within 63 bits
constexpr int64_t kMaxRow = (int64_t{1} << 31) - 1;      // of the attention: a row in bytes within 32 bits
// lse / scale, at which the scores of the backward pass start, stays within binary32 for
// any sum of 2^24 exponentials, and so does scale log2(e)
constexpr float kMinScale = 0x1p-100f, kMaxScale = 0x1p100f;
constexpr int32_t kMaxRotaryDim = 4096;
constexpr int32_t kMaxWindow = 1 << 26;  // beyond any two rows' distance

long long ll(int64_t x) { return static_cast<long long>(x); }
int64_t esize(dp_dtype d) { return d == DP_F32 ? 4 : 2; }
dp_status launched(hipError_t e, const char* what) { return e == hipSuccess ? DP_OK : hip_fail(e, what); }
bool multiple(const void* p, int64_t bytes) { return reinterpret_cast<uintptr_t>(p) % static_cast<uintptr_t>(bytes) == 0; }

dp_status check_tokens(const char* where, const char* what, int64_t tokens) {
    if (tokens < 0 || tokens > DPA_MAX_TOKENS)
        return fail(DP_ERR_INVALID_ARG, "%s: %lld %s outside [0, %lld]", where, ll(tokens), what, ll(DPA_MAX_TOKENS));
    return DP_OK;
}

dp_status check_heads(const char* where, const char* what, const dpa_rows* r, int64_t tokens, int64_t heads, int64_t dim,
                      int64_t elem, bool output, int64_t most_ld) {
    if (!r) return fail(DP_ERR_INVALID_ARG, "%s: %s is null", where, what);
    if (tokens > 0 && !r->p) return fail(DP_ERR_INVALID_ARG, "%s: the memory of %s is null", where, what);
    if (!multiple(r->p, elem)) return fail(DP_ERR_INVALID_ARG, "%s: %s is not aligned to its elements", where, what);
    if (r->ld < 0 || r->head < 0 || r->head > kMaxStride || (tokens > 1 && r->ld > most_ld))
        return fail(DP_ERR_INVALID_ARG, "%s: %s: strides %lld and %lld", where, what, ll(r->ld), ll(r->head));
    if (!output || tokens == 0) return DP_OK;
    const bool heads_in_rows = (heads == 1 || r->head >= dim) && (tokens == 1 || r->ld >= (heads - 1) * r->head + dim);
    const bool rows_in_heads = (tokens == 1 || r->ld >= dim) && (heads == 1 || r->head >= (tokens - 1) * r->ld + dim);
    if (!heads_in_rows && !rows_in_heads)
        return fail(DP_ERR_INVALID_ARG, "%s: %s: rows or heads overlap at strides %lld and %lld", where, what, ll(r->ld), ll(r->head));
    return DP_OK;
}

dp_status check_lengths(const char* where, const char* what, int64_t rows, int64_t sequences) {
    if (sequences > 0 && rows % sequences != 0)
        return fail(DP_ERR_INVALID_ARG, "%s: %lld %s are no %lld sequences of one length", where, ll(rows), what, ll(sequences));
    return DP_OK;
}

dp_status check_attention(const char* where, const dpa_attention_desc* d, dp_dtype dtype, dpk::Sequences* s) {
    if (!d) return fail(DP_ERR_INVALID_ARG, "%s: null argument", where);
    if (dtype != DP_BF16 && dtype != DP_F16) return fail(DP_ERR_INVALID_ARG, "%s: dtype must be DP_BF16 or DP_F16", where);
    if (d->heads < 1 || d->heads > DPA_MAX_HEADS || d->kv_heads < 1 || d->heads % d->kv_heads != 0)
        return fail(DP_ERR_INVALID_ARG, "%s: %d heads that read %d", where, d->heads, d->kv_heads);
    if (d->dim < 8 || d->dim > DPA_MAX_DIM || d->dim % 8 != 0)
        return fail(DP_ERR_INVALID_ARG, "%s: heads of %d elements (a multiple of 8 up to %d)", where, d->dim, DPA_MAX_DIM);
    const float scale = static_cast<float>(d->scale);
    if (!(scale >= kMinScale && scale <= kMaxScale))
        return fail(DP_ERR_INVALID_ARG, "%s: a scale of %g outside [2^-100, 2^100]", where, d->scale);
    if (d->window < 0) return fail(DP_ERR_INVALID_ARG, "%s: a window of %lld", where, ll(d->window));
    dp_status st = check_tokens(where, "query rows", d->tokens);
    if (st == DP_OK) st = check_tokens(where, "key rows", d->tokens_k);
    if (st == DP_OK) st = check_tokens(where, "sequences", d->sequences);
    if (st != DP_OK) return st;
    if (d->offsets || d->offsets_k) {
        if (d->offset_bytes != 4 && d->offset_bytes != 8)
            return fail(DP_ERR_INVALID_ARG, "%s: offsets of %d bytes (4 or 8)", where, d->offset_bytes);
        if (d->step != 1 && d->step != 2) return fail(DP_ERR_INVALID_ARG, "%s: offsets with step %d (1 or 2)", where, d->step);
        if (!multiple(d->offsets, d->offset_bytes) || !multiple(d->offsets_k, d->offset_bytes))
            return fail(DP_ERR_INVALID_ARG, "%s: offsets are not aligned to their elements", where);
    }
    if (!d->offsets) st = check_lengths(where, "query rows", d->tokens, d->sequences);
    if (st == DP_OK && !d->offsets && !d->offsets_k) st = check_lengths(where, "key rows", d->tokens_k, d->sequences);
    if (st != DP_OK) return st;
    if (d->offsets && !d->offsets_k && d->tokens_k != d->tokens)
        return fail(DP_ERR_INVALID_ARG, "%s: %lld query and %lld key rows at the same offsets", where, ll(d->tokens), ll(d->tokens_k));
    s->offsets[0] = d->offsets;
    s->offsets[1] = d->offsets_k ? d->offsets_k : d->offsets;
    s->rows[0] = d->tokens;
    s->rows[1] = d->tokens_k;
    s->length[0] = d->sequences > 0 ? d->tokens / d->sequences : 0;
    s->length[1] = d->sequences > 0 ? d->tokens_k / d->sequences : 0;
    s->offset_bytes = d->offset_bytes;
    s->step = d->step;
    s->count = static_cast<int32_t>(d->sequences);
    s->heads = d->heads;
    s->kv_heads = d->kv_heads;
    s->dim = d->dim;
    s->causal = d->causal != 0;
    s->window = d->window < kMaxWindow ? static_cast<int32_t>(d->window) : kMaxWindow;
    s->scale = scale;
    if (dpk::attention_groups(*s) > kMaxGroups)
        return fail(DP_ERR_INVALID_ARG, "%s: %lld rows of %d heads are too many for one call", where, ll(d->tokens), d->heads);
    return DP_OK;
}

dp_status check_lse(const char* where, const float* lse, int64_t tokens) {
    if (tokens > 0 && (!lse || !multiple(lse, 4)))
        return fail(DP_ERR_INVALID_ARG, "%s: lse is null or not aligned to its elements", where);
    return DP_OK;
}

}  // namespace

extern "C" {

dp_status dpa_rotary(const dpa_rotary_desc* d, int64_t tokens, int32_t dim, const void* positions, int32_t position_bytes,
                     int64_t position_ld, int64_t position_axis, int32_t count, const dpa_rotary_rows* rows, dp_dtype dtype,
                     int32_t inverse, hipStream_t stream) {
    const char* where = "dpa_rotary";
    if (!d || !rows) return fail(DP_ERR_INVALID_ARG, "%s: null argument", where);
    dp_status s = check_tokens(where, "rows", tokens);
    if (s != DP_OK) return s;
    if (dtype != DP_F32 && dtype != DP_F16 && dtype != DP_BF16)
        return fail(DP_ERR_INVALID_ARG, "%s: unknown dtype %d", where, static_cast<int>(dtype));
    if (d->axes < 1 || d->axes > DPA_MAX_AXES) return fail(DP_ERR_INVALID_ARG, "%s: %d axes outside [1, %d]", where, d->axes, DPA_MAX_AXES);
    if (!(d->base > 0.0) || !std::isfinite(d->base)) return fail(DP_ERR_INVALID_ARG, "%s: the base must be a positive number", where);
    int64_t pairs = 0;
    for (int32_t i = 0; i < d->axes; ++i) {
        if (d->sections[i] < 0) return fail(DP_ERR_INVALID_ARG, "%s: a section of %d pairs", where, d->sections[i]);
        pairs += d->sections[i];
    }
    if (dim < 1 || dim > kMaxRotaryDim) return fail(DP_ERR_INVALID_ARG, "%s: heads of %d elements outside [1, %d]", where, dim, kMaxRotaryDim);
    if (pairs > DPA_MAX_PAIRS || 2 * pairs > dim)
        return fail(DP_ERR_INVALID_ARG, "%s: %lld pairs in heads of %d elements (at most %d)", where, ll(pairs), dim, DPA_MAX_PAIRS);
    if (position_bytes != 4 && position_bytes != 8)
        return fail(DP_ERR_INVALID_ARG, "%s: positions of %d bytes (4 or 8)", where, position_bytes);
    if (position_ld < 0 || position_axis < 0 || position_ld > kMaxStride || position_axis > kMaxStride)
        return fail(DP_ERR_INVALID_ARG, "%s: position strides %lld and %lld", where, ll(position_ld), ll(position_axis));
    if (tokens > 0 && (!positions || !multiple(positions, position_bytes)))
        return fail(DP_ERR_INVALID_ARG, "%s: positions are null or not aligned to their elements", where);
    if (count < 1 || count > DPA_MAX_TENSORS) return fail(DP_ERR_INVALID_ARG, "%s: %d tensors outside [1, %d]", where, count, DPA_MAX_TENSORS);
    dpk::RotaryArgs a{};
    for (int32_t i = 0; i < count; ++i) {
        const dpa_rotary_rows& r = rows[i];
        if (r.heads < 1 || r.heads > DPA_MAX_HEADS) return fail(DP_ERR_INVALID_ARG, "%s: %d heads outside [1, %d]", where, r.heads, DPA_MAX_HEADS);
        s = check_heads(where, "x", &r.x, tokens, r.heads, dim, esize(dtype), false, kMaxStride);
        if (s == DP_OK) s = check_heads(where, "y", &r.y, tokens, r.heads, dim, esize(dtype), true, kMaxStride);
        if (s != DP_OK) return s;
        if (tokens > 0 && r.x.p == r.y.p && ((tokens > 1 && r.x.ld != r.y.ld) || (r.heads > 1 && r.x.head != r.y.head)))
            return fail(DP_ERR_INVALID_ARG, "%s: y in place of x needs its strides", where);
        for (int32_t k = 0; k < count; ++k)
            if (tokens > 0 && k != i && (r.y.p == rows[k].y.p || r.y.p == rows[k].x.p))
                return fail(DP_ERR_INVALID_ARG, "%s: y of tensor %d overlaps tensor %d", where, i, k);
        a.rows[i] = r;
    }
    const double log_base = std::log(d->base);
    int32_t at = 0;
    for (int32_t x = 0; x < d->axes; ++x)
        for (int32_t j = 0; j < d->sections[x]; ++j, ++at) {
            const double power = d->own_ladder ? static_cast<double>(j) / d->sections[x] : static_cast<double>(at) / static_cast<double>(pairs);
            a.frequency[at] = std::exp(-power * log_base);  // off by 1e-15 of it where it is below 1/e, less above
            a.axis[at] = static_cast<unsigned char>(x);
        }
    a.positions = positions;
    a.position_ld = position_ld;
    a.position_axis = position_axis;
    a.tokens = tokens;
    a.position_bytes = position_bytes;
    a.count = count;
    a.dim = dim;
    a.pairs = at;
    a.interleaved = d->interleaved != 0;
    a.inverse = inverse != 0;
    // 16383 tokens of 40 heads of 128, f16: 62 us with streaming stores, 67 without; what the
    // L2 caches hold is left to them, for the attention to read
    int64_t heads = 0;
    for (int32_t i = 0; i < count; ++i) heads += rows[i].heads;
    a.once = tokens * heads * dim * esize(dtype) > int64_t{64} << 20;
    return launched(dpk::launch_rotary(dtype, a, stream), "rotary position launch");
}

dp_status dpa_attention(const dpa_attention_desc* d, dp_dtype dtype, const dpa_rows* q, const dpa_rows* k, const dpa_rows* v,
                        const dpa_rows* out, float* lse, hipStream_t stream) {
    const char* where = "dpa_attention";
    dpk::AttentionArgs a{};
    dp_status s = check_attention(where, d, dtype, &a.s);
    if (s == DP_OK) s = check_heads(where, "q", q, d->tokens, d->heads, d->dim, 2, false, kMaxRow);
    if (s == DP_OK) s = check_heads(where, "k", k, d->tokens_k, d->kv_heads, d->dim, 2, false, kMaxRow);
    if (s == DP_OK) s = check_heads(where, "v", v, d->tokens_k, d->kv_heads, d->dim, 2, false, kMaxRow);
    if (s == DP_OK) s = check_heads(where, "out", out, d->tokens, d->heads, d->dim, 2, true, kMaxRow);
    if (s == DP_OK) s = check_lse(where, lse, d->tokens);
    if (s != DP_OK) return s;
    if (d->tokens > 0 && (out->p == q->p || out->p == k->p || out->p == v->p))
        return fail(DP_ERR_INVALID_ARG, "%s: out overlaps an input", where);
    a.q = *q;
    a.k = *k;
    a.v = *v;
    a.out = *out;
    a.lse = lse;
    return launched(dpk::launch_attention(dtype, a, stream), "attention launch");
}

dp_status dpa_attention_workspace(int64_t tokens, int32_t heads, size_t* bytes) {
    const char* where = "dpa_attention_workspace";
    dp_status s = check_tokens(where, "query rows", tokens);
    if (s != DP_OK) return s;
    if (heads < 1 || heads > DPA_MAX_HEADS) return fail(DP_ERR_INVALID_ARG, "%s: %d heads outside [1, %d]", where, heads, DPA_MAX_HEADS);
    if (!bytes) return fail(DP_ERR_INVALID_ARG, "%s: null argument", where);
    *bytes = static_cast<size_t>(tokens) * static_cast<size_t>(heads) * 4;
    return DP_OK;
}

dp_status dpa_attention_backward(const dpa_attention_desc* d, dp_dtype dtype, const dpa_rows* q, const dpa_rows* k,
                                 const dpa_rows* v, const dpa_rows* out, const float* lse, const dpa_rows* dout,
                                 const dpa_rows* dq, const dpa_rows* dk, const dpa_rows* dv, void* workspace,
                                 size_t workspace_bytes, hipStream_t stream) {
    const char* where = "dpa_attention_backward";
    dpk::AttentionArgs a{};
    dp_status s = check_attention(where, d, dtype, &a.s);
    if (s != DP_OK) return s;
    const struct {
        const char* name;
        const dpa_rows* rows;
        bool keys, output;
        dpa_rows* to;
    } all[] = {{"q", q, false, false, &a.q},       {"k", k, true, false, &a.k},   {"v", v, true, false, &a.v},
               {"out", out, false, false, &a.out}, {"dout", dout, false, false, &a.dout},
               {"dq", dq, false, true, &a.dq},     {"dk", dk, true, true, &a.dk}, {"dv", dv, true, true, &a.dv}};
    for (const auto& x : all) {
        s = check_heads(where, x.name, x.rows, x.keys ? d->tokens_k : d->tokens, x.keys ? d->kv_heads : d->heads, d->dim, 2, x.output, kMaxRow);
        if (s != DP_OK) return s;
        *x.to = *x.rows;
    }
    for (const auto& x : all)
        for (const auto& y : all)
            if (x.output && x.rows->p && &x != &y && x.rows->p == y.rows->p && (x.keys ? d->tokens_k : d->tokens) > 0 &&
                (y.keys ? d->tokens_k : d->tokens) > 0)
                return fail(DP_ERR_INVALID_ARG, "%s: %s overlaps %s", where, x.name, y.name);
    s = check_lse(where, lse, d->tokens);
    if (s != DP_OK) return s;
    const size_t want = static_cast<size_t>(d->tokens) * static_cast<size_t>(d->heads) * 4;
    if (workspace_bytes < want)
        return fail(DP_ERR_INVALID_ARG, "%s: workspace of %zu bytes, %zu are needed", where, workspace_bytes, want);
    if (want > 0 && (!workspace || !multiple(workspace, 256)))
        return fail(DP_ERR_INVALID_ARG, "%s: the workspace must be aligned to 256 bytes", where);
    a.lse = const_cast<float*>(lse);
    a.delta = static_cast<float*>(workspace);
    return launched(dpk::launch_attention_grad(dtype, a, stream), "attention gradient launch");
}

}  // extern "C"

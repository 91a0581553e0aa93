// C ABI of the distillation loss (dploss.h): argument checks and the launch.  The
// kernel lives in distill.hip.
#include <hip/hip_runtime.h>

#include <cmath>

#include "dp_attention.h"
#include "dploss.h"
#include "plan.h"

using dpapi::fail;

namespace {

constexpr int64_t kMaxStride = int64_t{1} << 38;  // 2^21 rows stay within 63 bits

long long ll(int64_t x) { return static_cast<long long>(x); }
int64_t esize(dp_dtype d) { return d == DP_F32 ? 4 : 2; }
bool dtype_ok(dp_dtype d) { return d == DP_F32 || d == DP_F16 || d == DP_BF16; }
bool multiple(const void* p, int64_t bytes) { return reinterpret_cast<uintptr_t>(p) % static_cast<uintptr_t>(bytes) == 0; }

dp_status check_rows(const char* what, const void* p, int64_t tokens, int64_t width, int64_t ld, int64_t elem) {
    if (tokens > 0 && width > 0 && !p) return fail(DP_ERR_INVALID_ARG, "dpd_distill: %s is null", what);
    if ((ld < width && tokens > 1) || ld < 0 || ld > kMaxStride)
        return fail(DP_ERR_INVALID_ARG, "dpd_distill: %s: row stride %lld for rows of %lld", what, ll(ld), ll(width));
    if (!multiple(p, elem)) return fail(DP_ERR_INVALID_ARG, "dpd_distill: %s is not aligned to its elements", what);
    return DP_OK;
}

}  // namespace

extern "C" dp_status dpd_distill(const dpd_distill_desc* d, int64_t tokens, dp_dtype dtype, const void* logits, int64_t ld,
                                 dp_dtype teacher_dtype, const void* teacher, int64_t ld_teacher, const void* ids,
                                 int64_t ld_ids, const float* total, const void* labels, const float* weight, float* loss,
                                 void* dlogits, int64_t ld_dlogits, hipStream_t stream) {
    if (!d) return fail(DP_ERR_INVALID_ARG, "dpd_distill: null argument");
    if (tokens < 0 || tokens > DPD_MAX_TOKENS)
        return fail(DP_ERR_INVALID_ARG, "dpd_distill: %lld rows outside [0, %lld]", ll(tokens), ll(DPD_MAX_TOKENS));
    if (!dtype_ok(dtype) || !dtype_ok(teacher_dtype))
        return fail(DP_ERR_INVALID_ARG, "dpd_distill: unknown dtype %d", static_cast<int>(dtype_ok(dtype) ? teacher_dtype : dtype));
    if (d->vocab < 1 || d->vocab > DPD_MAX_VOCAB)
        return fail(DP_ERR_INVALID_ARG, "dpd_distill: a vocabulary of %lld outside [1, %lld]", ll(d->vocab), ll(DPD_MAX_VOCAB));
    if (d->top < 0 || d->top > DPD_MAX_TOP)
        return fail(DP_ERR_INVALID_ARG, "dpd_distill: lists of %d outside [0, %d]", d->top, DPD_MAX_TOP);
    if (d->id_bytes != 4 && d->id_bytes != 8) return fail(DP_ERR_INVALID_ARG, "dpd_distill: ids of %d bytes (4 or 8)", d->id_bytes);
    const float tau = static_cast<float>(d->temperature), soft = static_cast<float>(d->soft), hard = static_cast<float>(d->hard);
    const float scale = static_cast<float>(d->scale);
    if (!(tau > 0.0f) || !std::isfinite(tau * tau) || !std::isfinite(1.0f / tau))
        return fail(DP_ERR_INVALID_ARG, "dpd_distill: the temperature must be a positive binary32 number");
    if (!std::isfinite(soft) || !std::isfinite(hard) || !std::isfinite(scale))
        return fail(DP_ERR_INVALID_ARG, "dpd_distill: a factor is not finite");
    dp_status s = check_rows("logits", logits, tokens, d->vocab, ld, esize(dtype));
    if (s == DP_OK) s = check_rows("teacher", teacher, tokens, d->top, ld_teacher, esize(teacher_dtype));
    if (s == DP_OK) s = check_rows("ids", ids, tokens, d->top, ld_ids, d->id_bytes);
    if (s == DP_OK && dlogits) s = check_rows("dlogits", dlogits, tokens, d->vocab, ld_dlogits, esize(dtype));
    if (s != DP_OK) return s;
    if (dlogits && dlogits == logits && tokens > 1 && ld != ld_dlogits)
        return fail(DP_ERR_INVALID_ARG, "dpd_distill: dlogits in place of the logits needs their row stride");
    if (!multiple(total, 4) || !multiple(weight, 4) || !multiple(loss, 4) || !multiple(labels, d->id_bytes))
        return fail(DP_ERR_INVALID_ARG, "dpd_distill: total, labels, weight or loss is not aligned to its elements");
    if (tokens > 0 && !loss && !dlogits) return fail(DP_ERR_INVALID_ARG, "dpd_distill: neither loss nor dlogits is given");
    dpk::DistillArgs a{};
    a.logits = logits;
    a.teacher = teacher;
    a.ids = ids;
    a.total = total;
    a.labels = labels;
    a.weight = weight;
    a.loss = loss;
    a.dlogits = dlogits;
    a.tokens = tokens;
    a.vocab = d->vocab;
    a.ld = ld;
    a.ld_teacher = ld_teacher;
    a.ld_ids = ld_ids;
    a.ld_dlogits = ld_dlogits;
    a.top = d->top;
    a.id_bytes = d->id_bytes;
    a.temperature = tau;
    a.soft = soft;
    a.hard = hard;
    a.scale = scale;
    const hipError_t e = dpk::launch_distill(dtype, teacher_dtype, a, stream);
    return e == hipSuccess ? DP_OK : dpapi::hip_fail(e, "distillation launch");
}

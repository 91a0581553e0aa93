// gfx950 kernel of the norms around a block, forward:
//   u = n(y) w_post + b_post,  s = alpha h + gate u,  x = n(s) w_pre + b_pre
// with n(v) the row v normalised (centred or not).
//
// Bound by HBM: two rows read and two written per token.  `NT` threads hold a
// row in registers, 8 consecutive elements each `NV` times, so the passes over
// it after the load cost no memory traffic, and the statistics are sums of
// deviations in binary32, never differences of sums (the mean is divided, so a
// row of equal values has none).  Rows up to 1024 elements take one wave and no
// barrier.  A workgroup keeps the weights of its columns in registers, walks
// over rows, and loads the next row before it computes the current one.  16384
// rows of 4096 f16 with both norms and the gate take 101 us, 5.3 TB/s; rows of
// 4095, which start at any element, 1.25 times as long.  With biases 8192 bf16 rows
// of 4096 take 53 us instead of 51, with the mean subtracted 55; rows of 8192 97, 111
// and 131 us.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "block_norm.h"
#include "dp_device.h"
#include "dp_layers.h"

namespace dpk {
namespace {

struct NormArgs {
    const void *h, *y;
    void *s, *x;
    int64_t ld_h, ld_y, ld_s, ld_x;
    int64_t tokens;
    int32_t dim;
    float eps, alpha;
    Weights w;
};

template <dp_dtype DT, dp_dtype PT, int NT, int NV, int VW, bool kCentered, bool kBias, bool kPost>
__global__ void __launch_bounds__(block_of(NT)) k_block_norm(NormArgs a) {
    constexpr int kRows = block_of(NT) / NT, kStep = VW * NT;
    __shared__ float lds[sum_scratch(NT)];
    int turn = 0;
    const int lane = threadIdx.x % NT, c0 = VW * lane;
    const float dim = static_cast<float>(a.dim), inv = 1.0f / dim;
    const bool has_gate = a.w.gate != nullptr, has_x = a.x != nullptr;
    Column<PT, NV, VW> post_w, post_b, gate, pre_w, pre_b;
    if constexpr (kPost) post_w.load(a.w.post_w, c0, kStep, a.dim);
    if constexpr (kPost && kBias) post_b.load(a.w.post_b, c0, kStep, a.dim);
    if (has_gate) gate.load(a.w.gate, c0, kStep, a.dim);
    if (has_x) {
        pre_w.load(a.w.pre_w, c0, kStep, a.dim);
        if constexpr (kBias) pre_b.load(a.w.pre_b, c0, kStep, a.dim);
    }
    // a workgroup's rows: in every turn all its rows run (the last turn's
    // beyond the end are computed on zeros and not stored), so that barriers meet
    const int64_t stride = static_cast<int64_t>(gridDim.x) * kRows;
    int64_t row = static_cast<int64_t>(blockIdx.x) * kRows + threadIdx.x / NT;
    int64_t base = static_cast<int64_t>(blockIdx.x) * kRows;
    Raw<DT, VW> nh[NV], ny[NV];
    auto fetch = [&](int64_t t) {
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const int c = c0 + k * kStep;
            const int valid = t < a.tokens ? valid_of<VW>(a.dim, c) : 0;
            nh[k] = load_raw<DT, VW>(a.h, t * a.ld_h + c, valid, a.dim >= VW);
            ny[k] = load_raw<DT, VW>(a.y, t * a.ld_y + c, valid, a.dim >= VW);
        }
    };
    fetch(row);
    for (; base < a.tokens; base += stride, row += stride) {
        float h[NV][VW], u[NV][VW];
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const int valid = row < a.tokens ? valid_of<VW>(a.dim, c0 + k * kStep) : 0;
            settle<DT, VW>(nh[k], valid, a.dim >= VW);
            settle<DT, VW>(ny[k], valid, a.dim >= VW);
            expand<DT, VW>(nh[k], h[k]);
            expand<DT, VW>(ny[k], u[k]);
        }
        if (base + stride < a.tokens) fetch(row + stride);
        if constexpr (kPost) {
            if constexpr (kCentered) {
                float m[1] = {0.0f};
#pragma unroll
                for (int k = 0; k < NV; ++k)
#pragma unroll
                    for (int j = 0; j < VW; ++j) m[0] += u[k][j];
                row_sum<NT>(m, lds, turn);
                const float mean = m[0] / dim;
#pragma unroll
                for (int k = 0; k < NV; ++k)
#pragma unroll
                    for (int j = 0; j < VW; ++j)
                        u[k][j] = j < valid_of<VW>(a.dim, c0 + k * kStep) ? u[k][j] - mean : 0.0f;
            }
            float q[1] = {0.0f};
#pragma unroll
            for (int k = 0; k < NV; ++k)
#pragma unroll
                for (int j = 0; j < VW; ++j) q[0] += u[k][j] * u[k][j];
            row_sum<NT>(q, lds, turn);
            const float r = 1.0f / sqrtf(q[0] * inv + a.eps);
#pragma unroll
            for (int k = 0; k < NV; ++k) {
                float w[VW], b[VW];
                expand<PT, VW>(post_w.q[k], w);
                if constexpr (kBias) expand<PT, VW>(post_b.q[k], b);
#pragma unroll
                for (int j = 0; j < VW; ++j) u[k][j] = u[k][j] * r * w[j] + (kBias ? b[j] : 0.0f);
            }
        }
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            if (has_gate) {
                float w[VW];
                expand<PT, VW>(gate.q[k], w);
#pragma unroll
                for (int j = 0; j < VW; ++j) u[k][j] *= w[j];
            }
            const int c = c0 + k * kStep;
            const int valid = row < a.tokens ? valid_of<VW>(a.dim, c) : 0;
#pragma unroll
            for (int j = 0; j < VW; ++j) h[k][j] = a.alpha * h[k][j] + u[k][j];
            store_n<DT, VW>(a.s, row * a.ld_s + c, valid, h[k]);
        }
        if (!has_x) continue;
        if constexpr (kCentered) {
            float m[1] = {0.0f};
#pragma unroll
            for (int k = 0; k < NV; ++k)
#pragma unroll
                for (int j = 0; j < VW; ++j) m[0] += h[k][j];
            row_sum<NT>(m, lds, turn);
            const float mean = m[0] / dim;
#pragma unroll
            for (int k = 0; k < NV; ++k)
#pragma unroll
                for (int j = 0; j < VW; ++j)
                    h[k][j] = j < valid_of<VW>(a.dim, c0 + k * kStep) ? h[k][j] - mean : 0.0f;
        }
        float q[1] = {0.0f};
#pragma unroll
        for (int k = 0; k < NV; ++k)
#pragma unroll
            for (int j = 0; j < VW; ++j) q[0] += h[k][j] * h[k][j];
        row_sum<NT>(q, lds, turn);
        const float r = 1.0f / sqrtf(q[0] * inv + a.eps);
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            float w[VW], b[VW];
            expand<PT, VW>(pre_w.q[k], w);
            if constexpr (kBias) expand<PT, VW>(pre_b.q[k], b);
#pragma unroll
            for (int j = 0; j < VW; ++j) h[k][j] = h[k][j] * r * w[j] + (kBias ? b[j] : 0.0f);
            const int c = c0 + k * kStep;
            const int valid = row < a.tokens ? valid_of<VW>(a.dim, c) : 0;
            store_n<DT, VW>(a.x, row * a.ld_x + c, valid, h[k]);
        }
    }
}

Shape shape_of(int64_t dim) {
    if (dim <= 512) return {64, 1, 8};
    if (dim <= 1024) return {64, 2, 8};
    if (dim <= 2048) return {256, 1, 8};
    if (dim <= 4096) return {256, 2, 8};
    return {512, 2, 8};
}

#define DP_SHAPES(GO)                                  \
    if (sh.nt == 64 && sh.nv == 1) GO(64, 1, 8)        \
    else if (sh.nt == 64) GO(64, 2, 8)                 \
    else if (sh.nt == 256 && sh.nv == 1) GO(256, 1, 8) \
    else if (sh.nt == 256) GO(256, 2, 8)               \
    else GO(512, 2, 8)

template <dp_dtype DT, dp_dtype PT, bool kCentered, bool kBias, bool kPost>
void forward(const NormArgs& a, hipStream_t stream) {
    const Shape sh = shape_of(a.dim);
    const int64_t rows = block_of(sh.nt) / sh.nt, want = (a.tokens + rows - 1) / rows;
    const dim3 grid(static_cast<unsigned>(want < 4096 ? want : 4096));
#define GO(T, V, W) \
    { hipLaunchKernelGGL((k_block_norm<DT, PT, T, V, W, kCentered, kBias, kPost>), grid, dim3(block_of(T)), 0, stream, a); }
    DP_SHAPES(GO)
#undef GO
}

}  // namespace

hipError_t launch_block_norm(dp_dtype dt, dp_dtype pdt, const BlockNorm& b, int64_t tokens, const void* h,
                             int64_t ld_h, const void* y, int64_t ld_y, void* s, int64_t ld_s, void* x, int64_t ld_x,
                             hipStream_t stream) {
    if (tokens == 0) return hipSuccess;
    NormArgs a{h,    y,    s,     x, ld_h, ld_y, ld_s, ld_x, tokens, static_cast<int32_t>(b.dim), b.eps, b.alpha,
               weights_of(b)};
    const bool post = b.weight[0] != nullptr;
#define GO(D, P, C, B, O) forward<D, P, C, B, O>(a, stream)
    DP_KINDS(GO);
#undef GO
    return hipGetLastError();
}

}  // namespace dpk

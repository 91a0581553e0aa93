// gfx950 kernels of the norms around a block, backward, with the gradients of
// weights and gate.
//
// Mathematics.  Let d = s - mean(s) (or s), r = 1 / sqrt(mean(d^2) + eps),
// n = d r, e = dx w_pre.  Then
//   t = ds + r (e - [mean(e)] - n mean(e n)),  dh = alpha t,
// the bracket only with the mean subtracted, and the same step on y with e =
// t gate w_post gives dy.  Column sums over the tokens: C = sum dx n(s) and E =
// sum dx are the gradients of w_pre and b_pre.  With A = sum t n(y) and B =
// sum t the others follow per column: dw_post = gate A, db_post = gate B, dgate
// = w_post A + b_post B, so a thread keeps four sums per column instead of
// five; without biases and without the mean, where nothing takes E and B, two.
//
// Bound by HBM: four rows read and two written per token, all of them held in
// registers as in the forward.  The sums of a row that do not depend on each
// other go through one reduction (RMS: 2 a row, centred: 3).  The column sums
// of a workgroup go to the workspace, and a second launch adds the
// workgroups' sums in a fixed order, so the bits depend on the sizes alone.
// 8191 rows of 4096 f16 with both norms and the gate take 83 us, 4.8 TB/s, and
// the second launch 7 us.  With biases, four sums instead of two, 8192 bf16 rows of
// 4096 take 98 us with the second launch instead of 92, and 113 with the mean
// subtracted.  Beyond 4096 elements four sums of a thread's 16 columns do not fit
// 256 registers: 8192 bf16 rows of 8192 take 171 us with two sums, 400 with four (35
// registers spilled), 463 with the mean (39).
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "block_norm.h"
#include "dp_device.h"
#include "dp_layers.h"

namespace dpk {
namespace {

// ---- backward ------------------------------------------------------------------
struct GradArgs {
    dpl_norm_rows rows[DP_MAX_REPLICAS];
    float* part;  // [n][groups][quantities][dim]
    int64_t tokens, ld;
    int32_t dim;
    float eps, alpha;
    Weights w;
};

// Column sums a workgroup leaves: C = sum dx n(s), A = sum t n(y) (t y without
// a post norm), and in the form with biases E = sum dx, B = sum t.
template <bool kBias>
constexpr int kSums = kBias ? 4 : 2;

template <dp_dtype DT, dp_dtype PT, int NT, int NV, int VW, bool kCentered, bool kBias, bool kPost>
__global__ void __launch_bounds__(block_of(NT)) k_block_grad(GradArgs a) {
    constexpr int kRows = block_of(NT) / NT, kStep = VW * NT, Q = kSums<kBias>;
    __shared__ float lds[sum_scratch(NT)];
    __shared__ float fold[kRows > 1 ? kRows - 1 : 1][kRows > 1 ? NT * VW * NV : 1];
    int turn = 0;
    const dpl_norm_rows p = a.rows[blockIdx.y];
    const int lane = threadIdx.x % NT, c0 = VW * lane;
    const float dim = static_cast<float>(a.dim), inv = 1.0f / dim;
    const bool has_gate = a.w.gate != nullptr, has_x = p.dx != nullptr, has_ds = p.ds != nullptr;
    const bool has_y = kPost || has_gate;
    Column<PT, NV, VW> post_w, gate, pre_w;
    if constexpr (kPost) post_w.load(a.w.post_w, c0, kStep, a.dim);
    if (has_gate) gate.load(a.w.gate, c0, kStep, a.dim);
    if (has_x) pre_w.load(a.w.pre_w, c0, kStep, a.dim);
    float sum[Q][NV][VW];
#pragma unroll
    for (int q = 0; q < Q; ++q)
#pragma unroll
        for (int k = 0; k < NV; ++k)
#pragma unroll
            for (int j = 0; j < VW; ++j) sum[q][k][j] = 0.0f;

    const int64_t stride = static_cast<int64_t>(gridDim.x) * kRows;
    int64_t base = static_cast<int64_t>(blockIdx.x) * kRows;
    int64_t row = base + threadIdx.x / NT;
    Raw<DT, VW> ns[NV], ny[NV], nx[NV], nd[NV];
    auto fetch = [&](int64_t t) {
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const int c = c0 + k * kStep;
            const int valid = t < a.tokens ? valid_of<VW>(a.dim, c) : 0;
            const int64_t at = t * a.ld + c;
            ns[k] = load_raw<DT, VW>(p.s, at, has_x ? valid : 0, a.dim >= VW);
            nx[k] = load_raw<DT, VW>(p.dx, at, has_x ? valid : 0, a.dim >= VW);
            ny[k] = load_raw<DT, VW>(p.y, at, has_y ? valid : 0, a.dim >= VW);
            nd[k] = load_raw<DT, VW>(p.ds, at, has_ds ? valid : 0, a.dim >= VW);
        }
    };
    fetch(row);
    for (; base < a.tokens; base += stride, row += stride) {
        float s[NV][VW], y[NV][VW], e[NV][VW], t[NV][VW];
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const int valid = row < a.tokens ? valid_of<VW>(a.dim, c0 + k * kStep) : 0;
            settle<DT, VW>(ns[k], valid, a.dim >= VW);
            settle<DT, VW>(nx[k], valid, a.dim >= VW);
            settle<DT, VW>(ny[k], valid, a.dim >= VW);
            settle<DT, VW>(nd[k], valid, a.dim >= VW);
            expand<DT, VW>(ns[k], s[k]);
            expand<DT, VW>(nx[k], e[k]);
            expand<DT, VW>(ny[k], y[k]);
            expand<DT, VW>(nd[k], t[k]);
        }
        if (base + stride < a.tokens) fetch(row + stride);
        if constexpr (kCentered) {
            float m[2] = {0.0f, 0.0f};
#pragma unroll
            for (int k = 0; k < NV; ++k)
#pragma unroll
                for (int j = 0; j < VW; ++j) {
                    m[0] += s[k][j];
                    m[1] += y[k][j];
                }
            row_sum<NT>(m, lds, turn);
            const float mean_s = m[0] / dim, mean_y = m[1] / dim;
#pragma unroll
            for (int k = 0; k < NV; ++k)
#pragma unroll
                for (int j = 0; j < VW; ++j) {
                    const bool in = j < valid_of<VW>(a.dim, c0 + k * kStep);
                    s[k][j] = in ? s[k][j] - mean_s : 0.0f;
                    if constexpr (kPost) y[k][j] = in ? y[k][j] - mean_y : 0.0f;
                }
        }
        // sums of s^2 and e s, of e with the mean subtracted, of y^2 with a post norm (e = dx w_pre)
        constexpr int kE = 2, kY = 2 + kCentered;
        float v[2 + kCentered + kPost] = {};
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            float w[VW];
            expand<PT, VW>(pre_w.q[k], w);
#pragma unroll
            for (int j = 0; j < VW; ++j) {
                const float f = has_x ? e[k][j] * w[j] : 0.0f;
                v[0] += s[k][j] * s[k][j];
                v[1] += f * s[k][j];
                if constexpr (kCentered) v[kE] += f;
                if constexpr (kPost) v[kY] += y[k][j] * y[k][j];
            }
        }
        row_sum<NT>(v, lds, turn);
        const float r = 1.0f / sqrtf(v[0] * inv + a.eps), mean_en = v[1] * r * inv;
        float ry = 1.0f, mean_e = 0.0f;
        if constexpr (kPost) ry = 1.0f / sqrtf(v[kY] * inv + a.eps);
        if constexpr (kCentered) mean_e = v[kE] * inv;
        if (has_x) {
#pragma unroll
            for (int k = 0; k < NV; ++k) {
                float w[VW];
                expand<PT, VW>(pre_w.q[k], w);
#pragma unroll
                for (int j = 0; j < VW; ++j) {
                    const float n = s[k][j] * r;
                    sum[0][k][j] += e[k][j] * n;
                    if constexpr (kBias) sum[2][k][j] += e[k][j];
                    t[k][j] += r * (e[k][j] * w[j] - mean_e - n * mean_en);
                }
            }
        }
        // t is the gradient of s; columns beyond the row's end hold what is never stored
        float g[2] = {0.0f, 0.0f};
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            float w[VW], f[VW];
            const int c = c0 + k * kStep, valid = row < a.tokens ? valid_of<VW>(a.dim, c) : 0;
#pragma unroll
            for (int j = 0; j < VW; ++j) f[j] = a.alpha * t[k][j];
            if (p.dh) store_n<DT, VW>(p.dh, row * a.ld + c, valid, f);
            if constexpr (kBias) {
#pragma unroll
                for (int j = 0; j < VW; ++j) sum[3][k][j] += j < valid ? t[k][j] : 0.0f;
            }
            if (kPost || has_gate) {
#pragma unroll
                for (int j = 0; j < VW; ++j) sum[1][k][j] += t[k][j] * (kPost ? y[k][j] * ry : y[k][j]);
            }
            if (has_gate) {
                expand<PT, VW>(gate.q[k], w);
#pragma unroll
                for (int j = 0; j < VW; ++j) t[k][j] *= w[j];
            }
            if constexpr (kPost) {
                expand<PT, VW>(post_w.q[k], w);
#pragma unroll
                for (int j = 0; j < VW; ++j) {
                    t[k][j] *= w[j];
                    g[0] += t[k][j] * y[k][j];
                    g[1] += j < valid_of<VW>(a.dim, c) ? t[k][j] : 0.0f;
                }
            }
        }
        if (!p.dy) continue;
        if constexpr (kPost) {
            row_sum<NT>(g, lds, turn);
            const float mean_tn = g[0] * ry * inv, mean_t = kCentered ? g[1] * inv : 0.0f;
#pragma unroll
            for (int k = 0; k < NV; ++k)
#pragma unroll
                for (int j = 0; j < VW; ++j) t[k][j] = ry * (t[k][j] - mean_t - y[k][j] * ry * mean_tn);
        }
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const int c = c0 + k * kStep, valid = row < a.tokens ? valid_of<VW>(a.dim, c) : 0;
            store_n<DT, VW>(p.dy, row * a.ld + c, valid, t[k]);
        }
    }
    // the rows' sums of this workgroup, in row order, then one slot of the workspace
    float* out = a.part + (static_cast<int64_t>(blockIdx.y) * gridDim.x + blockIdx.x) * Q * a.dim;
#pragma unroll
    for (int q = 0; q < Q; ++q) {
        if constexpr (kRows > 1) {
            __syncthreads();
            const int w = threadIdx.x / NT;
            if (w > 0)
#pragma unroll
                for (int k = 0; k < NV; ++k)
#pragma unroll
                    for (int j = 0; j < VW; ++j) fold[w - 1][(k * VW + j) * NT + lane] = sum[q][k][j];
            __syncthreads();
            if (w == 0)
                for (int i = 0; i < kRows - 1; ++i)
#pragma unroll
                    for (int k = 0; k < NV; ++k)
#pragma unroll
                        for (int j = 0; j < VW; ++j) sum[q][k][j] += fold[i][(k * VW + j) * NT + lane];
        }
        if (threadIdx.x < NT)
#pragma unroll
            for (int k = 0; k < NV; ++k)
                store_n<DP_F32, VW>(out + q * a.dim, c0 + k * kStep, valid_of<VW>(a.dim, c0 + k * kStep), sum[q][k]);
    }
}

struct JoinArgs {
    const float* part;
    float* acc[5][DP_MAX_REPLICAS];  // post_w, post_b, gate, pre_w, pre_b; null: none
    bool overwrite[5];
    int32_t dim, groups;
    Weights w;
};

constexpr int kJoinColumns = 32, kJoinLanes = 16;

template <dp_dtype PT>
__device__ __forceinline__ float weight_at(const void* p, int c, float none) {
    return p ? load1<PT>(p, c) : none;
}

// Adds the workgroups' sums of 32 columns of one replica: 16 threads a column
// each take every 16th group, then their sums are added in order.
template <dp_dtype PT, int Q>
__global__ void __launch_bounds__(kJoinColumns* kJoinLanes) k_block_join(JoinArgs a) {
    __shared__ float lds[Q][kJoinLanes][kJoinColumns];
    const int col = threadIdx.x % kJoinColumns, lane = threadIdx.x / kJoinColumns;
    const int c = blockIdx.x * kJoinColumns + col, r = blockIdx.y;
    const float* part = a.part + static_cast<int64_t>(r) * a.groups * Q * a.dim + c;
    float s[Q] = {};
    if (c < a.dim)
#pragma unroll 4
        for (int g = lane; g < a.groups; g += kJoinLanes)
#pragma unroll
            for (int q = 0; q < Q; ++q) s[q] += part[(static_cast<int64_t>(g) * Q + q) * a.dim];
#pragma unroll
    for (int q = 0; q < Q; ++q) lds[q][lane][col] = s[q];
    __syncthreads();
    if (lane != 0 || c >= a.dim) return;
    float total[4] = {};
#pragma unroll
    for (int q = 0; q < Q; ++q)
#pragma unroll
        for (int i = 0; i < kJoinLanes; ++i) total[q] += lds[q][i][col];
    const float C = total[0], A = total[1], E = total[2], B = total[3];
    const float gate = weight_at<PT>(a.w.gate, c, 1.0f);
    const float grads[5] = {gate * A, gate * B,
                            a.w.post_w ? weight_at<PT>(a.w.post_w, c, 1.0f) * A + weight_at<PT>(a.w.post_b, c, 0.0f) * B : A,
                            C, E};
#pragma unroll
    for (int i = 0; i < 5; ++i)
        if (a.acc[i][r]) a.acc[i][r][c] = a.overwrite[i] ? grads[i] : a.acc[i][r][c] + grads[i];
}

// One wave a row up to 1024 elements needs no barriers.  32768 rows of 768,
// centred, bf16: 128 threads with 8 elements each took 112 us, one wave with 2 x
// 8 took 94 us and with 3 x 4 (every lane busy, 196 registers) 77 us; forcing a
// third wave a SIMD spilled 29 registers and took 92 to 114 us.  Without
// branches around its loads the last form takes 57 us, 4.4 TB/s of the five
// rows a token that it moves (y is read only for a post norm or a gate).
Shape shape_of(int64_t dim) {
    if (dim <= 512) return {64, 1, 8};
    if (dim <= 768) return {64, 3, 4};
    if (dim <= 1024) return {64, 2, 8};
    if (dim <= 2048) return {256, 1, 8};
    if (dim <= 4096) return {512, 1, 8};
    return {512, 2, 8};
}

#define DP_SHAPES(GO)                           \
    if (sh.nt == 64 && sh.nv == 1) GO(64, 1, 8) \
    else if (sh.vw == 4) GO(64, 3, 4)           \
    else if (sh.nt == 64) GO(64, 2, 8)          \
    else if (sh.nt == 256) GO(256, 1, 8)        \
    else if (sh.nv == 1) GO(512, 1, 8)          \
    else GO(512, 2, 8)

// Workgroups of one replica's backward: as many as the chip holds at a time
// (two of 4 one-wave rows a CU; 1024 threads a CU else), shared by the replicas.
// Twice as many for the one-wave rows costs 4% of the pass, and the second
// launch doubles.
int64_t groups_of(int64_t dim, int64_t tokens, int n) {
    const int nt = shape_of(dim).nt;
    const int64_t most = (256 * (nt == 64 ? 512 : 1024) / block_of(nt) + n - 1) / n, rows = block_of(nt) / nt;
    const int64_t want = (tokens + rows - 1) / rows;
    return want < most ? want : most;
}

template <dp_dtype DT, dp_dtype PT, bool kCentered, bool kBias, bool kPost>
void backward(const GradArgs& a, int groups, int n, hipStream_t stream) {
    const Shape sh = shape_of(a.dim);
    const dim3 grid(static_cast<unsigned>(groups), static_cast<unsigned>(n));
#define GO(T, V, W) \
    { hipLaunchKernelGGL((k_block_grad<DT, PT, T, V, W, kCentered, kBias, kPost>), grid, dim3(block_of(T)), 0, stream, a); }
    DP_SHAPES(GO)
#undef GO
}

}  // namespace

size_t block_norm_workspace(const BlockNorm& b, int64_t tokens, int n) {
    return static_cast<size_t>(4) * n * groups_of(b.dim, tokens, n) * (b.centered || b.bias ? 4 : 2) * b.dim;
}

hipError_t launch_block_grad(dp_dtype dt, dp_dtype pdt, const BlockNorm& b, int64_t tokens, int n,
                             const dpl_norm_rows* rows, int64_t ld, float* const* acc, const int* at,
                             const bool* overwrite, void* workspace, hipStream_t stream) {
    GradArgs a{};
    for (int r = 0; r < n; ++r) a.rows[r] = rows[r];
    a.part = static_cast<float*>(workspace);
    a.tokens = tokens;
    a.ld = ld;
    a.dim = static_cast<int32_t>(b.dim);
    a.eps = b.eps;
    a.alpha = b.alpha;
    a.w = weights_of(b);
    const bool post = b.weight[0] != nullptr;
    const int groups = static_cast<int>(groups_of(b.dim, tokens, n));
    if (tokens > 0) {
#define GO(D, P, C, B, O) backward<D, P, C, B, O>(a, groups, n, stream)
        DP_KINDS(GO);
#undef GO
        hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    JoinArgs j{};
    bool any = false;
    for (int i = 0; i < 5; ++i) {
        if (at[i] < 0) continue;
        any = true;
        j.overwrite[i] = overwrite[at[i]];
        for (int r = 0; r < n; ++r) j.acc[i][r] = acc[at[i] * n + r];
    }
    if (!any) return hipSuccess;
    j.part = a.part;
    j.dim = a.dim;
    j.groups = tokens > 0 ? groups : 0;
    j.w = a.w;
    const dim3 grid(static_cast<unsigned>((b.dim + kJoinColumns - 1) / kJoinColumns), static_cast<unsigned>(n));
#define GO(P, S) hipLaunchKernelGGL((k_block_join<P, S>), grid, dim3(kJoinColumns * kJoinLanes), 0, stream, j)
    const bool four = b.centered || b.bias;
    if (pdt == DP_BF16 && four) GO(DP_BF16, 4);
    else if (pdt == DP_BF16) GO(DP_BF16, 2);
    else if (four) GO(DP_F16, 4);
    else GO(DP_F16, 2);
#undef GO
    return hipGetLastError();
}

}  // namespace dpk

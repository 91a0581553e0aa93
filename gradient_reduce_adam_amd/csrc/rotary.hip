// gfx950 kernel of rotary positions on several axes, forward and back.
//
// Every head of a token turns by the same angles, so a workgroup takes some tokens
// whole: its threads first compute the tokens' cosines and sines, once, into LDS,
// the angle as a product in binary64 reduced by whole turns there, and then turn
// pieces of eight pairs of every head.  Memory bound: 16383 tokens of 40 heads of 128,
// f16, 62 us, 5.4 TB/s of the 336 MB read and written (a large copy 4.9; with one piece of a
// thread on its way and ordinary stores 69 us).
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "dp_attention.h"
#include "dp_device.h"

namespace dpk {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxTokens = 16;  // of a workgroup

// The units of a thread, kThreads apart: unit u of head h of token t, without a
// division for each.
struct Walk {
    int u, h, t, step_u, step_h, step_t, units, heads;
    __device__ __forceinline__ Walk(int units_, int heads_) : units(units_), heads(heads_) {
        const int head = threadIdx.x / units, step = kThreads / units;
        u = threadIdx.x - head * units;
        t = head / heads;
        h = head - t * heads;
        step_u = kThreads % units;
        step_t = step / heads;
        step_h = step - step_t * heads;
    }
    __device__ __forceinline__ void next() {
        u += step_u;
        h += step_h + (u >= units ? 1 : 0);
        u -= u >= units ? units : 0;
        t += step_t + (h >= heads ? 1 : 0);
        h -= h >= heads ? heads : 0;
    }
};

// kWhole: every piece has eight pairs, so that no load lies behind a branch and a
// thread has several pieces on their way.
template <dp_dtype DT, bool kWhole, bool kInterleaved, bool kOnce>
__global__ void __launch_bounds__(kThreads) k_rotary(RotaryArgs a, int tokens) {
    constexpr int kBatch = kWhole ? (DT == DP_F32 ? 2 : 4) : 1;
    extern __shared__ f32x2 turn[];  // [tokens][pairs]: cosine, sine
    const int64_t first = static_cast<int64_t>(blockIdx.x) * tokens;
    const int here = static_cast<int>(a.tokens - first < tokens ? a.tokens - first : tokens);
    const int P = a.pairs;
    for (int i = threadIdx.x; i < here * P; i += kThreads) {
        const int t = i / P, p = i - t * P;
        const int64_t where = (first + t) * a.position_ld + a.axis[p] * a.position_axis;
        const double x = a.frequency[p] * static_cast<double>(a.position_bytes == 4 ? gload<int32_t>(a.positions, where)
                                                                                       : gload<int64_t>(a.positions, where));
        const double n = __builtin_rint(x * 0.15915494309189533577);  // whole turns, 2 pi in two parts
        const float r = static_cast<float>(__builtin_fma(-n, 2.4492935982947064e-16, __builtin_fma(-n, 6.283185307179586477, x)));
        float s, c;
        sincosf(r, &s, &c);
        turn[i] = f32x2{c, a.inverse ? -s : s};
    }
    __syncthreads();
    const int pieces = (P + 7) / 8;
    for (int k = 0; k < a.count; ++k) {
        const dpa_rotary_rows& m = a.rows[k];
        if (pieces > 0) {
            for (Walk w(pieces, m.heads); w.t < here;) {
                float lo[kBatch][8], hi[kBatch][8];  // interleaved: the first and last four pairs
                int64_t y[kBatch];
                int at[kBatch], valid[kBatch];
#pragma unroll
                for (int b = 0; b < kBatch; ++b) {
                    // past the last token the last unit's place is read, and not written
                    const bool there = w.t < here;
                    const int t = there ? w.t : here - 1, p = 8 * w.u;
                    const int64_t x = (first + t) * m.x.ld + w.h * m.x.head;
                    y[b] = (first + t) * m.y.ld + w.h * m.y.head;
                    at[b] = t * P + p;
                    const int left = kWhole ? 8 : P - p;
                    if constexpr (kInterleaved) {
                        load_n<DT, 8>(m.x.p, x + 2 * p, kWhole ? 8 : 2 * left, lo[b]);
                        load_n<DT, 8>(m.x.p, x + 2 * p + 8, kWhole ? 8 : 2 * left - 8, hi[b]);
                        y[b] += 2 * p;
                    } else {
                        load_n<DT, 8>(m.x.p, x + p, left, lo[b]);
                        load_n<DT, 8>(m.x.p, x + P + p, left, hi[b]);
                        y[b] += p;
                    }
                    valid[b] = there ? left : 0;
                    w.next();
                }
#pragma unroll
                for (int b = 0; b < kBatch; ++b) {
                    float l2[8], h2[8];
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        const f32x2 q = kWhole || j < valid[b] ? turn[at[b] + j] : f32x2{1.0f, 0.0f};
                        float& x0 = kInterleaved ? (j < 4 ? lo[b][(2 * j) & 7] : hi[b][(2 * j) & 7]) : lo[b][j];
                        float& x1 = kInterleaved ? (j < 4 ? lo[b][(2 * j + 1) & 7] : hi[b][(2 * j + 1) & 7]) : hi[b][j];
                        const float y0 = __builtin_fmaf(x0, q[0], -(x1 * q[1])), y1 = __builtin_fmaf(x0, q[1], x1 * q[0]);
                        (kInterleaved ? (j < 4 ? l2[(2 * j) & 7] : h2[(2 * j) & 7]) : l2[j]) = y0;
                        (kInterleaved ? (j < 4 ? l2[(2 * j + 1) & 7] : h2[(2 * j + 1) & 7]) : h2[j]) = y1;
                    }
                    if (kWhole && valid[b] == 0) continue;
                    if constexpr (kInterleaved) {
                        store_n<DT, 8, kOnce>(m.y.p, y[b], kWhole ? 8 : 2 * valid[b], l2);
                        store_n<DT, 8, kOnce>(m.y.p, y[b] + 8, kWhole ? 8 : 2 * valid[b] - 8, h2);
                    } else {
                        store_n<DT, 8, kOnce>(m.y.p, y[b], kWhole ? 8 : valid[b], l2);
                        store_n<DT, 8, kOnce>(m.y.p, y[b] + P, kWhole ? 8 : valid[b], h2);
                    }
                }
            }
        }
        const int rest = (a.dim - 2 * P + 7) / 8;  // elements that do not turn
        if (rest > 0 && m.x.p != m.y.p) {
            for (Walk w(rest, m.heads); w.t < here; w.next()) {
                const int d = 2 * P + 8 * w.u;
                float v[8];
                load_n<DT, 8>(m.x.p, (first + w.t) * m.x.ld + w.h * m.x.head + d, a.dim - d, v);
                store_n<DT, 8, kOnce>(m.y.p, (first + w.t) * m.y.ld + w.h * m.y.head + d, a.dim - d, v);
            }
        }
    }
}

template <dp_dtype DT, bool kWhole, bool kInterleaved>
void launch_kind(const RotaryArgs& a, int tokens, dim3 grid, size_t lds, hipStream_t stream) {
    if (a.once) hipLaunchKernelGGL((k_rotary<DT, kWhole, kInterleaved, true>), grid, dim3(kThreads), lds, stream, a, tokens);
    else hipLaunchKernelGGL((k_rotary<DT, kWhole, kInterleaved, false>), grid, dim3(kThreads), lds, stream, a, tokens);
}

template <dp_dtype DT>
void launch_type(const RotaryArgs& a, int tokens, dim3 grid, size_t lds, hipStream_t stream) {
    if (a.pairs % 8 == 0 && a.interleaved) launch_kind<DT, true, true>(a, tokens, grid, lds, stream);
    else if (a.pairs % 8 == 0) launch_kind<DT, true, false>(a, tokens, grid, lds, stream);
    else if (a.interleaved) launch_kind<DT, false, true>(a, tokens, grid, lds, stream);
    else launch_kind<DT, false, false>(a, tokens, grid, lds, stream);
}

}  // namespace

hipError_t launch_rotary(dp_dtype dt, const RotaryArgs& a, hipStream_t stream) {
    if (a.tokens == 0) return hipSuccess;
    // tokens of a workgroup: enough for a thread to have an angle, as long as there
    // are eight workgroups for each CU
    int64_t tokens = a.pairs > 0 ? kThreads / a.pairs : kMaxTokens;
    if (tokens > a.tokens / 2048) tokens = a.tokens / 2048;
    tokens = tokens < 1 ? 1 : tokens > kMaxTokens ? kMaxTokens : tokens;
    if (a.tokens / tokens >= int64_t{1} << 23) tokens *= 2;  // a launch has fewer than 2^32 threads
    const dim3 grid(static_cast<unsigned>((a.tokens + tokens - 1) / tokens));
    const size_t lds = static_cast<size_t>(tokens) * a.pairs * sizeof(f32x2);
    const int n = static_cast<int>(tokens);
    if (dt == DP_F32) launch_type<DP_F32>(a, n, grid, lds, stream);
    else if (dt == DP_F16) launch_type<DP_F16>(a, n, grid, lds, stream);
    else launch_type<DP_BF16>(a, n, grid, lds, stream);
    return hipGetLastError();
}

}  // namespace dpk

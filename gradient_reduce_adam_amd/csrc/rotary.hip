// gfx950 kernel of rotary positions on several axes, forward and back.
//
// Every head of a token turns by the same angles, so a workgroup takes some tokens
// whole: its threads first compute the tokens' cosines and sines, once, into LDS,
// the angle as a product in binary64 reduced by whole turns there, and then turn
// pieces of eight pairs of every head.  Memory bound.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "dp_attention.h"
#include "dp_device.h"

namespace dpk {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxTokens = 16;  // of a workgroup

template <dp_dtype DT>
__global__ void __launch_bounds__(kThreads) k_rotary(RotaryArgs a, int tokens) {
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
    const int pieces = (P + 7) / 8, rest = a.dim - 2 * P;
    for (int k = 0; k < a.count; ++k) {
        const dpa_rotary_rows& m = a.rows[k];
        const bool copy = m.x.p != m.y.p;
        const int units = pieces + (copy ? (rest + 7) / 8 : 0);  // of a head
        for (int i = threadIdx.x; i < here * m.heads * units; i += kThreads) {
            const int head = i / units, u = i - head * units;  // of all the tokens' heads
            const int t = head / m.heads, h = head - t * m.heads;
            const int64_t x = (first + t) * m.x.ld + h * m.x.head, y = (first + t) * m.y.ld + h * m.y.head;
            if (u >= pieces) {  // elements that do not turn
                const int d = 2 * P + 8 * (u - pieces);
                float v[8];
                load_n<DT, 8>(m.x.p, x + d, a.dim - d, v);
                store_n<DT, 8>(m.y.p, y + d, a.dim - d, v);
                continue;
            }
            const int p = 8 * u, valid = P - p;
            const f32x2* cs = turn + t * P + p;
            float lo[8], hi[8], l2[8], h2[8];
            if (a.interleaved) {
                float v[16];
                load_n<DT, 8>(m.x.p, x + 2 * p, 2 * valid, v);
                load_n<DT, 8>(m.x.p, x + 2 * p + 8, 2 * valid - 8, v + 8);
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    lo[j] = v[2 * j];
                    hi[j] = v[2 * j + 1];
                }
            } else {
                load_n<DT, 8>(m.x.p, x + p, valid, lo);
                load_n<DT, 8>(m.x.p, x + P + p, valid, hi);
            }
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const f32x2 q = j < valid ? cs[j] : f32x2{1.0f, 0.0f};
                l2[j] = __builtin_fmaf(lo[j], q[0], -(hi[j] * q[1]));
                h2[j] = __builtin_fmaf(lo[j], q[1], hi[j] * q[0]);
            }
            if (a.interleaved) {
                float v[16];
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    v[2 * j] = l2[j];
                    v[2 * j + 1] = h2[j];
                }
                store_n<DT, 8>(m.y.p, y + 2 * p, 2 * valid, v);
                store_n<DT, 8>(m.y.p, y + 2 * p + 8, 2 * valid - 8, v + 8);
            } else {
                store_n<DT, 8>(m.y.p, y + p, valid, l2);
                store_n<DT, 8>(m.y.p, y + P + p, valid, h2);
            }
        }
    }
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
    if (dt == DP_F32) hipLaunchKernelGGL(k_rotary<DP_F32>, grid, dim3(kThreads), lds, stream, a, n);
    else if (dt == DP_F16) hipLaunchKernelGGL(k_rotary<DP_F16>, grid, dim3(kThreads), lds, stream, a, n);
    else hipLaunchKernelGGL(k_rotary<DP_BF16>, grid, dim3(kThreads), lds, stream, a, n);
    return hipGetLastError();
}

}  // namespace dpk

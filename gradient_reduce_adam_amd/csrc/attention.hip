// gfx950 kernel of the attention's forward pass: out = softmax(scale q k^T) v and
// the logarithm of each row's sum, in one pass over the keys.
//
// A workgroup takes 128 kB queries of one head and goes over the keys that they
// see in tiles of 64 rows of k and v.  Each of its four waves has 32 kB queries:
//   S^T = k q^T       rows are keys, columns queries: a lane holds its query's scores
//   p = exp2(c S - c m), c = scale log2(e), m a running maximum of the query
//   out^T += v^T p     p goes into the product from the registers it is in
// with v^T read by the transposing LDS load, and sums and maxima kept by each lane.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "attention.h"

namespace dpk {
namespace {

using namespace attn;

constexpr int kKeys = 64;  // of a tile

template <dp_dtype DT, int kD, int kB>
__global__ void __launch_bounds__(kThreads, kB == 1 ? 2 : 1) k_attention(AttentionArgs a) {
    using T = Tile<kD>;
    constexpr int kTileBytes = kKeys * T::kRowBytes, kRows = 128 * kB, kBlocks = kD / 32;
    __shared__ __align__(1024) unsigned char lds[4 * kTileBytes];  // two turns of a k and a v tile
    const Sequences& sq = a.s;
    Place at;
    if (!find<kRows>(sq, 0, sq.heads, sq.causal, at)) return;
    const int h = at.head, hk = h / (sq.heads / sq.kv_heads), tile = at.tile;
    const int L = at.length[0], M = at.length[1], shift = M - L;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), half = threadIdx.x >> 5 & 1;
    const int first = tile * kRows, mine = first + wave * 32 * kB;  // queries of the workgroup, of the wave

    // The keys that a query sees: [lo, hi].
    const auto lowest = [&](int i) { return sq.window > 0 && i + shift >= sq.window ? i + shift - sq.window + 1 : 0; };
    const auto highest = [&](int i) { return sq.causal && i + shift < M ? i + shift : M - 1; };
    const int behind = first + kRows < L ? first + kRows : L;  // the workgroup's queries end
    const int from = lowest(first) / kKeys * kKeys, to = highest(behind - 1) + 1;

    const Head q = head_of(a.q, at.begin[0], h), k = head_of(a.k, at.begin[1], hk), v = head_of(a.v, at.begin[1], hk);
    u32x4 qf[kB][kD / 16];
    f32x16 o[kB][kBlocks];
    float m[kB], sum[kB];
    int lo[kB], hi[kB];
#pragma unroll
    for (int b = 0; b < kB; ++b) {
        const int i = mine + 32 * b + (threadIdx.x & 31);
        load_right<kD>(q, i, i < L, sq.dim, qf[b]);
        m[b] = -kInf;
        sum[b] = 0.0f;
        lo[b] = lowest(i);
        hi[b] = highest(i);
#pragma unroll
        for (int n = 0; n < kBlocks; ++n) o[b][n] = zeros();
    }
    // Tiles that some query of this wave sees, and those that all of them see whole.
    const int last = mine + 32 * kB - 1;
    const int some_lo = lowest(mine), some_hi = highest(last), all_lo = lowest(last), all_hi = highest(mine);

    const float c = sq.scale * kLog2e;
    lds_u8* const base = (lds_u8*)lds;
    const int along = T::along(), across = T::across();
    if (from < to) {
        Stage<kD, kKeys> ks, vs;
        const auto load = [&](int t) {
            ks.load(k, t, M, sq.dim);
            vs.load(v, t, M, sq.dim);
        };
        const auto store = [&](int turn) {
            ks.store(base + turn, sq.dim);
            vs.store(base + turn + kTileBytes, sq.dim);
        };
#pragma unroll
        for (int i = 0; i < 4; ++i) ks.clear(base + i * kTileBytes, sq.dim);
        load(from);
        store(0);
        load(from + kKeys < to ? from + kKeys : from);
        __syncthreads();
        const auto step = [&](const lds_u8* kt, int t) {
            const lds_u8* vt = kt + kTileBytes;
            f32x16 s[kB][2];
#pragma unroll
            for (int b = 0; b < kB; ++b) s[b][0] = s[b][1] = zeros();
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int j = 0; j < 2; ++j)
#pragma unroll
                for (int n = 0; n < kD / 16; ++n) {
                    const u32x4 kf = T::read_along(kt, along, j, n);
#pragma unroll
                    for (int b = 0; b < kB; ++b) s[b][j] = mma<DT>(kf, qf[b][n], s[b][j]);
                }
            ahead<2 * (kD / 16), kB, 1, 6>();
            u32x4 p[kB][2][2];
#pragma unroll
            for (int b = 0; b < kB; ++b) {
                if (t < all_lo || t + kKeys - 1 > all_hi) {  // scores that do not count
                    const int up = hi[b] - t - 4 * half, down = lo[b] - t - 4 * half;
#pragma unroll
                    for (int j = 0; j < 2; ++j)
#pragma unroll
                        for (int e = 0; e < 16; ++e) {
                            const int key = 32 * j + 8 * (e >> 2) + (e & 3);
                            s[b][j][e] = key > up || key < down ? -kInf : s[b][j][e];
                        }
                }
                float top = s[b][0][0];
#pragma unroll
                for (int j = 0; j < 2; ++j)
#pragma unroll
                    for (int e = 0; e < 16; ++e) top = fmaxf(top, s[b][j][e]);
                const f32x2 both = halves(top);
                top = fmaxf(fmaxf(both[0], both[1]), m[b]);
                // The sums follow the maximum only where it has risen by more than 8
                // powers of two: below that, p stays within 2^8 and keeps all its bits.
                if (__ballot(c * (top - m[b]) > 8.0f || m[b] == -kInf)) {
                    const float alpha = m[b] == -kInf ? 0.0f : __builtin_amdgcn_exp2f(c * (m[b] - top));
                    sum[b] *= alpha;
#pragma unroll
                    for (int n = 0; n < kBlocks; ++n)
#pragma unroll
                        for (int e = 0; e < 16; ++e) o[b][n][e] *= alpha;
                    m[b] = top;
                }
            }
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int b = 0; b < kB; ++b) {
                const float less = m[b] == -kInf ? 0.0f : c * m[b];
                float part[2] = {0.0f, 0.0f};
#pragma unroll
                for (int j = 0; j < 2; ++j)
#pragma unroll
                    for (int n = 0; n < 2; ++n) {
#pragma unroll
                        for (int e = 8 * n; e < 8 * n + 8; ++e) {
                            s[b][j][e] = __builtin_amdgcn_exp2f(__builtin_fmaf(c, s[b][j][e], -less));
                            part[e & 1] += s[b][j][e];
                        }
                        p[b][j][n] = pack8<DT>(s[b][j], n);
                    }
                sum[b] += part[0] + part[1];
            }
#pragma unroll
            for (int j = 0; j < 2; ++j)
#pragma unroll
                for (int n = 0; n < 2; ++n)
#pragma unroll
                    for (int x = 0; x < kBlocks; ++x) {
                        const u32x4 vf = T::read_across(vt, across, 2 * j + n, x);
#pragma unroll
                        for (int b = 0; b < kB; ++b) o[b][x] = mma<DT>(vf, p[b][j][n], o[b][x]);
                    }
            ahead<4 * kBlocks, kB, 2, 4>();
            __builtin_amdgcn_sched_barrier(0);
        };
        int turn = 0;
        for (int t = from; t < to; t += kKeys) {
            if (mine < L && t <= some_hi && t + kKeys > some_lo) step(base + turn, t);
            if (t + kKeys < to) {
                turn ^= 2 * kTileBytes;
                store(turn);
                // past the last tile this one is loaded again, and not used
                load(t + 2 * kKeys < to ? t + 2 * kKeys : t + kKeys);
                __syncthreads();
            }
        }
    }
#pragma unroll
    for (int b = 0; b < kB; ++b) {
        const int i = mine + 32 * b + (threadIdx.x & 31);
        const f32x2 both = halves(sum[b]);
        const float total = both[0] + both[1];
        // a query that sees no key: total 0, m -infinity
        store_columns<DT, kD>(a.out, at.begin[0] + i, h, i < L, sq.dim, o[b], total == 0.0f ? 0.0f : 1.0f / total);
        if (i < L && half == 0)
            a.lse[h * sq.rows[0] + at.begin[0] + i] = total == 0.0f ? -kInf : sq.scale * m[b] + kLn2 * __builtin_amdgcn_logf(total);
    }
}

template <dp_dtype DT, int kB>
void launch_dim(const AttentionArgs& a, hipStream_t stream) {
    const dim3 grid(static_cast<unsigned>(attention_slots(a.s, 0, 128 * kB) * a.s.heads)), block(kThreads);
    if (grid.x == 0) return;
    if (a.s.dim <= 32) hipLaunchKernelGGL((k_attention<DT, 32, kB>), grid, block, 0, stream, a);
    else if (a.s.dim <= 64) hipLaunchKernelGGL((k_attention<DT, 64, kB>), grid, block, 0, stream, a);
    else if (a.s.dim <= 96) hipLaunchKernelGGL((k_attention<DT, 96, kB>), grid, block, 0, stream, a);
    else hipLaunchKernelGGL((k_attention<DT, 128, kB>), grid, block, 0, stream, a);
}

}  // namespace

int64_t attention_slots(const Sequences& s, int side, int64_t tile) {
    if (s.count == 0) return 0;
    return s.offsets[side] ? s.rows[side] / tile + s.count : s.count * ((s.length[side] + tile - 1) / tile);
}

int64_t attention_groups(const Sequences& s) {
    const int64_t q = attention_slots(s, 0, 128) * s.heads, k = attention_slots(s, 1, 128) * s.heads;
    return q > k ? q : k;
}

hipError_t launch_attention(dp_dtype dt, const AttentionArgs& a, hipStream_t stream) {
    if (dt == DP_BF16) launch_dim<DP_BF16, 1>(a, stream);
    else launch_dim<DP_F16, 1>(a, stream);
    return hipGetLastError();
}

}  // namespace dpk

// gfx950 kernel of the attention's forward pass: out = softmax(scale q k^T) v and
// the logarithm of each row's sum, in one pass over the keys.
//
// A workgroup takes 128 queries of one head and goes over the keys that they see in
// tiles of 64 rows of k and v.  Each of its four waves has 32 queries:
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

template <dp_dtype DT, int kD, int kWaves>
__global__ void __launch_bounds__(64 * kWaves, kWaves == 4 ? 2 : 1) k_attention(AttentionArgs a) {
    using T = Tile<kD>;
    constexpr int kTileBytes = kKeys * T::kRowBytes, kRows = 32 * kWaves, kBlocks = kD / 32;
    __shared__ __align__(1024) unsigned char lds[4 * kTileBytes];  // two turns of a k and a v tile
    const Sequences& sq = a.s;
    Place at;
    if (!find<kRows>(sq, 0, sq.heads, sq.causal, at)) return;
    const int h = at.head, hk = h / (sq.heads / sq.kv_heads);
    const int L = at.length[0], M = at.length[1], shift = M - L;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), half = threadIdx.x >> 5 & 1;
    const int first = at.tile * kRows, mine = first + wave * 32;  // queries of the workgroup, of the wave

    // The keys that a query sees: [lo, hi].
    const auto lowest = [&](int i) { return sq.window > 0 && i + shift >= sq.window ? i + shift - sq.window + 1 : 0; };
    const auto highest = [&](int i) { return sq.causal && i + shift < M ? i + shift : M - 1; };
    const int behind = first + kRows < L ? first + kRows : L;  // the workgroup's queries end
    const int from = lowest(first) / kKeys * kKeys, to = highest(behind - 1) + 1;
    const int i = mine + (threadIdx.x & 31);
    const int lo = lowest(i), hi = highest(i);
    // Tiles that some query of this wave sees, and those that all of them see whole.
    const int some_lo = lowest(mine), some_hi = highest(mine + 31), all_lo = lowest(mine + 31), all_hi = highest(mine);

    const Head q = head_of(a.q, at.begin[0], h), k = head_of(a.k, at.begin[1], hk), v = head_of(a.v, at.begin[1], hk);
    u32x4 qf[kD / 16];
    load_right<kD>(q, i, i < L, sq.dim, qf);
    f32x16 o[kBlocks];
#pragma unroll
    for (int n = 0; n < kBlocks; ++n) o[n] = zeros();
    float m = -kInf, sum = 0.0f;

    const float c = sq.scale * kLog2e;
    lds_u8* const base = (lds_u8*)lds;
    const int along = T::along(), across = T::across();
    if (from < to) {
        Stage<kD, kKeys, 64 * kWaves> ks, vs;
        const auto load = [&](int t) {
            ks.load(k, t, M, sq.dim);
            vs.load(v, t, M, sq.dim);
        };
        const auto store = [&](int turn) {
            ks.store(base + turn, sq.dim);
            vs.store(base + turn + kTileBytes, sq.dim);
        };
        const auto step = [&](const lds_u8* kt, int t) {
            const lds_u8* vt = kt + kTileBytes;
            f32x16 s[2] = {zeros(), zeros()};
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int j = 0; j < 2; ++j)
#pragma unroll
                for (int n = 0; n < kD / 16; ++n) s[j] = mma<DT>(T::read_along(kt, along, j, n), qf[n], s[j]);
            ahead<2 * (kD / 16), 1, 1, 6>();
            if (t < all_lo || t + kKeys - 1 > all_hi) {  // scores that do not count
                const int up = hi - t - 4 * half, down = lo - t - 4 * half;
#pragma unroll
                for (int j = 0; j < 2; ++j)
#pragma unroll
                    for (int e = 0; e < 16; ++e) {
                        const int key = 32 * j + 8 * (e >> 2) + (e & 3);
                        s[j][e] = key > up || key < down ? -kInf : s[j][e];
                    }
            }
            float top = s[0][0];
#pragma unroll
            for (int j = 0; j < 2; ++j)
#pragma unroll
                for (int e = 0; e < 16; ++e) top = fmaxf(top, s[j][e]);
            const f32x2 both = halves(top);
            top = fmaxf(fmaxf(both[0], both[1]), m);
            // The sums follow the maximum only where it has risen by more than 8
            // powers of two: below that, p stays within 2^8 and keeps all its bits.
            if (__ballot(c * (top - m) > 8.0f || m == -kInf)) {
                const float alpha = m == -kInf ? 0.0f : __builtin_amdgcn_exp2f(c * (m - top));
                sum *= alpha;
#pragma unroll
                for (int n = 0; n < kBlocks; ++n)
#pragma unroll
                    for (int e = 0; e < 16; ++e) o[n][e] *= alpha;
                m = top;
            }
            __builtin_amdgcn_sched_barrier(0);
            const float less = m == -kInf ? 0.0f : c * m;
            float part[2] = {0.0f, 0.0f};
            u32x4 p[2][2];
#pragma unroll
            for (int j = 0; j < 2; ++j)
#pragma unroll
                for (int n = 0; n < 2; ++n) {
#pragma unroll
                    for (int e = 8 * n; e < 8 * n + 8; ++e) {
                        s[j][e] = __builtin_amdgcn_exp2f(__builtin_fmaf(c, s[j][e], -less));
                        part[e & 1] += s[j][e];
                    }
                    p[j][n] = pack8<DT>(s[j], n);
                }
            sum += part[0] + part[1];
#pragma unroll
            for (int j = 0; j < 2; ++j)
#pragma unroll
                for (int n = 0; n < 2; ++n)
#pragma unroll
                    for (int x = 0; x < kBlocks; ++x) o[x] = mma<DT>(T::read_across(vt, across, 2 * j + n, x), p[j][n], o[x]);
            ahead<4 * kBlocks, 1, 2, 4>();
            __builtin_amdgcn_sched_barrier(0);
        };
#pragma unroll
        for (int n = 0; n < 4; ++n) ks.clear(base + n * kTileBytes, sq.dim);
        load(from);
        store(0);
        load(from + kKeys < to ? from + kKeys : from);
        __syncthreads();
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
    const f32x2 both = halves(sum);
    const float total = both[0] + both[1];
    // a query that sees no key: total 0, m -infinity
    store_columns<DT, kD>(a.out, at.begin[0] + i, h, i < L, sq.dim, o, total == 0.0f ? 0.0f : 1.0f / total);
    if (i < L && half == 0)
        a.lse[h * sq.rows[0] + at.begin[0] + i] = total == 0.0f ? -kInf : sq.scale * m + kLn2 * __builtin_amdgcn_logf(total);
}

template <dp_dtype DT, int kD, int kWaves>
void launch_one(const AttentionArgs& a, hipStream_t stream) {
    const dim3 grid(static_cast<unsigned>(attention_slots(a.s, 0, 32 * kWaves) * a.s.heads));
    if (grid.x > 0) hipLaunchKernelGGL((k_attention<DT, kD, kWaves>), grid, dim3(64 * kWaves), 0, stream, a);
}

template <dp_dtype DT>
void launch_dim(const AttentionArgs& a, hipStream_t stream) {
    if (a.s.dim <= 32) launch_one<DT, 32, 4>(a, stream);
    else if (a.s.dim <= 64) launch_one<DT, 64, 4>(a, stream);
    else if (a.s.dim <= 96) launch_one<DT, 96, 4>(a, stream);
    else if (attention_wide(a.s)) launch_one<DT, 128, 8>(a, stream);
    else launch_one<DT, 128, 4>(a, stream);
}

}  // namespace

int64_t attention_slots(const Sequences& s, int side, int64_t tile) {
    if (s.count == 0) return 0;
    return s.offsets[side] ? s.rows[side] / tile + s.count : s.count * ((s.length[side] + tile - 1) / tile);
}

// Eight waves in a workgroup load each tile of keys half as often and leave more
// registers to fragments that are read ahead, but wait for each other twice as
// many, and their 256 queries cross the mask's edge further.  Heads of 128, four
// against eight waves, forward and dq, TFLOP/s of their products: sequences of 8192
// 980 and 1055 against 1038 and 1122, of 4096 874 and 967 against 894 and 1020, of
// 2048 859 and 849 against 856 and 836.  They have to be enough to fill the CUs.
bool attention_wide(const Sequences& s) {
    return s.count > 0 && s.rows[1] / s.count >= 3500 && attention_slots(s, 0, 256) * s.heads >= 512;
}

int64_t attention_groups(const Sequences& s) {
    const int64_t q = attention_slots(s, 0, 128) * s.heads, k = attention_slots(s, 1, 128) * s.heads;
    return q > k ? q : k;
}

hipError_t launch_attention(dp_dtype dt, const AttentionArgs& a, hipStream_t stream) {
    if (dt == DP_BF16) launch_dim<DP_BF16>(a, stream);
    else launch_dim<DP_F16>(a, stream);
    return hipGetLastError();
}

}  // namespace dpk

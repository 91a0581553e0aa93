// gfx950 kernels of the attention's backward pass.  Probabilities are computed
// again from q, k and the rows' lse, p = exp2(c S - log2(e) lse), c = scale log2(e):
//   dq = scale ds k,  dk = scale ds^T q,  dv = p^T dout,  ds = p (dout v^T - delta),
// delta_i = dout_i out_i.  dq is a sum over keys, dk and dv over queries.  Two
// launches, one for each direction, give each sum to one wave, in a fixed order
// and in registers; the price is computing the scores and dout v^T in both, seven
// products instead of five.  (One launch would need sums in memory that many
// workgroups add to, in an order that changes.)
//
// k_attention_dq   32 kB queries a wave, over tiles of keys, as the forward pass:
//   S^T = k q^T, dP^T = v dout^T, dq^T += k^T ds^T.  It leaves delta for the other.
// k_attention_dkv  32 kB keys a wave, over tiles of queries of every head that
//   shares the keys: S = q k^T, dP = dout v^T, dv^T += dout^T p, dk^T += q^T ds.  The
//   scores' accumulators start at -lse / scale and dP's at -delta, so p = exp2(c S)
//   and ds = p dP.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "attention.h"

namespace dpk {
namespace {

using namespace attn;

constexpr int kKeys = 64;     // of a tile in k_attention_dq
constexpr int kQueries = 32;  // of a tile in k_attention_dkv

template <dp_dtype DT, int kD, int kB>
__global__ void __launch_bounds__(kThreads, kB == 1 ? 2 : 1) k_attention_dq(AttentionArgs a) {
    using T = Tile<kD>;
    constexpr int kTileBytes = kKeys * T::kRowBytes, kRows = 128 * kB, kBlocks = kD / 32;
    __shared__ __align__(1024) unsigned char lds[4 * kTileBytes];  // two turns of a k and a v tile
    const Sequences& sq = a.s;
    const int slots = gridDim.x / sq.heads, job = job_of(blockIdx.x, gridDim.x);
    const int h = job / slots, hk = h / (sq.heads / sq.kv_heads);
    Place at;
    if (!find<kRows>(sq, 0, job % slots, at)) return;
    const int L = at.length[0], M = at.length[1], shift = M - L;
    const int tile = sq.causal ? at.tiles - 1 - at.tile : at.tile;  // those with the most keys first
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), half = threadIdx.x >> 5 & 1;
    const int first = tile * kRows, mine = first + wave * 32 * kB;

    const auto lowest = [&](int i) { return sq.window > 0 && i + shift >= sq.window ? i + shift - sq.window + 1 : 0; };
    const auto highest = [&](int i) { return sq.causal && i + shift < M ? i + shift : M - 1; };
    const int behind = first + kRows < L ? first + kRows : L;
    const int from = lowest(first) / kKeys * kKeys, to = highest(behind - 1) + 1;

    const Head q = head_of(a.q, at.begin[0], h), k = head_of(a.k, at.begin[1], hk), v = head_of(a.v, at.begin[1], hk);
    const Head out = head_of(a.out, at.begin[0], h), dout = head_of(a.dout, at.begin[0], h);
    u32x4 qf[kB][kD / 16], df[kB][kD / 16];
    f32x16 o[kB][kBlocks];
    float less[kB], delta[kB];
    int lo[kB], hi[kB];
#pragma unroll
    for (int b = 0; b < kB; ++b) {
        const int i = mine + 32 * b + (threadIdx.x & 31);
        load_right<kD>(q, i, i < L, sq.dim, qf[b]);
        load_right<kD>(dout, i, i < L, sq.dim, df[b]);
        u32x4 of[kD / 16];
        load_right<kD>(out, i, i < L, sq.dim, of);
        float d = 0.0f;
#pragma unroll
        for (int s = 0; s < kD / 16; ++s)
#pragma unroll
            for (int w = 0; w < 4; ++w) {
                float x[2], y[2];
                unpack2<DT>(of[s][w], x);
                unpack2<DT>(df[b][s][w], y);
                d = __builtin_fmaf(x[0], y[0], d);
                d = __builtin_fmaf(x[1], y[1], d);
            }
        const f32x2 both = halves(d);
        delta[b] = both[0] + both[1];
        const int64_t row = h * sq.rows[0] + at.begin[0] + i;
        // p = 0 throughout for a query that sees no key, and for one that is not there
        less[b] = kInf;
        if (i < L) {
            const float lse = a.lse[row];
            less[b] = lse == -kInf ? kInf : kLog2e * lse;
            if (half == 0) a.delta[row] = delta[b];
        }
        lo[b] = lowest(i);
        hi[b] = highest(i);
#pragma unroll
        for (int n = 0; n < kBlocks; ++n) o[b][n] = zeros();
    }
    const int last = mine + 32 * kB - 1;
    const int some_lo = lowest(mine), some_hi = highest(last), all_lo = lowest(last), all_hi = highest(mine);

    const float c = sq.scale * kLog2e;
    lds_u8* const base = (lds_u8*)lds;
    const int along = T::along(), across = T::across();
    if (from < to) {
        Stage<kD, kKeys> ks, vs;
        ks.load(k, from, M, sq.dim);
        vs.load(v, from, M, sq.dim);
        ks.store(base);
        vs.store(base + kTileBytes);
        if (from + kKeys < to) {
            ks.load(k, from + kKeys, M, sq.dim);
            vs.load(v, from + kKeys, M, sq.dim);
        }
        __syncthreads();
        int turn = 0;
        for (int t = from; t < to; t += kKeys) {
            if (mine < L && t <= some_hi && t + kKeys > some_lo) {
                const lds_u8* kt = base + turn;
                const lds_u8* vt = kt + kTileBytes;
                const bool masked = t < all_lo || t + kKeys - 1 > all_hi;
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    f32x16 s[kB], dp[kB];
#pragma unroll
                    for (int b = 0; b < kB; ++b) s[b] = dp[b] = zeros();
#pragma unroll
                    for (int n = 0; n < kD / 16; ++n) {
                        const u32x4 kf = T::read_along(kt, along, j, n), vf = T::read_along(vt, along, j, n);
#pragma unroll
                        for (int b = 0; b < kB; ++b) {
                            s[b] = mma<DT>(kf, qf[b][n], s[b]);
                            dp[b] = mma<DT>(vf, df[b][n], dp[b]);
                        }
                    }
                    u32x4 ds[kB][2];
#pragma unroll
                    for (int b = 0; b < kB; ++b) {
                        if (masked) {
                            const int up = hi[b] - t - 4 * half, down = lo[b] - t - 4 * half;
#pragma unroll
                            for (int e = 0; e < 16; ++e) {
                                const int key = 32 * j + 8 * (e >> 2) + (e & 3);
                                s[b][e] = key > up || key < down ? -kInf : s[b][e];
                            }
                        }
#pragma unroll
                        for (int e = 0; e < 16; ++e)
                            s[b][e] = __builtin_amdgcn_exp2f(__builtin_fmaf(c, s[b][e], -less[b])) * (dp[b][e] - delta[b]);
#pragma unroll
                        for (int n = 0; n < 2; ++n) ds[b][n] = pack8<DT>(s[b], n);
                    }
#pragma unroll
                    for (int n = 0; n < 2; ++n)
#pragma unroll
                        for (int x = 0; x < kBlocks; ++x) {
                            const u32x4 kf = T::read_across(kt, across, 2 * j + n, x);
#pragma unroll
                            for (int b = 0; b < kB; ++b) o[b][x] = mma<DT>(kf, ds[b][n], o[b][x]);
                        }
                }
            }
            if (t + kKeys < to) {
                const int other = turn ^ (2 * kTileBytes);
                ks.store(base + other);
                vs.store(base + other + kTileBytes);
                if (t + 2 * kKeys < to) {
                    ks.load(k, t + 2 * kKeys, M, sq.dim);
                    vs.load(v, t + 2 * kKeys, M, sq.dim);
                }
                __syncthreads();
                turn = other;
            }
        }
    }
#pragma unroll
    for (int b = 0; b < kB; ++b) {
        const int i = mine + 32 * b + (threadIdx.x & 31);
        store_columns<DT, kD>(a.dq, at.begin[0] + i, h, i < L, sq.dim, o[b], sq.scale);
    }
}

template <dp_dtype DT, int kD, int kB>
__global__ void __launch_bounds__(kThreads, kB == 1 && kD <= 96 ? 2 : 1) k_attention_dkv(AttentionArgs a) {
    using T = Tile<kD>;
    constexpr int kTileBytes = kQueries * T::kRowBytes, kRows = 128 * kB, kBlocks = kD / 32;
    constexpr int kTurn = 2 * kTileBytes + 2 * kQueries * 4;  // a q and a dout tile, -lse / scale and -delta of their rows
    __shared__ __align__(1024) unsigned char lds[2 * kTurn];
    const Sequences& sq = a.s;
    const int slots = gridDim.x / sq.kv_heads, job = job_of(blockIdx.x, gridDim.x);
    const int hk = job / slots, group = sq.heads / sq.kv_heads;
    Place at;
    if (!find<kRows>(sq, 1, job % slots, at)) return;
    const int L = at.length[0], M = at.length[1], shift = M - L;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), half = threadIdx.x >> 5 & 1;
    const int first = at.tile * kRows, mine = first + wave * 32 * kB;  // keys of the workgroup, of the wave

    // The queries that see a key: [lo, hi].
    const auto lowest = [&](int j) { return sq.causal && j - shift > 0 ? j - shift : 0; };
    const auto highest = [&](int j) { return sq.window > 0 && j - shift + sq.window - 1 < L ? j - shift + sq.window - 1 : L - 1; };
    const int behind = first + kRows < M ? first + kRows : M;
    const int from = lowest(first) / kQueries * kQueries, to = highest(behind - 1) + 1;
    const int each = to > from ? (to - from + kQueries - 1) / kQueries : 0;  // tiles of a head

    const Head k = head_of(a.k, at.begin[1], hk), v = head_of(a.v, at.begin[1], hk);
    u32x4 kf[kB][kD / 16], vf[kB][kD / 16];
    f32x16 dk[kB][kBlocks], dv[kB][kBlocks];
    int lo[kB], hi[kB];
#pragma unroll
    for (int b = 0; b < kB; ++b) {
        const int j = mine + 32 * b + (threadIdx.x & 31);
        load_right<kD>(k, j, j < M, sq.dim, kf[b]);
        load_right<kD>(v, j, j < M, sq.dim, vf[b]);
        lo[b] = lowest(j);
        hi[b] = highest(j);
#pragma unroll
        for (int n = 0; n < kBlocks; ++n) dk[b][n] = dv[b][n] = zeros();
    }
    const int last = mine + 32 * kB - 1;
    const int some_lo = lowest(mine), some_hi = highest(last), all_lo = lowest(last), all_hi = highest(mine);

    const float c = sq.scale * kLog2e, unit = 1.0f / sq.scale;
    lds_u8* const base = (lds_u8*)lds;
    const int along = T::along(), across = T::across();
    const int tiles = each * group;
    if (tiles > 0) {
        Stage<kD, kQueries> qs, ds;
        float row = 0.0f;  // of threads 0 .. 31: -lse / scale of a query, of 32 .. 63: -delta
        int g = 0, next = from;  // the next tile to load
        const auto load = [&]() {
            const int h = hk * group + g;
            qs.load(head_of(a.q, at.begin[0], h), next, L, sq.dim);
            ds.load(head_of(a.dout, at.begin[0], h), next, L, sq.dim);
            if (threadIdx.x < 2 * kQueries) {
                const int i = next + (threadIdx.x & 31);
                const int64_t place = h * sq.rows[0] + at.begin[0] + i;
                row = threadIdx.x < kQueries ? -kInf : 0.0f;
                if (i < L) {
                    if (threadIdx.x < kQueries) {
                        const float lse = a.lse[place];
                        row = lse == -kInf ? -kInf : -lse * unit;  // p = 0 for a query that sees no key
                    } else {
                        row = -a.delta[place];
                    }
                }
            }
            next += kQueries;
            if (next >= to) {
                next = from;
                ++g;
            }
        };
        const auto store = [&](int turn) {
            qs.store(base + turn);
            ds.store(base + turn + kTileBytes);
            if (threadIdx.x < 2 * kQueries) *(lds_f32*)(base + turn + 2 * kTileBytes + 4 * threadIdx.x) = row;
        };
        load();
        store(0);
        if (tiles > 1) load();
        __syncthreads();
        int turn = 0, t = from;
        for (int i = 0; i < tiles; ++i) {
            if (mine < M && t <= some_hi && t + kQueries > some_lo) {
                const lds_u8* qt = base + turn;
                const lds_u8* dt = qt + kTileBytes;
                const lds_u8* rt = dt + kTileBytes + 16 * half;
                const bool masked = t < all_lo || t + kQueries - 1 > all_hi;
                u32x4 p[kB][2], w[kB][2];
#pragma unroll
                for (int b = 0; b < kB; ++b) {
                    f32x16 s, dp;
#pragma unroll
                    for (int n = 0; n < 4; ++n) {
                        const f32x4 x = *(const lds_f32x4*)(rt + 32 * n), y = *(const lds_f32x4*)(rt + 4 * kQueries + 32 * n);
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            s[4 * n + e] = x[e];
                            dp[4 * n + e] = y[e];
                        }
                    }
#pragma unroll
                    for (int n = 0; n < kD / 16; ++n) {
                        s = mma<DT>(T::read_along(qt, along, 0, n), kf[b][n], s);
                        dp = mma<DT>(T::read_along(dt, along, 0, n), vf[b][n], dp);
                    }
                    if (masked) {
                        const int up = hi[b] - t - 4 * half, down = lo[b] - t - 4 * half;
#pragma unroll
                        for (int e = 0; e < 16; ++e) {
                            const int query = 8 * (e >> 2) + (e & 3);
                            s[e] = query > up || query < down ? -kInf : s[e];
                        }
                    }
#pragma unroll
                    for (int e = 0; e < 16; ++e) {
                        s[e] = __builtin_amdgcn_exp2f(c * s[e]);
                        dp[e] *= s[e];
                    }
#pragma unroll
                    for (int n = 0; n < 2; ++n) {
                        p[b][n] = pack8<DT>(s, n);
                        w[b][n] = pack8<DT>(dp, n);
                    }
                }
#pragma unroll
                for (int n = 0; n < 2; ++n)
#pragma unroll
                    for (int x = 0; x < kBlocks; ++x) {
                        const u32x4 df = T::read_across(dt, across, n, x), qf = T::read_across(qt, across, n, x);
#pragma unroll
                        for (int b = 0; b < kB; ++b) {
                            dv[b][x] = mma<DT>(df, p[b][n], dv[b][x]);
                            dk[b][x] = mma<DT>(qf, w[b][n], dk[b][x]);
                        }
                    }
            }
            t = t + kQueries >= to ? from : t + kQueries;
            if (i + 1 < tiles) {
                const int other = turn ? 0 : kTurn;
                store(other);
                if (i + 2 < tiles) load();
                __syncthreads();
                turn = other;
            }
        }
    }
#pragma unroll
    for (int b = 0; b < kB; ++b) {
        const int j = mine + 32 * b + (threadIdx.x & 31);
        store_columns<DT, kD>(a.dk, at.begin[1] + j, hk, j < M, sq.dim, dk[b], sq.scale);
        store_columns<DT, kD>(a.dv, at.begin[1] + j, hk, j < M, sq.dim, dv[b], 1.0f);
    }
}

template <dp_dtype DT, int kD>
void launch_both(const AttentionArgs& a, hipStream_t stream) {
    const dim3 block(kThreads), gq(static_cast<unsigned>(attention_slots(a.s, 0, 128) * a.s.heads)),
        gk(static_cast<unsigned>(attention_slots(a.s, 1, 128) * a.s.kv_heads));
    if (gq.x > 0) hipLaunchKernelGGL((k_attention_dq<DT, kD, 1>), gq, block, 0, stream, a);
    if (gk.x > 0) hipLaunchKernelGGL((k_attention_dkv<DT, kD, 1>), gk, block, 0, stream, a);
}

template <dp_dtype DT>
void launch_dim(const AttentionArgs& a, hipStream_t stream) {
    if (a.s.dim <= 32) launch_both<DT, 32>(a, stream);
    else if (a.s.dim <= 64) launch_both<DT, 64>(a, stream);
    else if (a.s.dim <= 96) launch_both<DT, 96>(a, stream);
    else launch_both<DT, 128>(a, stream);
}

}  // namespace

hipError_t launch_attention_grad(dp_dtype dt, const AttentionArgs& a, hipStream_t stream) {
    if (dt == DP_BF16) launch_dim<DP_BF16>(a, stream);
    else launch_dim<DP_F16>(a, stream);
    return hipGetLastError();
}

}  // namespace dpk

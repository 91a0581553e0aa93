// gfx950 kernels of the attention's backward pass.  Probabilities are computed
// again from q, k and the rows' lse, p = exp2(c S - log2(e) lse), c = scale log2(e):
//   dq = scale ds k,  dk = scale ds^T q,  dv = p^T dout,  ds = p (dout v^T - delta),
// delta_i = dout_i out_i.  dq is a sum over keys, dk and dv over queries.  Two
// launches, one for each direction, give each sum to one wave, in a fixed order
// and in registers; the price is computing the scores and dout v^T in both, seven
// products instead of five.  (One launch would need sums in memory that many
// workgroups add to, in an order that changes.)
//
// k_attention_dq   32 queries a wave, over tiles of keys, as the forward pass:
//   S^T = k q^T, dP^T = v dout^T, dq^T += k^T ds^T.  It leaves delta for the other.
// k_attention_dkv  32 keys a wave, over tiles of queries of every head that
//   shares the keys: S = q k^T, dP = dout v^T, dv^T += dout^T p, dk^T += q^T ds.  The
//   scores' accumulators start at -lse / scale and dP's at -delta, so p = exp2(c S)
//   and ds = p dP.
//
// What bounds them: matrix pipes busy 52% (dq) and 47% (dk and dv) of the time that the
// CUs are, for heads of 128 with two waves a SIMD at 2.0 to 2.1 GHz.  2 x 4096 rows of 32
// heads of 128, causal, bf16: dq 395 to 420 us, 980 to 1040 TFLOP/s of its three products, dk
// and dv 548 to 575 us, 955 to 1000 of their four.  In dkv half of the products read both operands from LDS, which is
// busy 39%.  Heads of 64, 32 x 1024 rows of 12 heads, f16: 122 and 148 us, the vector
// units busy 51% and 48%, the matrix pipes 36 and 37%.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "attention.h"

namespace dpk {
namespace {

using namespace attn;

// kShare: so many neighbouring waves have the same 32 queries, and 32 keys each of
// every tile; with 1 a wave takes all 64 keys.
template <dp_dtype DT, int kD, int kWaves, int kShare>
__global__ void __launch_bounds__(64 * kWaves, kWaves == 4 && kShare == 1 ? 2 : 1) k_attention_dq(AttentionArgs a) {
    using T = Tile<kD>;
    constexpr int kRows = 32 * kWaves / kShare, kKeys = kShare == 1 ? 64 : 32 * kShare, kBlocks = (kD + 31) / 32;
    constexpr int kOwn = kShare == 1 ? 2 : 1;  // times 32 keys of a tile that a wave takes
    constexpr int kTileBytes = kKeys * T::kRowBytes;
    __shared__ __align__(1024) unsigned char lds[4 * kTileBytes];  // two turns of a k and a v tile
    const Sequences& sq = a.s;
    Place at;
    if (!find<kRows>(sq, 0, sq.heads, sq.causal, at)) return;
    const int h = at.head, hk = h / (sq.heads / sq.kv_heads);
    const int L = at.length[0], M = at.length[1], shift = M - L;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), half = threadIdx.x >> 5 & 1;
    const int first = at.tile * kRows, mine = first + wave / kShare * 32;  // queries of the workgroup, of the wave

    // The keys that a query sees: [lo, hi].
    const auto lowest = [&](int i) { return sq.window > 0 && i + shift >= sq.window ? i + shift - sq.window + 1 : 0; };
    const auto highest = [&](int i) { return sq.causal && i + shift < M ? i + shift : M - 1; };
    const int behind = first + kRows < L ? first + kRows : L;
    const int from = lowest(first) / kKeys * kKeys, to = highest(behind - 1) + 1;
    const int i = mine + (threadIdx.x & 31);
    const int lo = lowest(i), hi = highest(i);
    const int some_lo = lowest(mine), some_hi = highest(mine + 31), all_lo = lowest(mine + 31), all_hi = highest(mine);

    const Head q = head_of(a.q, at.begin[0], h), k = head_of(a.k, at.begin[1], hk), v = head_of(a.v, at.begin[1], hk);
    const Head out = head_of(a.out, at.begin[0], h), dout = head_of(a.dout, at.begin[0], h);
    // the first tile is on its way while delta is computed
    Stage<kD, kKeys, 64 * kWaves> ks, vs;
    const auto load = [&](int t) {
        ks.load(k, t, M, sq.dim);
        vs.load(v, t, M, sq.dim);
    };
    u32x4 qf[kD / 16], df[kD / 16], of[kD / 16];
    load_right<kD>(q, i, i < L, sq.dim, qf);
    load_right<kD>(dout, i, i < L, sq.dim, df);
    load_right<kD>(out, i, i < L, sq.dim, of);
    if (from < to) load(from);
    float delta = 0.0f;
#pragma unroll
    for (int n = 0; n < kD / 16; ++n)
#pragma unroll
        for (int w = 0; w < 4; ++w) {
            float x[2], y[2];
            unpack2<DT>(of[n][w], x);
            unpack2<DT>(df[n][w], y);
            delta = __builtin_fmaf(x[0], y[0], delta);
            delta = __builtin_fmaf(x[1], y[1], delta);
        }
    const f32x2 both = halves(delta);
    delta = both[0] + both[1];
    // p = 0 throughout for a query that sees no key, and for one that is not there
    float less = kInf;
    if (i < L) {
        const int64_t row = h * sq.rows[0] + at.begin[0] + i;
        const float lse = a.lse[row];
        less = lse == -kInf ? kInf : kLog2e * lse;
        if (half == 0 && wave % kShare == 0) a.delta[row] = delta;
    }
    f32x16 o[kBlocks];
#pragma unroll
    for (int n = 0; n < kBlocks; ++n) o[n] = zeros();

    const float c = sq.scale * kLog2e;
    lds_u8* const base = (lds_u8*)lds;
    const int along = T::along(), across = T::across();
    if (from < to) {
        const auto store = [&](int turn) {
            ks.store(base + turn, sq.dim);
            vs.store(base + turn + kTileBytes, sq.dim);
        };
        // The wave's keys of a tile, from t on.
        const auto step = [&](const lds_u8* kt, int t) {
            const lds_u8* vt = kt + kTileBytes;
#pragma unroll
            for (int j = 0; j < kOwn; ++j) {
                f32x16 s = zeros(), dp = zeros();
                __builtin_amdgcn_sched_barrier(0);
#pragma unroll
                for (int n = 0; n < kD / 16; ++n) {
                    s = mma<DT>(T::read_along(kt, along, j, n), qf[n], s);
                    dp = mma<DT>(T::read_along(vt, along, j, n), df[n], dp);
                }
                ahead<kD / 16, 2, 2, 3>();
                if (t + 32 * j + 31 > all_hi) hide_behind(s, hi - t - 32 * j - 4 * half);
                if (t + 32 * j < all_lo) hide_before(s, lo - t - 32 * j - 4 * half);
                __builtin_amdgcn_sched_barrier(0);
                u32x4 ds[2];
#pragma unroll
                for (int e = 0; e < 16; ++e) s[e] = __builtin_amdgcn_exp2f(__builtin_fmaf(c, s[e], -less)) * (dp[e] - delta);
#pragma unroll
                for (int n = 0; n < 2; ++n) ds[n] = pack8<DT>(s, n);
#pragma unroll
                for (int n = 0; n < 2; ++n)
#pragma unroll
                    for (int x = 0; x < kBlocks; ++x) o[x] = mma<DT>(T::read_across(kt, across, 2 * j + n, x), ds[n], o[x]);
                ahead<2 * kBlocks, 1, 2, 4>();
                __builtin_amdgcn_sched_barrier(0);
            }
        };
#pragma unroll
        for (int n = 0; n < 4; ++n) ks.clear(base + n * kTileBytes, sq.dim);
        store(0);
        load(from + kKeys < to ? from + kKeys : from);
        __syncthreads();
        int turn = 0;
        for (int t = from; t < to; t += kKeys) {
            const int skip = 32 * (wave % kShare);
            if (mine < L && t + skip <= some_hi && t + skip + 32 * kOwn > some_lo)
                step(base + turn + skip * T::kRowBytes, t + skip);
            if (t + kKeys < to) {
                turn ^= 2 * kTileBytes;
                store(turn);
                // past the last tile this one is loaded again, and not used
                load(t + 2 * kKeys < to ? t + 2 * kKeys : t + kKeys);
                __syncthreads();
            }
        }
    }
    unsigned short* const p = static_cast<unsigned short*>(a.dq.p) + (at.begin[0] + i) * a.dq.ld + h * a.dq.head;
    if constexpr (kShare == 4) {  // the waves' shares, added in their order
        static_assert(kBlocks <= kWaves && kWaves * kBlocks * 4096 <= 4 * kTileBytes, "the shares fit the tiles' memory");
        __syncthreads();
#pragma unroll
        for (int x = 0; x < kBlocks; ++x) share_block(base, kBlocks, wave, x, o[x]);
        __syncthreads();
        if (wave < kBlocks) {
            f32x16 sum = zeros();
#pragma unroll
            for (int w = 0; w < kWaves; ++w) add_block(base, kBlocks, w, wave, 1.0f, sum);
            store_block<DT>(p, 32 * wave, i < L, sq.dim, sum, sq.scale);
        }
    } else if constexpr (kShare == 2) {
        static_assert(kWaves * 4096 <= 4 * kTileBytes, "the shares fit the tiles' memory");
        join_pairs<kBlocks>(base, wave, 1.0f, 1.0f, o,
                            [&](int x, const f32x16& sum) { store_block<DT>(p, 32 * x, i < L, sq.dim, sum, sq.scale); });
    } else {
        store_columns<DT, kD>(a.dq, at.begin[0] + i, h, i < L, sq.dim, o, sq.scale);
    }
}

// p of a long row lies below f16's normal numbers, 2^-14, where a bit is lost with each
// power of two: in the product for dv it is taken 2^10 times, enough for the flat rows of 2^24
// keys.  Room is left for p > 1: scores of 2^24 and their lse are off by some powers of two.
// ds has no such bound, so it is rounded as it is.
template <dp_dtype DT>
constexpr float kLift = DT == DP_F16 ? 0x1p10f : 1.0f;

// v's fragments are read from LDS for each tile: in registers they would leave too few
// for two waves a SIMD (heads of 128: 925 us, from LDS 601) or three (of 64).
// kShare: so many neighbouring waves have the same 32 keys, and share the queries of
// every tile.
template <dp_dtype DT, int kD, int kWaves, int kQueries, int kShare>
__global__ void __launch_bounds__(64 * kWaves, kWaves == 8 || kShare == 4 ? 1 : kD <= 32 ? 4 : kD <= 64 ? 3 : 2) k_attention_dkv(AttentionArgs a) {
    using T = Tile<kD>;
    constexpr int kTileBytes = kQueries * T::kRowBytes, kRows = 32 * kWaves / kShare, kBlocks = (kD + 31) / 32;
    constexpr int kTurn = 2 * kTileBytes + 2 * kQueries * 4;  // a q and a dout tile, -lse / scale and -delta of their rows
    constexpr int kValues = kRows * T::kRowBytes;  // v
    __shared__ __align__(1024) unsigned char lds[kValues + 2 * kTurn];
    const Sequences& sq = a.s;
    Place at;
    if (!find<kRows>(sq, 1, sq.kv_heads, false, at)) return;
    const int hk = at.head, group = sq.heads / sq.kv_heads;
    const int L = at.length[0], M = at.length[1], shift = M - L;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), half = threadIdx.x >> 5 & 1;
    const int first = at.tile * kRows, run = wave / kShare, mine = first + 32 * run;  // keys of the workgroup, of the wave

    // The queries that see a key: [lo, hi].
    const auto lowest = [&](int j) { return sq.causal && j - shift > 0 ? j - shift : 0; };
    const auto highest = [&](int j) { return sq.window > 0 && j - shift + sq.window - 1 < L ? j - shift + sq.window - 1 : L - 1; };
    const int behind = first + kRows < M ? first + kRows : M;
    const int from = lowest(first) / kQueries * kQueries, to = highest(behind - 1) + 1;
    const int each = to > from ? (to - from + kQueries - 1) / kQueries : 0;  // tiles of a head

    const Head k = head_of(a.k, at.begin[1], hk), v = head_of(a.v, at.begin[1], hk);
    const int key = mine + (threadIdx.x & 31);
    const int lo = lowest(key), hi = highest(key);
    u32x4 kf[kD / 16];
    f32x16 dk[kBlocks], dv[kBlocks];
    load_right<kD>(k, key, key < M, sq.dim, kf);
#pragma unroll
    for (int n = 0; n < kBlocks; ++n) dk[n] = dv[n] = zeros();
    const int last = mine + 31;
    const int some_lo = lowest(mine), some_hi = highest(last), all_lo = lowest(last), all_hi = highest(mine);

    const float c = sq.scale * kLog2e, unit = 1.0f / sq.scale;
    lds_u8* const base = (lds_u8*)lds + kValues;
    const int along = T::along(), across = T::across();
    const int tiles = each * group;
    if (tiles > 0) {
        Stage<kD, kQueries, 64 * kWaves> qs, ds;
#pragma unroll
        for (int i = 0; i < 4; ++i) qs.clear(base + (i >> 1) * kTurn + (i & 1) * kTileBytes, sq.dim);
        // Of the first kQueries threads: -lse / scale of a query, of the next: -delta.  p = 0 for a
        // query that sees no key, and for one that is not there.
        float row = 0.0f;
        bool exists = false;
        int g = 0, next = from;  // the next tile to load
        const auto load = [&]() {
            const int h = hk * group + g;
            qs.load(head_of(a.q, at.begin[0], h), next, L, sq.dim);
            ds.load(head_of(a.dout, at.begin[0], h), next, L, sq.dim);
            const int i = next + (threadIdx.x & (kQueries - 1)), there = i < L ? i : L - 1;
            row = gload<float>(threadIdx.x & kQueries ? a.delta : a.lse, h * sq.rows[0] + at.begin[0] + there);
            exists = i < L;
            next += kQueries;
            if (next >= to) {
                next = from;
                g = g + 1 < group ? g + 1 : g;  // past the last tile: tiles that are not used
            }
        };
        const auto store = [&](int turn) {
            qs.store(base + turn, sq.dim);
            ds.store(base + turn + kTileBytes, sq.dim);
            const float start = threadIdx.x & kQueries ? -row : exists && row != -kInf ? -row * unit : -kInf;
            if (threadIdx.x < 2 * kQueries) *(lds_f32*)(base + turn + 2 * kTileBytes + 4 * threadIdx.x) = start;
        };
        // 32 queries from t on, row r of a tile.
        const auto step = [&](const lds_u8* tile, int r, int t) {
            const lds_u8* qt = tile + r * T::kRowBytes;
            const lds_u8* dt = qt + kTileBytes;
            const lds_u8* rt = tile + 2 * kTileBytes + 4 * r + 16 * half;
            f32x16 s, dp;
            __builtin_amdgcn_sched_barrier(0);
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
                s = mma<DT>(T::read_along(qt, along, 0, n), kf[n], s);
                dp = mma<DT>(T::read_along(dt, along, 0, n), T::read_along((lds_u8*)lds, along, run, n), dp);
            }
            reads<8>();
            ahead<kD / 16, 2, 3, 2>();
            if (t + 31 > all_hi) hide_behind(s, hi - t - 4 * half);
            if (t < all_lo) hide_before(s, lo - t - 4 * half);
            __builtin_amdgcn_sched_barrier(0);
            u32x4 p[2], w[2];
#pragma unroll
            for (int n = 0; n < 2; ++n) {
#pragma unroll
                for (int e = 8 * n; e < 8 * n + 8; ++e) {
                    s[e] = __builtin_amdgcn_exp2f(c * s[e]);
                    dp[e] *= s[e];
                    s[e] *= kLift<DT>;
                }
                p[n] = pack8<DT>(s, n);
                w[n] = pack8<DT>(dp, n);
            }
#pragma unroll
            for (int n = 0; n < 2; ++n)
#pragma unroll
                for (int x = 0; x < kBlocks; ++x) {
                    dv[x] = mma<DT>(T::read_across(dt, across, n, x), p[n], dv[x]);
                    dk[x] = mma<DT>(T::read_across(qt, across, n, x), w[n], dk[x]);
                }
            ahead<4 * kBlocks, 1, 2, 4>();
            __builtin_amdgcn_sched_barrier(0);
        };
        Stage<kD, kRows, 64 * kWaves> vs;
        vs.clear((lds_u8*)lds, sq.dim);
        vs.load(v, first, M, sq.dim);
        load();
        vs.store((lds_u8*)lds, sq.dim);
        store(0);
        load();
        __syncthreads();
        int turn = 0, t = from;
        for (int i = 0; i < tiles; ++i) {
#pragma unroll 1
            for (int r = 32 * (wave % kShare); r < kQueries; r += 32 * kShare)
                if (mine < M && t + r <= some_hi && t + r + 32 > some_lo) step(base + turn, r, t + r);
            t = t + kQueries >= to ? from : t + kQueries;
            if (i + 1 < tiles) {
                turn = kTurn - turn;
                store(turn);
                load();
                __syncthreads();
            }
        }
    }
    unsigned short* const pk = static_cast<unsigned short*>(a.dk.p) + (at.begin[1] + key) * a.dk.ld + hk * a.dk.head;
    unsigned short* const pv = static_cast<unsigned short*>(a.dv.p) + (at.begin[1] + key) * a.dv.ld + hk * a.dv.head;
    if constexpr (kShare == 4) {  // the waves' shares, added in their order
        static_assert(kBlocks <= kWaves && 2 * kWaves * kBlocks * 4096 <= kValues + 2 * kTurn, "the shares fit the tiles' memory");
        lds_u8* const at_dk = (lds_u8*)lds;
        lds_u8* const at_dv = at_dk + kWaves * kBlocks * 4096;
        __syncthreads();
#pragma unroll
        for (int x = 0; x < kBlocks; ++x) {
            share_block(at_dk, kBlocks, wave, x, dk[x]);
            share_block(at_dv, kBlocks, wave, x, dv[x]);
        }
        __syncthreads();
        if (wave < kBlocks) {
            f32x16 sum_k = zeros(), sum_v = zeros();
#pragma unroll
            for (int w = 0; w < kWaves; ++w) {
                add_block(at_dk, kBlocks, w, wave, 1.0f, sum_k);
                add_block(at_dv, kBlocks, w, wave, 1.0f, sum_v);
            }
            store_block<DT>(pk, 32 * wave, key < M, sq.dim, sum_k, sq.scale);
            store_block<DT>(pv, 32 * wave, key < M, sq.dim, sum_v, 1.0f / kLift<DT>);
        }
    } else if constexpr (kShare == 2) {  // the even wave of a pair sums dk, the odd one dv, a block at a time
        static_assert(kWaves * 4096 <= kValues + 2 * kTurn, "the shares fit the tiles' memory");
#pragma unroll
        for (int x = 0; x < kBlocks; ++x) {
            __syncthreads();
            share_block((lds_u8*)lds, 1, wave, 0, wave & 1 ? dk[x] : dv[x]);
            __syncthreads();
            f32x16 sum = wave & 1 ? dv[x] : dk[x];
            add_block((lds_u8*)lds, 1, wave ^ 1, 0, 1.0f, sum);
            store_block<DT>(wave & 1 ? pv : pk, 32 * x, key < M, sq.dim, sum, wave & 1 ? 1.0f / kLift<DT> : sq.scale);
        }
    } else {
        store_columns<DT, kD>(a.dk, at.begin[1] + key, hk, key < M, sq.dim, dk, sq.scale);
        store_columns<DT, kD>(a.dv, at.begin[1] + key, hk, key < M, sq.dim, dv, 1.0f / kLift<DT>);
    }
}

template <dp_dtype DT, int kD, int kWaves, int kShare>
void launch_dq(const AttentionArgs& a, hipStream_t stream) {
    const dim3 grid(static_cast<unsigned>(attention_slots(a.s, 0, 32 * kWaves / kShare) * a.s.heads));
    if (grid.x > 0) hipLaunchKernelGGL((k_attention_dq<DT, kD, kWaves, kShare>), grid, dim3(64 * kWaves), 0, stream, a);
}
template <dp_dtype DT, int kD, int kWaves, int kQueries, int kShare>
void launch_dkv(const AttentionArgs& a, hipStream_t stream) {
    const dim3 grid(static_cast<unsigned>(attention_slots(a.s, 1, 32 * kWaves / kShare) * a.s.kv_heads));
    if (grid.x > 0)
        hipLaunchKernelGGL((k_attention_dkv<DT, kD, kWaves, kQueries, kShare>), grid, dim3(64 * kWaves), 0, stream, a);
}

// In k_attention_dkv heads of more than 96 elements take eight waves and tiles of 64
// queries (2 x 4096 rows of 32 heads of 128: 546 us, four waves and 32 queries 573);
// those of up to 64 leave room for three waves a SIMD, which four waves fill better (heads of
// 64, 1024 rows: 143 us against 169), those of 72 to 96 for two.
template <dp_dtype DT, int kD>
void launch_both(const AttentionArgs& a, hipStream_t stream) {
    constexpr bool kLarge = kD > 96;
    const AttentionShape q = attention_shape(a.s, 0), k = attention_shape(a.s, 1);
    if (q == AttentionShape::kSplit) launch_dq<DT, kD, 4, 4>(a, stream);
    else if (q == AttentionShape::kPairs) launch_dq<DT, kD, 8, 2>(a, stream);
    else if (kLarge && q == AttentionShape::kWide) launch_dq<DT, kD, kLarge ? 8 : 4, 1>(a, stream);
    else launch_dq<DT, kD, 4, 1>(a, stream);
    if (k == AttentionShape::kSplit) launch_dkv<DT, kD, 4, 128, 4>(a, stream);
    else if (k == AttentionShape::kPairs) launch_dkv<DT, kD, 8, 64, 2>(a, stream);
    else launch_dkv<DT, kD, kLarge ? 8 : 4, kLarge ? 64 : 32, 1>(a, stream);
}

template <dp_dtype DT>
void launch_dim(const AttentionArgs& a, hipStream_t stream) {
    if (a.s.dim <= 32) launch_both<DT, 32>(a, stream);
    else if (a.s.dim <= 64) launch_both<DT, 64>(a, stream);
    else if (a.s.dim <= 80) launch_both<DT, 80>(a, stream);
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

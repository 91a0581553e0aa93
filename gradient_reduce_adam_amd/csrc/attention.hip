// gfx950 kernel of the attention's forward pass: out = softmax(scale q k^T) v and
// the logarithm of each row's sum, in one pass over the keys.
//
// A workgroup takes 128 queries of one head and goes over the keys that they see in
// tiles of 64 rows of k and v, or 32.  Each of its four waves has 32 queries:
//   S^T = k q^T       rows are keys, columns queries: a lane holds its query's scores
//   p = exp2(c S - c m), c = scale log2(e), m a running maximum of the query
//   out^T += v^T p     p goes into the product from the registers it is in
// with v^T read by the transposing LDS load, and sums and maxima kept by each lane.
// Queries that see many keys: eight waves, whose halves take turns at the matrix and
// the vector units.  Few queries: two or all four of the waves have the same 32, and
// share the keys of a tile.
//
// What bounds it.  Heads of 128: matrix pipes and vector units each 54% of the time that
// the CUs are busy (47% without turns), two waves a SIMD (o, the queries and two tiles on
// their way fill the registers), at the clock that power allows, 1.9 GHz: 4 x 4096 rows of
// 32 heads, causal, bf16 587 to 637 us on several machines, 863 to 937 TFLOP/s of the products
// that count, 1071 at 8192 rows; a large library product reaches 1420.  Heads of 64: the exponentials; 16 of
// a quarter of the rate, with their scaling, sum, maximum and rounding, take 450 cycles
// beside 256 of products, and the vector units are busy 70%: 32 x 1024 rows of 12 heads,
// f16 90 to 97 us.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "attention.h"

namespace dpk {
namespace {

using namespace attn;

// Tiles of 32 keys leave heads of 72 to 96 elements registers for a third wave a SIMD: 8 x
// 1024 rows of 32 heads of 96 76 us, with 64 keys 79.  (A fourth for heads of 64 gained
// nothing: 16384 rows of 12 heads 267 us with 64 keys, 280 with 32.)
template <int kD, int kWaves, int kShare>
constexpr int keys_of_tile() {
    return kShare > 1 ? 32 * kShare : kWaves == 4 && kD > 64 && kD <= 96 ? 32 : 64;
}

// Probabilities are taken 2^kLift times, so that those far below the row's greatest, of
// which a long row may have many, stay in f16's normal range.  It costs nothing, for c m
// carries it.  Room is left for the running maximum's 2^8, and for c m as rounded, by up to
// one at scores of 2^24.
template <dp_dtype DT>
constexpr float kLift = DT == DP_F16 ? 6.0f : 0.0f;

// kShare: so many neighbouring waves have the same 32 queries, and 32 keys each of
// every tile; with 1 a wave takes all its keys.
template <dp_dtype DT, int kD, int kWaves, int kShare>
__global__ void __launch_bounds__(64 * kWaves, kWaves == 4 && kShare == 1 ? (kD > 64 && kD <= 96 ? 3 : 2) : 1) k_attention(AttentionArgs a) {
    using T = Tile<kD>;
    constexpr int kRows = 32 * kWaves / kShare, kKeys = keys_of_tile<kD, kWaves, kShare>(), kBlocks = (kD + 31) / 32;
    constexpr int kOwn = kKeys / kShare / 32;  // times 32 keys of a tile that a wave takes
    constexpr int kTileBytes = kKeys * T::kRowBytes;
    constexpr bool kTurns = kWaves == 8 && kShare == 1;  // halves of the waves in turns
    // two turns of a k and a v tile; then, where waves share queries, their sums and maxima
    constexpr int kShares = kShare == 1 ? 0 : kWaves * (kShare == 4 ? kBlocks : 1) * 4096;
    constexpr int kBytes = 4 * kTileBytes > kShares + kWaves * 512 ? 4 * kTileBytes : kShares + kWaves * 512;
    __shared__ __align__(1024) unsigned char lds[kBytes];
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
        f32x16 s[kOwn];
        u32x4 p[kOwn][2];
        const auto clear = [&]() {
#pragma unroll
            for (int j = 0; j < kOwn; ++j) s[j] = zeros();
            __builtin_amdgcn_sched_barrier(0);
        };
        // The scores of the wave's keys of a tile.
        const auto score = [&](const lds_u8* kt) {
#pragma unroll
            for (int j = 0; j < kOwn; ++j)
#pragma unroll
                for (int n = 0; n < kD / 16; ++n) s[j] = mma<DT>(T::read_along(kt, along, j, n), qf[n], s[j]);
        };
        // Their probabilities, with those keys from t on that count.
        const auto soften = [&](int t) {
            if (t + 32 * kOwn - 1 > all_hi)
#pragma unroll
                for (int j = 0; j < kOwn; ++j) hide_behind(s[j], hi - t - 32 * j - 4 * half);
            if (t < all_lo)
#pragma unroll
                for (int j = 0; j < kOwn; ++j) hide_before(s[j], lo - t - 32 * j - 4 * half);
            float top = s[0][0];
#pragma unroll
            for (int j = 0; j < kOwn; ++j)
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
            const float less = m == -kInf ? 0.0f : c * m - kLift<DT>;
            float part[2] = {0.0f, 0.0f};
#pragma unroll
            for (int j = 0; j < kOwn; ++j)
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
        };
        const auto add = [&](const lds_u8* vt) {
#pragma unroll
            for (int j = 0; j < kOwn; ++j)
#pragma unroll
                for (int n = 0; n < 2; ++n)
#pragma unroll
                    for (int x = 0; x < kBlocks; ++x) o[x] = mma<DT>(T::read_across(vt, across, 2 * j + n, x), p[j][n], o[x]);
        };
#pragma unroll
        for (int n = 0; n < 4; ++n) ks.clear(base + n * kTileBytes, sq.dim);
        if constexpr (kTurns) {
            // Half of the waves, one on each SIMD, run one phase behind the other half: while
            // these multiply, those take exponentials.  Tile i of k is read in phases 2 i and
            // 2 i + 1, of v in the next two, and each is stored in the two phases before its
            // first, k by a wave behind its products and v behind its exponentials: alone beside
            // either, the moves made that phase the longer one (8192 rows 1039 TFLOP/s instead
            // of 1071; both in front of the exponentials 948).
            const int late = wave >> 2, n = (to - from + kKeys - 1) / kKeys;
            const bool works = mine < L;
            const auto tile_k = [&](int i) { return base + (i & 1) * kTileBytes; };
            const auto tile_v = [&](int i) { return base + (2 + (i & 1)) * kTileBytes; };
            // past the last tile the first one is loaded again, and not used
            const auto place = [&](int i) { return i < n ? from + i * kKeys : from; };
            const auto move_k = [&](int i) {
                if (i < n) ks.store(tile_k(i), sq.dim);
                ks.load(k, place(i + 1), M, sq.dim);
            };
            const auto move_v = [&](int i) {
                if (i < n) vs.store(tile_v(i), sq.dim);
                vs.load(v, place(i + 1), M, sq.dim);
            };
            ks.load(k, from, M, sq.dim);
            vs.load(v, from, M, sq.dim);
            move_k(0);
            __syncthreads();
            if (late) {
                move_v(0);
                __syncthreads();
            }
            if (works) {
                clear();
                score(tile_k(0));
                ahead<kOwn * (kD / 16), 1, 1, 6>();
                __builtin_amdgcn_sched_barrier(0);
            }
            move_k(1);
            __syncthreads();
            for (int i = 0; i < n; ++i) {
                if (works) soften(from + i * kKeys);
                __builtin_amdgcn_sched_barrier(0);
                move_v(i + late);
                __syncthreads();
                if (i + 1 < n) {
                    if (works) {
                        clear();
                        add(tile_v(i));
                        score(tile_k(i + 1));
                        ahead<2 * kOwn * kBlocks, 1, 2, 4>();
                        ahead<kOwn * (kD / 16), 1, 1, 6>();
                        __builtin_amdgcn_sched_barrier(0);
                    }
                    move_k(i + 2);
                    __syncthreads();
                }
            }
            if (works) {
                __builtin_amdgcn_sched_barrier(0);
                add(tile_v(n - 1));
                ahead<2 * kOwn * kBlocks, 1, 2, 4>();
                __builtin_amdgcn_sched_barrier(0);
            }
            // (as many barriers for the waves in front as for those behind)
            if (!late) __syncthreads();
        } else {
            const auto load = [&](int t) {
                ks.load(k, t, M, sq.dim);
                vs.load(v, t, M, sq.dim);
            };
            const auto store = [&](int turn) {
                ks.store(base + turn, sq.dim);
                vs.store(base + turn + kTileBytes, sq.dim);
            };
            load(from);
            store(0);
            load(from + kKeys < to ? from + kKeys : from);
            __syncthreads();
            int turn = 0;
            for (int t = from; t < to; t += kKeys) {
                const int own = t + 32 * (wave % kShare);
                if (mine < L && own <= some_hi && own + 32 * kOwn > some_lo) {
                    const lds_u8* const kt = base + turn + (own - t) * T::kRowBytes;
                    clear();
                    score(kt);
                    ahead<kOwn * (kD / 16), 1, 1, 6>();
                    soften(own);
                    add(kt + kTileBytes);
                    ahead<2 * kOwn * kBlocks, 1, 2, 4>();
                    __builtin_amdgcn_sched_barrier(0);
                }
                if (t + kKeys < to) {
                    turn ^= 2 * kTileBytes;
                    store(turn);
                    // past the last tile this one is loaded again, and not used
                    load(t + 2 * kKeys < to ? t + 2 * kKeys : t + kKeys);
                    __syncthreads();
                }
            }
        }
    }
    const f32x2 both = halves(sum);
    float total = both[0] + both[1];
    if constexpr (kShare == 4) {
        // Each wave's sums follow the greatest of the waves' maxima, and are added in
        // the waves' order, a block of elements by one wave.
        static_assert(kBlocks <= kWaves, "a block of elements for each wave");
        lds_f32* const stats = (lds_f32*)(base + kShares);
        __syncthreads();
#pragma unroll
        for (int x = 0; x < kBlocks; ++x) share_block(base, kBlocks, wave, x, o[x]);
        stats[wave * 128 + (threadIdx.x & 63)] = m;
        stats[wave * 128 + 64 + (threadIdx.x & 63)] = total;
        __syncthreads();
        float factor[kWaves];
        m = -kInf;
#pragma unroll
        for (int w = 0; w < kWaves; ++w) m = fmaxf(m, stats[w * 128 + (threadIdx.x & 63)]);
        total = 0.0f;
#pragma unroll
        for (int w = 0; w < kWaves; ++w) {
            const float own = stats[w * 128 + (threadIdx.x & 63)];
            factor[w] = own == -kInf ? 0.0f : __builtin_amdgcn_exp2f(c * (own - m));
            total = __builtin_fmaf(factor[w], stats[w * 128 + 64 + (threadIdx.x & 63)], total);
        }
        if (wave < kBlocks) {
            f32x16 sum_o = zeros();
#pragma unroll
            for (int w = 0; w < kWaves; ++w) add_block(base, kBlocks, w, wave, factor[w], sum_o);
            unsigned short* p = static_cast<unsigned short*>(a.out.p) + (at.begin[0] + i) * a.out.ld + h * a.out.head;
            store_block<DT>(p, 32 * wave, i < L, sq.dim, sum_o, total == 0.0f ? 0.0f : 1.0f / total);
        }
    } else if constexpr (kShare == 2) {
        lds_f32* const stats = (lds_f32*)(base + kShares);
        __syncthreads();
        stats[wave * 128 + (threadIdx.x & 63)] = m;
        stats[wave * 128 + 64 + (threadIdx.x & 63)] = total;
        __syncthreads();
        const float m2 = stats[(wave ^ 1) * 128 + (threadIdx.x & 63)], top = fmaxf(m, m2);
        const float own = m == -kInf ? 0.0f : __builtin_amdgcn_exp2f(c * (m - top));
        const float other = m2 == -kInf ? 0.0f : __builtin_amdgcn_exp2f(c * (m2 - top));
        total = own * total + other * stats[(wave ^ 1) * 128 + 64 + (threadIdx.x & 63)];
        m = top;
        const float norm = total == 0.0f ? 0.0f : 1.0f / total;
        unsigned short* const p = static_cast<unsigned short*>(a.out.p) + (at.begin[0] + i) * a.out.ld + h * a.out.head;
        join_pairs<kBlocks>(base, wave, own, other, o,
                            [&](int x, const f32x16& sum_o) { store_block<DT>(p, 32 * x, i < L, sq.dim, sum_o, norm); });
    } else {
        // a query that sees no key: total 0, m -infinity
        store_columns<DT, kD>(a.out, at.begin[0] + i, h, i < L, sq.dim, o, total == 0.0f ? 0.0f : 1.0f / total);
    }
    if (i < L && half == 0 && wave % kShare == 0)
        a.lse[h * sq.rows[0] + at.begin[0] + i] = total == 0.0f ? -kInf : sq.scale * m + kLn2 * (__builtin_amdgcn_logf(total) - kLift<DT>);
}

template <dp_dtype DT, int kD, int kWaves, int kShare>
void launch_one(const AttentionArgs& a, hipStream_t stream) {
    const dim3 grid(static_cast<unsigned>(attention_slots(a.s, 0, 32 * kWaves / kShare) * a.s.heads));
    if (grid.x > 0) hipLaunchKernelGGL((k_attention<DT, kD, kWaves, kShare>), grid, dim3(64 * kWaves), 0, stream, a);
}

template <dp_dtype DT, int kD>
void launch_shape(const AttentionArgs& a, hipStream_t stream) {
    const AttentionShape shape = attention_shape(a.s, 0);
    if (shape == AttentionShape::kSplit) return launch_one<DT, kD, 4, 4>(a, stream);
    if (shape == AttentionShape::kPairs) return launch_one<DT, kD, 8, 2>(a, stream);
    if constexpr (kD > 64)
        if (shape == AttentionShape::kWide) return launch_one<DT, kD, 8, 1>(a, stream);
    launch_one<DT, kD, 4, 1>(a, stream);
}

template <dp_dtype DT>
void launch_dim(const AttentionArgs& a, hipStream_t stream) {
    if (a.s.dim <= 32) launch_shape<DT, 32>(a, stream);
    else if (a.s.dim <= 64) launch_shape<DT, 64>(a, stream);
    else if (a.s.dim <= 80) launch_shape<DT, 80>(a, stream);
    else if (a.s.dim <= 96) launch_shape<DT, 96>(a, stream);
    else launch_shape<DT, 128>(a, stream);
}

}  // namespace

int64_t attention_slots(const Sequences& s, int side, int64_t tile) {
    if (s.count == 0) return 0;
    return s.offsets[side] ? s.rows[side] / tile + s.count : s.count * ((s.length[side] + tile - 1) / tile);
}

// Workgroups of four waves with 32 rows each (of the queries, or in k_attention_dkv of
// the keys) where these are enough for the 256 CUs, but
//  - where they are too few, waves with the same 32 rows share what they go over, and join
//    their sums at the end: two of eight waves, or all four (whose tiles are larger, so that
//    one workgroup, or two for heads of up to 64 elements, fits a CU).  One causal sequence,
//    us as one wave | two | four a run of 32 rows, by workgroups of 128 rows:
//                                    forward        dq             dk and dv
//      heads of 64, 2048 rows   128   30  28  21     39  32  24     61  43  29
//                               256   31  30  32     41  34  38     63  43  42
//                   4096 rows   512   63  59  86     81  70 103    127  91 127
//                               768   77  77 128    100 109 152    149 136
//                              1024                                160 165
//      heads of 128, 2048 rows  128   44  41  36     66  49  47    108  66  50
//                               256   45  42  67     69  51  91    111  72  96
//                    4096 rows  512   99  91 231    146 117 308
//                               768  124 142 345    170 183 464    235 237 494
//                              1024                                291 301 679
//    (between 128 and 256 all four waves' times rise with the workgroups)
//  - eight waves for heads of more than 64 elements whose queries see many keys.  These
//    load each tile half as often, and in the forward pass their halves take turns; but
//    they wait for each other twice as many, and their 256 rows cross the mask's edges
//    further.  Four against eight waves, forward, TFLOP/s of the products that count: causal
//    heads of 128, 8192 rows 981 and 1071, 4096 869 and 963, 2048 867 and 838, 1024 665 and
//    609; without a mask, 2048 rows 923 and 1028; 8192 rows, window 1000, 162 and 178 us; heads of
//    96, 4096 rows 819 and 881, 2048 751 and 742.  dq, heads of 128: 8192 rows 1055 and
//    1122, 4096 967 and 1020, 2048 849 and 836.  They have to be enough to fill the CUs.
// Rows and keys are what the tensors have, for offsets are in device memory: padding counts,
// and a batch of one long sequence and many short ones gets the rule of their mean length.
AttentionShape attention_shape(const Sequences& s, int side) {
    const int heads = side == 0 ? s.heads : s.kv_heads;
    const int64_t groups = attention_slots(s, side, 128) * heads;
    if (groups < (s.dim > 64 ? 160 : 240)) return AttentionShape::kSplit;
    if (groups < (side == 0 ? 640 : 800)) return AttentionShape::kPairs;
    int64_t seen = s.rows[1 - side] / s.count / (s.causal ? 2 : 1);
    if (s.window > 0 && s.window < seen) seen = s.window;
    const bool wide = seen >= 1750 && attention_slots(s, side, 256) * heads >= 512;
    return wide && s.dim > 64 ? AttentionShape::kWide : AttentionShape::kPlain;
}

int64_t attention_groups(const Sequences& s) {
    // (those of 32 rows are taken only where these are few)
    const int64_t q = attention_slots(s, 0, 128) * s.heads, k = attention_slots(s, 1, 128) * s.heads;
    return q > k ? q : k;
}

hipError_t launch_attention(dp_dtype dt, const AttentionArgs& a, hipStream_t stream) {
    if (dt == DP_BF16) launch_dim<DP_BF16>(a, stream);
    else launch_dim<DP_F16>(a, stream);
    return hipGetLastError();
}

}  // namespace dpk

// What the attention's kernels share: tiles of rows in LDS and the fragments
// that the matrix instructions take from them, and the place of a workgroup's
// rows among the sequences.
//
// Products.  mfma 32x32x16 takes from lane l of the left operand row l % 32 and
// of the right one column l % 32, in both the eight positions 8 (l / 32) + 0 .. 7
// of the summed axis; element e of its result is row 8 (e / 4) + 4 (l / 32) +
// e % 4, column l % 32.  A product whose columns are queries (or keys) therefore
// leaves a lane 16 values of its own column, and a sum over the product's rows
// can take them as its right operand where they are: positions 16 s + {4 h, ..,
// 4 h + 3, 8 + 4 h, .., 8 + 4 h + 3} of lane half h = l / 32 are the result's
// elements 8 s .. 8 s + 7.  The left operand of that sum is read in the same
// order.  So probabilities never leave their registers, and row sums and maxima
// are a lane's own but for one exchange between the halves.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "dp_attention.h"
#include "dp_device.h"

namespace dpk {
namespace attn {

typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef short s16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef __attribute__((address_space(3))) s16x4 lds_s16x4;
typedef __attribute__((address_space(3))) u32x4 lds_u32x4;
typedef __attribute__((address_space(3))) f32x4 lds_f32x4;
typedef __attribute__((address_space(3))) float lds_f32;
typedef __attribute__((address_space(3))) unsigned char lds_u8;

constexpr int kThreads = 256;  // of a workgroup, but where it has more waves

constexpr float kLog2e = 1.44269504088896340736f;
constexpr float kLn2 = 0.69314718055994530942f;
constexpr float kInf = __builtin_inff();

template <dp_dtype DT>
__device__ __forceinline__ f32x16 mma(u32x4 a, u32x4 b, f32x16 c) {
    if constexpr (DT == DP_BF16)
        return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
    else
        return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
}

__device__ __forceinline__ f32x16 zeros() {
    f32x16 z;
#pragma unroll
    for (int e = 0; e < 16; ++e) z[e] = 0.0f;
    return z;
}

// Elements 8 s .. 8 s + 7 of a product as a right operand.
template <dp_dtype DT>
__device__ __forceinline__ u32x4 pack8(const f32x16& x, int s) {
    return u32x4{pack2<DT>(x[8 * s], x[8 * s + 1]), pack2<DT>(x[8 * s + 2], x[8 * s + 3]),
                 pack2<DT>(x[8 * s + 4], x[8 * s + 5]), pack2<DT>(x[8 * s + 6], x[8 * s + 7])};
}

// -infinity in the rows of a product behind `last`, or before `first` (of the lane's
// rows 8 (e / 4) + e % 4).
__device__ __forceinline__ void hide_behind(f32x16& x, int last) {
#pragma unroll
    for (int e = 0; e < 16; ++e) x[e] = 8 * (e >> 2) + (e & 3) > last ? -kInf : x[e];
}
__device__ __forceinline__ void hide_before(f32x16& x, int first) {
#pragma unroll
    for (int e = 0; e < 16; ++e) x[e] = 8 * (e >> 2) + (e & 3) < first ? -kInf : x[e];
}

// {x of the lower half's lane, x of the upper half's} of the two lanes that share
// a column, in both of them.
__device__ __forceinline__ f32x2 halves(float x) {
    const unsigned int u = __builtin_bit_cast(unsigned int, x);
    const auto r = __builtin_amdgcn_permlane32_swap(u, u, false, false);
    // (a bit cast of an element of a vector, where it is, takes the first one)
    const unsigned int lower = r[0], upper = r[1];
    return f32x2{__builtin_bit_cast(float, lower), __builtin_bit_cast(float, upper)};
}

// ---- tiles in LDS ------------------------------------------------------------------
// Rows of kD elements lie kLd elements apart (64 or 128: 128 or 256 bytes) in slots
// of 16 bytes.  The slot of a row is permuted by `twist` of the row, so that 16
// rows of one slot (a fragment read along the rows), and four rows of four slots (a
// transposing read), each fall on all 256 bytes that one cycle pair of the banks
// serves.  The permutation is an exclusive or, so a lane's address for the
// next fragment is its first address exclusive-or a constant.
template <int kD>
struct Tile {
    static constexpr int kLd = kD <= 64 ? 64 : 128;
    static constexpr int kRowBytes = 2 * kLd;
    static constexpr int kSlots = kD / 8;  // of a row in use

    static __device__ __forceinline__ int twist(int row) {
        if constexpr (kLd == 128) return (row & 3) << 2 | (row >> 2 & 3);
        else return (row >> 1 & 1) << 2 | (row >> 2 & 3);
    }
    static __device__ __forceinline__ int place(int row, int slot) { return row * kRowBytes + ((slot ^ twist(row)) << 4); }

    // Left operand with the tile's rows as its rows and the elements of a row as
    // the summed axis: rows 32 j + l % 32, elements 16 s + 8 (l / 32) + 0 .. 7, at
    // (along() ^ 32 s) + 32 j rows.
    static __device__ __forceinline__ int along() { return place(threadIdx.x & 31, threadIdx.x >> 5 & 1); }
    static __device__ __forceinline__ u32x4 read_along(const lds_u8* tile, int at, int j, int s) {
        return *(const lds_u32x4*)(tile + (at ^ (32 * s)) + 32 * j * kRowBytes);
    }

    // Left operand with the elements of a row as its rows and the tile's rows as
    // the summed axis: elements 32 b + l % 32, rows 16 s + 4 (l / 32) + 0 .. 3 and 8
    // further.  One transposing load takes a 4 x 16 piece through 16 lanes: lane i of
    // them addresses row i / 4, elements 4 (i % 4), and receives element i of all
    // four rows.
    static __device__ __forceinline__ int across() {
        const int l = threadIdx.x & 63, i = l & 15, row = 4 * (l >> 5) + (i >> 2);
        return place(row, (l & 16) >> 3 | (i >> 1 & 1)) + 8 * (i & 1);
    }
    static __device__ __forceinline__ u32x4 read_across(const lds_u8* tile, int at, int s, int b) {
        const lds_u8* p = tile + 16 * s * kRowBytes;
        const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(p + (at ^ (64 * b))));
        const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(p + 8 * kRowBytes + (at ^ (64 * b) ^ 32)));
        return __builtin_bit_cast(u32x4, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
    }
};

// ---- rows in memory ------------------------------------------------------------------
// One head of a tensor, from its first row.
struct Head {
    const unsigned short* p;
    int64_t ld;
};
__device__ __forceinline__ Head head_of(const dpa_rows& r, int64_t row, int h) {
    return {static_cast<const unsigned short*>(r.p) + row * r.ld + h * r.head, r.ld};
}

// Eight elements of a row, zeros where they do not exist.
__device__ __forceinline__ u32x4 load8(const Head& m, int64_t row, int d, bool there) {
    u32x4 v = {0, 0, 0, 0};
    if (there) v = gload<u32x4, 2>(m.p + row * m.ld + d, 0);
    return v;
}

// Right operands of 32 rows, one a lane: row l % 32, elements 16 s + 8 (l / 32) + 0 .. 7.
template <int kD>
__device__ __forceinline__ void load_right(const Head& m, int64_t row, bool there, int dim, u32x4* o) {
    const int half = threadIdx.x >> 5 & 1;
#pragma unroll
    for (int s = 0; s < kD / 16; ++s) o[s] = load8(m, row, 16 * s + 8 * half, there && 16 * s + 8 * half < dim);
}

// A thread's pieces of a tile of kRows rows on the way through registers: piece i
// is slot threadIdx.x % kWide of row threadIdx.x / kWide + i kStep.  Nothing here
// depends on a branch, so that no load is waited for where it is issued: rows
// behind the last one are read from that one (their scores do not count), and slots
// without elements from the first one; these are zeroed once and never stored.
template <int kD, int kRows, int kAll = kThreads>
struct Stage {
    static constexpr int kWide = Tile<kD>::kLd / 8, kStep = kAll / kWide, kEach = kRows / kStep;
    static_assert(kRows % kStep == 0, "a piece of every row");
    static_assert(kStep % 16 == 0, "the slots' order repeats every 16 rows");
    u32x4 v[kEach];

    static __device__ __forceinline__ int slot() { return threadIdx.x % kWide; }
    static __device__ __forceinline__ int row() { return threadIdx.x / kWide; }
    static __device__ __forceinline__ bool active(int dim) { return 8 * slot() < dim; }

    // The tile that starts at row `first` of `end` > first rows.
    __device__ __forceinline__ void load(const Head& m, int first, int end, int dim) {
        const char* p = reinterpret_cast<const char*>(m.p + first * m.ld) + (active(dim) ? 16 * slot() : 0);
        const uint32_t last = end - 1 - first, ld = static_cast<uint32_t>(2 * m.ld);
#pragma unroll
        for (int i = 0; i < kEach; ++i) {
            const uint32_t r = row() + i * kStep;
            v[i] = gload<u32x4, 2>(p + static_cast<uint64_t>(r < last ? r : last) * ld, 0);
        }
    }
    __device__ __forceinline__ void store(lds_u8* tile, int dim) const {
        const int at = Tile<kD>::place(row(), slot());
        if (active(dim)) {
#pragma unroll
            for (int i = 0; i < kEach; ++i) *(lds_u32x4*)(tile + at + i * kStep * Tile<kD>::kRowBytes) = v[i];
        }
    }
    static __device__ __forceinline__ void clear(lds_u8* tile, int dim) {
        const int at = Tile<kD>::place(row(), slot());
        if (!active(dim)) {
#pragma unroll
            for (int i = 0; i < kEach; ++i) *(lds_u32x4*)(tile + at + i * kStep * Tile<kD>::kRowBytes) = u32x4{0, 0, 0, 0};
        }
    }
};

// The order of instructions between two branches, for the scheduler: next are n
// matrix products or LDS reads.  Left alone, it reads each fragment right before
// its product and waits for it there.
template <int n>
__device__ __forceinline__ void products() { __builtin_amdgcn_sched_group_barrier(0x008, n, 0); }
template <int n>
__device__ __forceinline__ void reads() { __builtin_amdgcn_sched_group_barrier(0x100, n, 0); }
// kCount times kProducts products with kReads reads, the reads kAhead times before.
template <int kCount, int kProducts, int kReads, int kAhead>
__device__ __forceinline__ void ahead() {
    constexpr int kFirst = kAhead < kCount ? kAhead : kCount;
    reads<kFirst * kReads>();
#pragma unroll
    for (int i = 0; i < kCount - kFirst; ++i) {
        products<kProducts>();
        reads<kReads>();
    }
    products<kFirst * kProducts>();
}

// 32 columns (one a lane) and 32 rows, d .. d + 31, of a product's sum as elements of
// rows in memory, of which the first `dim` exist: each pair of lanes first exchanges
// the words of two groups of eight, so that every lane stores 16 bytes.
template <dp_dtype DT>
__device__ __forceinline__ void store_block(unsigned short* p, int d, bool there, int dim, const f32x16& x, float factor) {
    const int half = threadIdx.x >> 5 & 1;
#pragma unroll
    for (int g = 0; g < 2; ++g) {
        unsigned int w[2][2];
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
            for (int e = 0; e < 2; ++e)
                w[u][e] = pack2<DT>(x[8 * g + 4 * u + 2 * e] * factor, x[8 * g + 4 * u + 2 * e + 1] * factor);
        const auto lo = __builtin_amdgcn_permlane32_swap(w[0][0], w[1][0], false, false);
        const auto hi = __builtin_amdgcn_permlane32_swap(w[0][1], w[1][1], false, false);
        const int at = d + 16 * g + 8 * half;
        if (there && at < dim) gstore<u32x4, 2>(p + at, 0, u32x4{lo[0], hi[0], lo[1], hi[1]});
    }
}
template <dp_dtype DT, int kD>
__device__ __forceinline__ void store_columns(const dpa_rows& r, int64_t row, int h, bool there, int dim, const f32x16* x,
                                              float factor) {
    unsigned short* p = static_cast<unsigned short*>(r.p) + row * r.ld + h * r.head;
#pragma unroll
    for (int b = 0; b < (kD + 31) / 32; ++b) store_block<DT>(p, 32 * b, there, dim, x[b], factor);
}

// The waves' shares of a sum in LDS: block b of this wave, and back that of wave w.
__device__ __forceinline__ void share_block(lds_u8* at, int blocks, int wave, int b, const f32x16& x) {
#pragma unroll
    for (int g = 0; g < 4; ++g)
        *(lds_f32x4*)(at + ((wave * blocks + b) * 4 + g) * 1024 + 16 * (threadIdx.x & 63)) =
            f32x4{x[4 * g], x[4 * g + 1], x[4 * g + 2], x[4 * g + 3]};
}
__device__ __forceinline__ void add_block(const lds_u8* at, int blocks, int wave, int b, float factor, f32x16& x) {
#pragma unroll
    for (int g = 0; g < 4; ++g) {
        const f32x4 v = *(const lds_f32x4*)(at + ((wave * blocks + b) * 4 + g) * 1024 + 16 * (threadIdx.x & 63));
#pragma unroll
        for (int e = 0; e < 4; ++e) x[4 * g + e] = __builtin_fmaf(factor, v[e], x[4 * g + e]);
    }
}

// The two waves of a pair (2 i and 2 i + 1) join their shares of a sum, a block of 32
// elements each at a time, the even one the even blocks: use(block, its sum).  Each
// wave's share counts `own` times, the other's `other` times.
template <int kBlocks, typename Use>
__device__ __forceinline__ void join_pairs(lds_u8* at, int wave, float own, float other, const f32x16* o, Use&& use) {
    const bool odd = wave & 1;
#pragma unroll
    for (int x = 0; x < kBlocks; x += 2) {
        const f32x16 even_block = o[x], odd_block = o[x + 1 < kBlocks ? x + 1 : x];
        f32x16 sum, give;
#pragma unroll
        for (int e = 0; e < 16; ++e) {
            sum[e] = own * (odd ? odd_block[e] : even_block[e]);
            give[e] = odd ? even_block[e] : odd_block[e];
        }
        __syncthreads();
        share_block(at, 1, wave, 0, give);
        __syncthreads();
        if (x + odd < kBlocks) {
            add_block(at, 1, wave ^ 1, 0, other, sum);
            use(x + odd, sum);
        }
    }
}

// ---- sequences --------------------------------------------------------------------------
// A workgroup's head, its sequence and its tile's place in it.
struct Place {
    int head;
    int64_t begin[2];  // first rows of the sequence, among the queries and the keys
    int length[2];
    int tile;   // of the sequence, in rows of the tile's size
    int tiles;  // of the sequence
};

__device__ __forceinline__ int64_t offset_at(const Sequences& s, int side, int64_t i) {
    const int64_t x = s.offset_bytes == 4 ? gload<int32_t>(s.offsets[side], i) : gload<int64_t>(s.offsets[side], i);
    return x < 0 ? 0 : x > s.rows[side] ? s.rows[side] : x;
}

// Member i of n, so that the members with the same i % 8, whose workgroups run on one
// XCD, are neighbours: heads that read the same keys share its cache.
__device__ __forceinline__ int neighbour(int i, int n) { return n % 8 == 0 ? i % 8 * (n / 8) + i / 8 : i; }

// The tile of this workgroup, of kRows rows of the queries (side 0) or keys (1), for
// one of `heads` heads; false where it has none.  Tiles of sequences of one length come
// in the order of their work, the most first (`last_first`: in a sequence from its end),
// for all sequences and heads at once, so that what is left at the end of the launch is
// small: head by head instead, a fifth to a quarter of the CUs' time was lost there.
//
// With offsets, tiles are found by slots in the order of the sequences, for all heads at
// once, and heaviest first in each sequence only: a long one behind short ones starts late
// (8191 packed rows: CUs busy 69 to 83% of the time).  Sequence s has the slots from begin / kRows + s on: these rise
// with s, and as the next sequence begins behind the last row of this one, there are
// enough of them for all its tiles.  Some are left over.
template <int kRows>
__device__ __forceinline__ bool find(const Sequences& s, int side, int heads, bool last_first, Place& o) {
    const int job = blockIdx.x;
    int n, rank;  // the sequence, and which of its tiles
    if (s.offsets[side]) {
        const int slot = job / heads;
        o.head = neighbour(job % heads, heads);
        // the last sequence whose first slot is not behind this one, 64 samples at a time
        int lo = 0, hi = s.count;  // in [lo, hi)
        while (hi - lo > 1) {
            const int each = (hi - lo + 63) / 64;
            const int at = lo + static_cast<int>(threadIdx.x & 63) * each;
            const bool before = at < hi && offset_at(s, side, static_cast<int64_t>(at) * s.step) / kRows + at <= slot;
            const int found = __popcll(__ballot(before));
            lo = found > 0 ? lo + (found - 1) * each : lo;
            hi = lo + each < hi ? lo + each : hi;
        }
        n = __builtin_amdgcn_readfirstlane(lo);
        rank = slot - (static_cast<int>(offset_at(s, side, static_cast<int64_t>(n) * s.step) / kRows) + n);
    } else {
        const int groups = heads * s.count;
        rank = job / groups;
        const int group = neighbour(job % groups, groups);
        n = group / heads;
        o.head = group % heads;
    }
#pragma unroll
    for (int x = 0; x < 2; ++x) {
        int64_t b, e;
        if (s.offsets[x]) {
            b = offset_at(s, x, static_cast<int64_t>(n) * s.step);
            e = offset_at(s, x, static_cast<int64_t>(n) * s.step + 1);
        } else {
            b = n * s.length[x];
            e = b + s.length[x];
        }
        o.begin[x] = b;
        o.length[x] = static_cast<int>(e > b ? e - b : 0);
    }
    o.tiles = (o.length[side] + kRows - 1) / kRows;
    o.tile = last_first ? o.tiles - 1 - rank : rank;
    return rank >= 0 && rank < o.tiles;
}

}  // namespace attn
}  // namespace dpk

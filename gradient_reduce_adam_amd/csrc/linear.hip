// gfx950 kernel of a linear layer's weight gradient from its 8-bit input:
// G[o][i] = sum over the tokens t of dy[t][o] x[t][i], added to (or written
// over) binary32 accumulators.
//
// A product on the matrix cores, with the token axis summed: both operands lie
// with that axis slow, so a tile of 64 tokens by 256 columns of each is staged
// in LDS as it lies in memory, in 16 bits, and fragments are read with the
// transposing LDS load, which gives a lane four consecutive tokens of its column.
//  - x is read as codes and scale bytes, half the bytes of 16 bits, and decoded
//    on the way to LDS (codes times a power of two are exact in 16 bits: one
//    conversion instruction for two).
//  - A workgroup of 8 waves makes a tile of 256 x 256 weights, each wave 128 x
//    64 as 4 x 2 products of 32 x 32 x 16, in 128 accumulator registers a
//    lane.  Two LDS buffers (128 KiB): while one is multiplied, the next 64
//    tokens are written to the other, and those after them are loaded.
//  - LDS rows are 512 bytes, so four consecutive tokens of one column would
//    hit the same banks: 64-byte slots are permuted by the token's low two
//    bits (slot ^ (token & 3)), which spreads every fragment read over all
//    banks.
// The matrix cores bound it, at the clock that they sustain (1.9 of 2.4 GHz):
// 11008 x 4096 weights from 8192 tokens take 628 to 704 us on different cards,
// 1050 to 1175 TFLOP/s, with the matrix pipes busy 67% of the time that the CUs
// are; the LDS reads (192 KiB a step, against 8.4 MFLOP) come next.
//
// Few tiles and many tokens leave CUs idle, so the token axis is then split
// over several workgroups, whose tiles go to the workspace and are added in
// order by a second launch.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "dp_device.h"
#include "dp_layers.h"

namespace dpk {
namespace {

constexpr int kTileCols = 256;  // columns of either operand per workgroup
constexpr int kTileTokens = 64;
constexpr int kThreads = 512;
constexpr int kTileBytes = kTileTokens * kTileCols * 2;

typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef short s16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef float f32x16 __attribute__((ext_vector_type(16)));

struct LinearArgs {
    const void* dy[DP_MAX_REPLICAS];
    const unsigned char* codes[DP_MAX_REPLICAS];
    const unsigned char* scales[DP_MAX_REPLICAS];
    float* acc[DP_MAX_REPLICAS];
    float* part;  // [splits][n][outputs * inputs] with splits > 1
    int64_t tokens, ld_dy, ld_codes, ld_scales;
    int64_t outputs, inputs;
    int32_t n, tiles_o, tiles_i, splits;
    int64_t split_tokens;  // of one split, a multiple of kTileTokens
    bool overwrite;
};

// Byte offset in a tile of column c (a multiple of 8) of token k.
__device__ __forceinline__ int at(int k, int c) { return k * (2 * kTileCols) + ((2 * c) ^ ((k & 3) << 6)); }

template <dp_dtype DT>
__device__ __forceinline__ unsigned int decode2(unsigned int codes, float unit, int half) {
    if constexpr (DT == DP_BF16) {
        return half ? __builtin_bit_cast(unsigned int, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(codes, unit, true))
                    : __builtin_bit_cast(unsigned int, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(codes, unit, false));
    } else {
        return half ? __builtin_bit_cast(unsigned int, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(codes, unit, true))
                    : __builtin_bit_cast(unsigned int, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(codes, unit, false));
    }
}

template <dp_dtype DT>
__device__ __forceinline__ f32x16 mma(s16x8 a, s16x8 b, f32x16 c) {
    if constexpr (DT == DP_BF16)
        return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
    else
        return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
}

typedef __attribute__((address_space(3))) s16x4 lds_s16x4;
typedef __attribute__((address_space(3))) u32x4 lds_u32x4;
typedef __attribute__((address_space(3))) unsigned char lds_u8;

// Fragments: of 32 columns and 16 tokens lane l gets column l % 32 and tokens
// 8 (l / 32) + 0 .. 7.  One transposing load takes a 4 x 16 piece through 16 lanes: lane
// i of them addresses token i / 4, columns 4 (i % 4), and receives column i of
// all four tokens.  `place` is this lane's offset in a tile for columns from c0
// (a multiple of 32); tokens from k0 (a multiple of 16) lie k0 rows further.
__device__ __forceinline__ int place(int c0) {
    const int l = threadIdx.x & 63, i = l & 15;
    const int k = 8 * (l >> 5) + (i >> 2), c = c0 + (l & 16) + 4 * (i & 3);
    return k * (2 * kTileCols) + ((2 * c) ^ ((k & 3) << 6));
}
__device__ __forceinline__ s16x8 fragment(const lds_u8* p) {
    const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)p);
    const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(p + 4 * 2 * kTileCols));
    return __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
}

// One workgroup's operands and place.
struct Job {
    const unsigned char* dy;
    const unsigned char* codes;
    const unsigned char* scales;
    int64_t o0, i0;  // first output and input of the tile
};

// ---- staging -------------------------------------------------------------------
// A thread's share of one tile on its way through registers: dy as 4 pieces of 8
// elements (piece q * 512 + thread: token piece / 32), x as the codes of 16
// columns of tokens thread / 16 and thread / 16 + 32, with their scale bytes.
struct Stage {
    u32x4 dy[4];
    u32x4 codes[2];
    unsigned int unit[2];
};

// Where a thread reads its pieces of a whole tile: offsets from the tile's first
// token.  A piece that starts before the last column is read whole, into the
// next token's row where the columns end within it (every whole tile has a
// token behind it); one that starts behind it is read from the last eight or
// sixteen columns.  The products of columns that do not exist are not stored.
struct Pieces {
    uint32_t dy, codes, scales;
};

__device__ __forceinline__ Pieces pieces(const LinearArgs& a, const Job& j, bool whole, int64_t ld_dy, int64_t ld_codes,
                                         int64_t ld_scales) {
    int64_t o = j.o0 + ((threadIdx.x & 31) << 3), i = j.i0 + ((threadIdx.x & 15) << 4);
    // without a whole tile nothing is used, and no piece may pass the row's end
    o = o < (whole ? a.outputs : a.outputs - 7) ? o : a.outputs - 8;
    i = i < (whole ? a.inputs : a.inputs - 15) ? i : a.inputs - 16;
    return {static_cast<uint32_t>(2 * ((threadIdx.x >> 5) * ld_dy + o)),
            static_cast<uint32_t>((threadIdx.x >> 4) * ld_codes + i),
            static_cast<uint32_t>((threadIdx.x >> 4) * ld_scales + i / DPL_GROUP)};
}

// The tile whose first token is row 0 of the three addresses.
__device__ __forceinline__ void load_full(const unsigned char* dy, const unsigned char* codes, const unsigned char* scales,
                                          int64_t ld_dy, int64_t ld_codes, int64_t ld_scales, const Pieces& p, Stage& s) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        s.dy[2 * h] = gload<u32x4, 2>(dy + 2 * h * 32 * ld_dy + p.dy, 0);
        s.dy[2 * h + 1] = gload<u32x4, 2>(dy + (2 * h + 1) * 32 * ld_dy + p.dy, 0);
        s.codes[h] = gload<u32x4, 1>(codes + h * 32 * ld_codes + p.codes, 0);
        s.unit[h] = gload<unsigned char>(scales + h * 32 * ld_scales + p.scales, 0);
    }
}

// 16 codes of which `valid` exist, for rows of at least 16: a piece that the
// row's end cuts short is loaded from 16 - valid columns earlier and moved down.
__device__ __forceinline__ u32x4 codes_piece(const unsigned char* p, int valid) {
    u32x4 v = gload<u32x4, 1>(p - (16 - valid), 0);
    const int s = 16 - valid;
    if (s & 8) v = u32x4{v[2], v[3], 0, 0};
    if (s & 4) v = u32x4{v[1], v[2], v[3], 0};
    const unsigned int bits = 8 * (s & 3);
    return u32x4{__builtin_amdgcn_alignbit(v[1], v[0], bits), __builtin_amdgcn_alignbit(v[2], v[1], bits),
                 __builtin_amdgcn_alignbit(v[3], v[2], bits), __builtin_amdgcn_alignbit(0, v[3], bits)};
}

// Tokens [t, end) of a tile, with zeros for tokens and columns that do not exist,
// which are not read.
__device__ __forceinline__ void load_checked(const LinearArgs& a, const Job& j, int64_t t, int64_t end, Stage& s) {
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        const int id = q * kThreads + threadIdx.x, k = id >> 5, c = (id & 31) << 3;
        const int64_t left = a.outputs - (j.o0 + c);
        const int valid = t + k < end ? left >= 8 ? 8 : left > 0 ? static_cast<int>(left) : 0 : 0;
        Raw<DP_BF16, 8> piece = load_raw<DP_BF16, 8>(j.dy, (t + k) * a.ld_dy + j.o0 + c, valid, a.outputs >= 8);
        settle<DP_BF16, 8>(piece, valid, a.outputs >= 8);  // of either 16-bit type
        s.dy[q] = u32x4{piece.w[0], piece.w[1], piece.w[2], piece.w[3]};
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const int k = (threadIdx.x >> 4) + 32 * h, c = (threadIdx.x & 15) << 4;
        const int64_t left = a.inputs - (j.i0 + c);
        const int valid = t + k < end ? left >= 16 ? 16 : left > 0 ? static_cast<int>(left) : 0 : 0;
        const unsigned char* p = j.codes + (t + k) * a.ld_codes + j.i0 + c;
        s.codes[h] = u32x4{0, 0, 0, 0};
        s.unit[h] = 127;
        if (valid == 0) continue;
        if (a.inputs >= 16) {
            s.codes[h] = codes_piece(p, valid);
        } else {
#pragma unroll
            for (int i = 0; i < 15; ++i)
                s.codes[h][i / 4] |= i < valid ? static_cast<unsigned int>(gload<unsigned char>(p, i)) << (8 * (i % 4)) : 0u;
        }
        s.unit[h] = gload<unsigned char>(j.scales, (t + k) * a.ld_scales + (j.i0 + c) / DPL_GROUP);
    }
}

// Half h of a stage into a pair of tiles (dy, x behind it): `dy`, `x` are this
// thread's places for token 0 of each.
template <dp_dtype DT>
__device__ __forceinline__ void store_half(const Stage& s, int h, lds_u8* dy, lds_u8* x) {
#pragma unroll
    for (int q = 2 * h; q < 2 * h + 2; ++q) *(lds_u32x4*)(dy + q * 16 * (2 * kTileCols)) = s.dy[q];
    const float unit = __builtin_bit_cast(float, s.unit[h] << 23);
#pragma unroll
    for (int e = 0; e < 2; ++e)
        *(lds_u32x4*)(x + h * 32 * (2 * kTileCols) + 16 * e) =
            u32x4{decode2<DT>(s.codes[h][2 * e], unit, 0), decode2<DT>(s.codes[h][2 * e], unit, 1),
                  decode2<DT>(s.codes[h][2 * e + 1], unit, 0), decode2<DT>(s.codes[h][2 * e + 1], unit, 1)};
}

// The order of a group of eight products and what goes on beside them: the
// twelve fragment loads for the next group behind the first products, then with
// kKind >= 1 four LDS writes, and with kKind 2 the eight global loads.  Left
// alone, the compiler gathers the loads right before their results are needed
// and the matrix cores wait.
template <int kKind>
__device__ __forceinline__ void spread() {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
        if (kKind == 0 && i < 6) __builtin_amdgcn_sched_group_barrier(0x100, 2, 0);
        if (kKind >= 1 && i < 4) __builtin_amdgcn_sched_group_barrier(0x100, 3, 0);
        if (kKind >= 1 && i >= 4) __builtin_amdgcn_sched_group_barrier(0x200, 1, 0);
        if (kKind == 2 && i >= 4) __builtin_amdgcn_sched_group_barrier(0x020, 2, 0);
    }
    __builtin_amdgcn_sched_barrier(0);
}

// Rows of the result are outputs (columns inputs), or inputs with kSwap; the
// lanes of a wave run along the columns.  The last 1 to 64 tokens are loaded
// with checks and multiplied first, then the whole tiles before them; without
// kPieces (fewer than 8 outputs or 16 inputs) those are loaded with checks too.
template <dp_dtype DT, bool kSwap, bool kPieces>
__global__ void __launch_bounds__(kThreads) k_linear(LinearArgs a) {
    __shared__ __align__(1024) unsigned char lds[4 * kTileBytes];  // two turns of a dy and an x tile
    // tiles in the order of their operands' reuse: neighbouring workgroups of one
    // XCD (every eighth) take tiles next to each other
    const int jobs = gridDim.x, per = jobs / 8, extra = jobs % 8, xcd = blockIdx.x % 8;
    const int id = xcd * per + (xcd < extra ? xcd : extra) + blockIdx.x / 8;
    const int tiles = a.tiles_o * a.tiles_i, tile = id % tiles;
    const int r = id / tiles % a.n, split = id / tiles / a.n;
    const int band = tile / (8 * a.tiles_i), rows = a.tiles_o - 8 * band < 8 ? a.tiles_o - 8 * band : 8;
    const int within = tile - band * 8 * a.tiles_i;
    Job j;
    j.dy = static_cast<const unsigned char*>(a.dy[r]);
    j.codes = a.codes[r];
    j.scales = a.scales[r];
    j.o0 = static_cast<int64_t>(8 * band + within % rows) * kTileCols;
    j.i0 = static_cast<int64_t>(within / rows) * kTileCols;
    const int64_t t0 = split * a.split_tokens;
    const int64_t t1 = t0 + a.split_tokens < a.tokens ? t0 + a.split_tokens : a.tokens;

    const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), l = threadIdx.x & 63;
    const int wm = (w >> 2) * 128, wn = (w & 3) * 64;  // this wave's part of the tile: rows, columns
    f32x16 c[4][2];
#pragma unroll
    for (int m = 0; m < 4; ++m)
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
            for (int e = 0; e < 16; ++e) c[m][n][e] = 0.0f;

    // Fragments are read one group of 16 tokens ahead of their products, also
    // across the barrier: while group 3 of a tile is multiplied, group 0 of the
    // next one is read.  A tile is loaded into registers one step before it is
    // written to LDS, and two before it is multiplied.
    lds_u8* const base = (lds_u8*)lds;
    int left[4], right[2];
#pragma unroll
    for (int m = 0; m < 4; ++m) left[m] = place(wm + 32 * m) + (kSwap ? kTileBytes : 0);
#pragma unroll
    for (int n = 0; n < 2; ++n) right[n] = place(wn + 32 * n) + (kSwap ? 0 : kTileBytes);
    const int put_dy = at(threadIdx.x >> 5, (threadIdx.x & 31) << 3);
    const int put_x = kTileBytes + at(threadIdx.x >> 4, (threadIdx.x & 15) << 4);
    s16x8 p[2][4], q[2][2];
    auto read = [&](int turn, int k, int b) {  // turn: byte offset of the pair of tiles
        const lds_u8* from = base + turn + k * 16 * (2 * kTileCols);
#pragma unroll
        for (int m = 0; m < 4; ++m) p[b][m] = fragment(from + left[m]);
#pragma unroll
        for (int n = 0; n < 2; ++n) q[b][n] = fragment(from + right[n]);
    };
    auto multiply = [&](int b) {
#pragma unroll
        for (int m = 0; m < 4; ++m)
#pragma unroll
            for (int n = 0; n < 2; ++n) c[m][n] = mma<DT>(p[b][m], q[b][n], c[m][n]);
    };
    const int64_t full = t1 > t0 ? (t1 - t0 - 1) / kTileTokens : -1;  // whole tiles before the last tokens
    if (full >= 0) {
        Stage s;
        load_checked(a, j, t0 + full * kTileTokens, t1, s);
        store_half<DT>(s, 0, base + put_dy, base + put_x);
        store_half<DT>(s, 1, base + put_dy, base + put_x);
        // Past the end the last whole tile is loaded again, and not used; without
        // a whole tile that is the first token, at a stride of 0.
        int64_t t = t0;  // the next tile to load
        const int64_t last = full > 0 ? t0 + (full - 1) * kTileTokens : t0;
        const int64_t ld_dy = full > 0 ? a.ld_dy : 0, ld_codes = full > 0 ? a.ld_codes : 0;
        const int64_t ld_scales = full > 0 ? a.ld_scales : 0;
        const Pieces at_row = pieces(a, j, full > 0, ld_dy, ld_codes, ld_scales);
        auto load = [&]() {
            const int64_t from = t < last ? t : last;
            if constexpr (kPieces)
                load_full(j.dy + 2 * from * a.ld_dy, j.codes + from * a.ld_codes, j.scales + from * a.ld_scales, ld_dy,
                          ld_codes, ld_scales, at_row, s);
            else load_checked(a, j, from, from + kTileTokens < t1 ? from + kTileTokens : t1, s);
            t += kTileTokens;
        };
        load();
        __syncthreads();
        int turn = 0;
        read(turn, 0, 0);
        for (int64_t i = 0; i <= full; ++i) {
            const int other = turn ^ (2 * kTileBytes);
            read(turn, 1, 1);
            multiply(0);
            spread<0>();
            read(turn, 2, 0);
            store_half<DT>(s, 0, base + other + put_dy, base + other + put_x);
            multiply(1);
            spread<1>();
            read(turn, 3, 1);
            store_half<DT>(s, 1, base + other + put_dy, base + other + put_x);
            load();
            multiply(0);
            spread<2>();
            __syncthreads();
            __builtin_amdgcn_sched_barrier(0);
            turn = other;
            read(turn, 0, 0);
            multiply(1);
            spread<0>();
        }
    }

    // Element e of a 32 x 32 product: row 8 (e / 4) + 4 (l / 32) + e % 4, column l % 32.
    // Products 2 m + n in turn, each as 16 rows of 32 columns twice, at a
    // uniform address and a lane's offset; the accumulators of the next two are
    // on their way while one is stored.
    const int64_t row0 = (kSwap ? j.i0 : j.o0) + wm, col0 = (kSwap ? j.o0 : j.i0) + wn;
    const int64_t height = kSwap ? a.inputs : a.outputs, width = kSwap ? a.outputs : a.inputs;
    const bool over = a.overwrite || a.splits > 1;
    float* out = a.splits > 1 ? a.part + (static_cast<int64_t>(split) * a.n + r) * height * width : a.acc[r];
    char* corner = reinterpret_cast<char*>(out + row0 * width + col0);
    const uint32_t lane = static_cast<uint32_t>(4 * ((l >> 5) * 4 * width + (l & 31)));
    auto place_of = [&](int k, int e) {
        return corner + 4 * ((32 * (k >> 1) + 8 * (e >> 2) + (e & 3)) * width + 32 * (k & 1)) + lane;
    };
    if (row0 + 128 <= height && col0 + 64 <= width) {  // all of the wave's 128 x 64 elements exist
        float old[3][16];
        auto fetch = [&](int k) {
#pragma unroll
            for (int e = 0; e < 16; ++e) old[k % 3][e] = gload<float>(place_of(k, e), 0);
        };
        if (!over) {
            fetch(0);
            fetch(1);
        }
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            __builtin_amdgcn_sched_barrier(0);
            if (!over && k + 2 < 8) fetch(k + 2);
#pragma unroll
            for (int e = 0; e < 16; ++e)
                gstore<float>(place_of(k, e), 0, over ? c[k >> 1][k & 1][e] : old[k % 3][e] + c[k >> 1][k & 1][e]);
        }
        return;
    }
    // At the matrix' edges eight rows at a time, most of them whole or absent.
    const int there = static_cast<int>(height - row0 < 128 ? height - row0 : 128);
    const int64_t cols = width - col0 - (l & 31);
#pragma unroll
    for (int k = 0; k < 8; ++k) {
        if (32 * (k & 1) >= cols) continue;
#pragma unroll
        for (int g = 0; g < 4; ++g) {
            const int row = 32 * (k >> 1) + 8 * g;
            if (row >= there) continue;
            const bool whole = row + 8 <= there;
            float v[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const bool in = whole || row + 4 * (l >> 5) + e < there;
                v[e] = c[k >> 1][k & 1][4 * g + e];
                if (!over && in) v[e] = gload<float>(place_of(k, 4 * g + e), 0) + v[e];
            }
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (whole || row + 4 * (l >> 5) + e < there) gstore<float>(place_of(k, 4 * g + e), 0, v[e]);
        }
    }
}

// Adds the splits' tiles of every replica, in order, into the accumulators.
__global__ void __launch_bounds__(256) k_linear_join(LinearArgs a) {
    const int64_t size = a.outputs * a.inputs;
    const int r = blockIdx.y;
    const int64_t i = (static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x) * 4;
    const int64_t left = size - i;
    const int valid = left >= 4 ? 4 : left > 0 ? static_cast<int>(left) : 0;
    float s[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    constexpr int kBatch = 8;  // partial sums on their way together
    for (int k0 = 0; k0 < a.splits; k0 += kBatch) {
        float v[kBatch][4];
#pragma unroll
        for (int k = 0; k < kBatch; ++k)
            load_n<DP_F32, 4>(a.part + (static_cast<int64_t>(k0 + k) * a.n + r) * size, i, k0 + k < a.splits ? valid : 0, v[k]);
#pragma unroll
        for (int k = 0; k < kBatch; ++k)
#pragma unroll
            for (int e = 0; e < 4; ++e) s[e] += v[k][e];
    }
    if (!a.overwrite) {
        float v[4];
        load_n<DP_F32, 4>(a.acc[r], i, valid, v);
#pragma unroll
        for (int e = 0; e < 4; ++e) s[e] = v[e] + s[e];
    }
    store_n<DP_F32, 4>(a.acc[r], i, valid, s);
}

int64_t tiles_of(int64_t outputs, int64_t inputs, int n) {
    return ((outputs + kTileCols - 1) / kTileCols) * ((inputs + kTileCols - 1) / kTileCols) * n;
}

// Workgroups that share the tokens of one tile, where all tiles together leave
// CUs idle: the number that takes least by what was measured, 1.7 us for 64
// tokens of a tile, and with more than one workgroup 4 us for the second launch,
// 0.12 us for each partial sum that it adds, and all of them written and read at
// 5 TB/s.
int splits_of(int64_t outputs, int64_t inputs, int64_t tokens, int n) {
    const int64_t steps = (tokens + kTileTokens - 1) / kTileTokens;
    const int64_t most = 256 / tiles_of(outputs, inputs, n);
    const double part = 0.12 + 8.0 * static_cast<double>(outputs * inputs) * n / 5e6;  // us a workgroup
    int best = 1;
    double least = 1.7 * static_cast<double>(steps);
    for (int64_t s = 2; s <= most && s <= steps; ++s) {
        const double t = 1.7 * static_cast<double>((steps + s - 1) / s) + 4.0 + part * static_cast<double>(s);
        if (t < least) {
            least = t;
            best = static_cast<int>(s);
        }
    }
    return best;
}

}  // namespace

int64_t linear_jobs(int64_t outputs, int64_t inputs, int64_t tokens, int n) {
    return tiles_of(outputs, inputs, n) * splits_of(outputs, inputs, tokens, n);
}

// For the most workgroups that any number of tokens up to this one may be
// shared by: at most 256 tiles, 64 MiB.
size_t linear_workspace(int64_t outputs, int64_t inputs, int64_t tokens, int n) {
    const int64_t steps = (tokens + kTileTokens - 1) / kTileTokens, most = 256 / tiles_of(outputs, inputs, n);
    const int64_t s = most < steps ? most : steps;
    return s > 1 ? static_cast<size_t>(4 * s * n) * static_cast<size_t>(outputs * inputs) : 0;
}

hipError_t launch_linear(dp_dtype dt, const LinearGrad& g, void* workspace, hipStream_t stream) {
    LinearArgs a{};
    for (int r = 0; r < g.n; ++r) {
        a.dy[r] = g.rows[r].dy;
        a.codes[r] = static_cast<const unsigned char*>(g.rows[r].codes);
        a.scales[r] = static_cast<const unsigned char*>(g.rows[r].scales);
        a.acc[r] = g.acc[r];
    }
    a.part = static_cast<float*>(workspace);
    a.tokens = g.tokens;
    a.ld_dy = g.ld_dy;
    a.ld_codes = g.ld_codes;
    a.ld_scales = g.ld_scales;
    a.outputs = g.outputs;
    a.inputs = g.inputs;
    a.n = g.n;
    a.tiles_o = static_cast<int32_t>((g.outputs + kTileCols - 1) / kTileCols);
    a.tiles_i = static_cast<int32_t>((g.inputs + kTileCols - 1) / kTileCols);
    a.splits = splits_of(g.outputs, g.inputs, g.tokens, g.n);
    a.split_tokens = ((g.tokens + a.splits - 1) / a.splits + kTileTokens - 1) / kTileTokens * kTileTokens;
    a.overwrite = g.overwrite;
    const dim3 grid(static_cast<unsigned>(linear_jobs(g.outputs, g.inputs, g.tokens, g.n)));
#define DP_GO(D, S)                                                                                              \
    if (dt == D && g.transposed == S) {                                                                         \
        if (g.pieces) hipLaunchKernelGGL((k_linear<D, S, true>), grid, dim3(kThreads), 0, stream, a);              \
        else hipLaunchKernelGGL((k_linear<D, S, false>), grid, dim3(kThreads), 0, stream, a);                   \
    }
    DP_GO(DP_BF16, false)
    DP_GO(DP_BF16, true)
    DP_GO(DP_F16, false)
    DP_GO(DP_F16, true)
#undef DP_GO
    hipError_t e = hipGetLastError();
    if (e != hipSuccess || a.splits == 1) return e;
    const dim3 jgrid(static_cast<unsigned>((g.outputs * g.inputs + 1023) / 1024), static_cast<unsigned>(g.n));
    hipLaunchKernelGGL(k_linear_join, jgrid, dim3(256), 0, stream, a);
    return hipGetLastError();
}

}  // namespace dpk

// gfx950 kernels of the embedding: the scaled lookup, and its gradient by
// sorted tokens.
//
// Lookup.  out[t] = scale * W[id_t]: a gather of rows, bound by HBM (the rows
// touched, once, and the output).  One wave64 workgroup moves up to 2048
// elements of one row, 8 per lane and access.
//
// Gradient.  G[v] = scale * sum over the tokens t with id_t = v of dy[t].  The
// sums need a fixed order, so no floating-point atomics: the tokens of each
// replica are sorted by id, stably, and every row's tokens are then one run
// of the sorted list, in token order.
//  - The sort is a radix sort with 8 bits a pass over (id, token) pairs.  A
//    pass gives each of at most 64 workgroups a contiguous span; a workgroup
//    counts the digits of its span, and a second launch places the pairs: the
//    position of a pair is the count of smaller digits, plus that of its digit
//    in earlier spans, plus its rank within the span.  Ranks within a wave come
//    from ballots (which lanes hold my digit), so equal ids keep their order.
//    Spans of at most 4096 tokens are sorted in LDS by one workgroup a replica
//    in a single launch.
//  - The sorted list is cut into chunks of 32 pairs.  One wave sums one chunk
//    over 256 columns (4 a lane), adding rows of dy in list order.  A run that
//    lies inside its chunk is finished there; one that crosses a boundary
//    leaves a partial sum in the workspace, and a second launch adds the
//    partials of each such run in chunk order.  A token that fills the whole
//    batch is thus summed by all waves, and the order depends on nothing but
//    the list.
//  - When the gradient overwrites the accumulators, rows without a token have
//    to become zero: further waves of the same launch find them by a binary
//    search in the sorted ids and write each element of the table once.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "dp_device.h"
#include "dp_layers.h"

namespace dpk {
namespace {

constexpr int kLookupSpan = 2048;  // elements of a row per lookup workgroup

__device__ __forceinline__ int64_t load_id(const void* ids, int id_bytes, int64_t i) {
    return id_bytes == 8 ? gload<int64_t>(ids, i) : static_cast<int64_t>(gload<int32_t>(ids, i));
}

template <dp_dtype PT, dp_dtype OT>
__global__ void __launch_bounds__(64) k_embed(const void* table, int64_t rows, int64_t dim, float scale,
                                              const void* ids, int id_bytes, void* out, int64_t ld, bool vec) {
    const int64_t t = blockIdx.x;
    const int64_t id = load_id(ids, id_bytes, t);
    const bool ok = id >= 0 && id < rows;
    const int64_t src = ok ? id * dim : 0;
    const int64_t c0 = static_cast<int64_t>(blockIdx.y) * kLookupSpan + threadIdx.x * 8;
    float v[4][8];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const int64_t c = c0 + k * 512;
        const int64_t left = dim - c;
        const int valid = left >= 8 ? 8 : left > 0 ? static_cast<int>(left) : 0;
        load_n<PT, 8>(table, src + c, valid, vec, v[k]);
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const int64_t c = c0 + k * 512;
        const int64_t left = dim - c;
        const int valid = left >= 8 ? 8 : left > 0 ? static_cast<int>(left) : 0;
#pragma unroll
        for (int j = 0; j < 8; ++j) v[k][j] = ok ? v[k][j] * scale : 0.0f;
        store_n<OT, 8>(out, t * ld + c, valid, vec, v[k]);
    }
}

// ---- the sort ----------------------------------------------------------------
constexpr int kSortThreads = 256;
constexpr int kSortItems = 16;
constexpr int kTile = kSortThreads * kSortItems;  // pairs one workgroup ranks at a time
constexpr int kMaxSpans = 64;
constexpr int kDigits = 256;

// The list of one replica during the sort, and the digit counts of its spans.
struct SortBuf {
    uint32_t* key[2];
    uint32_t* pos[2];
    uint32_t* counts;  // [n][kMaxSpans][kDigits]
};

struct Ids {
    const void* p[DP_MAX_REPLICAS];
    int32_t id_bytes;
};

// The sort key of token t: its id, or `rows` for an id outside the table (they
// sort behind every row and belong to none).
__device__ __forceinline__ uint32_t key_of(const void* ids, int id_bytes, int64_t t, int64_t rows) {
    const int64_t id = load_id(ids, id_bytes, t);
    return static_cast<uint32_t>(id >= 0 && id < rows ? id : rows);
}

__device__ __forceinline__ int lane_id() { return threadIdx.x & 63; }

// How many lanes below this one hold the same 8-bit digit, and whether this is
// the last that does (`mask`: the lanes that hold one at all).
__device__ __forceinline__ uint64_t same_digit(uint32_t d, uint64_t mask) {
#pragma unroll
    for (int b = 0; b < 8; ++b) {
        const bool set = (d >> b) & 1;
        const uint64_t m = __ballot(set);
        mask &= set ? m : ~m;
    }
    return mask;
}

// Ranks the pairs of one tile by a digit: item k of lane l of wave w is pair
// (w * kSortItems + k) * 64 + l of the tile, so that waves hold consecutive
// pairs.  `wave_count` [4][256] is cleared by the caller; afterwards it holds the
// digits' counts of each wave, and rank[k] the number of earlier pairs of the
// same wave with the same digit.
__device__ __forceinline__ void rank_tile(const uint32_t (&key)[kSortItems], int shift, int valid,
                                          volatile uint32_t (*wave_count)[kDigits],
                                          uint32_t (&rank)[kSortItems]) {
    const int w = threadIdx.x >> 6, l = lane_id();
#pragma unroll
    for (int k = 0; k < kSortItems; ++k) {
        const bool in = (w * kSortItems + k) * 64 + l < valid;
        const uint32_t d = (key[k] >> shift) & (kDigits - 1);
        const uint64_t peers = same_digit(d, __ballot(in));
        if (in) {
            const int before = __popcll(peers & ((uint64_t{1} << l) - 1));
            rank[k] = wave_count[w][d] + before;
            // the last of the peers moves the count on (the wave's lanes have
            // all read it: they run in step and LDS accesses keep their order)
            __builtin_amdgcn_wave_barrier();
            if ((peers >> l) == 1) wave_count[w][d] = rank[k] + 1;
        }
        __builtin_amdgcn_wave_barrier();
    }
}

// Exclusive sums over 256 values, one per thread of the workgroup.
__device__ __forceinline__ uint32_t exclusive_scan(uint32_t x, uint32_t* wave_sum) {
    const int l = lane_id(), w = threadIdx.x >> 6;
    uint32_t s = x;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const uint32_t up = __shfl_up(s, d);
        if (l >= d) s += up;
    }
    if (l == 63) wave_sum[w] = s;
    __syncthreads();
    uint32_t base = 0;
#pragma unroll
    for (int k = 0; k < kSortThreads / 64; ++k) base += k < w ? wave_sum[k] : 0;
    __syncthreads();
    return base + s - x;
}

// The whole sort of a list of at most kTile pairs, in LDS: one workgroup a replica.
__global__ void __launch_bounds__(kSortThreads) k_sort_small(Ids ids, SortBuf sb, int64_t rows, int64_t tokens,
                                                             int passes) {
    __shared__ uint32_t lk[kTile], lp[kTile];
    __shared__ uint32_t wave_count[kSortThreads / 64][kDigits];
    __shared__ uint32_t wave_sum[kSortThreads / 64];
    const int r = blockIdx.x, w = threadIdx.x >> 6, l = lane_id();
    const int valid = static_cast<int>(tokens);
    uint32_t key[kSortItems], pos[kSortItems], rank[kSortItems];
#pragma unroll
    for (int k = 0; k < kSortItems; ++k) {
        const int i = (w * kSortItems + k) * 64 + l;
        pos[k] = i;
        key[k] = i < valid ? key_of(ids.p[r], ids.id_bytes, i, rows) : 0;
    }
    for (int p = 0; p < passes; ++p) {
        for (int i = threadIdx.x; i < kDigits * (kSortThreads / 64); i += kSortThreads) (&wave_count[0][0])[i] = 0;
        __syncthreads();
        rank_tile(key, 8 * p, valid, wave_count, rank);
        __syncthreads();
        uint32_t total = 0;
#pragma unroll
        for (int k = 0; k < kSortThreads / 64; ++k) total += wave_count[k][threadIdx.x];
        uint32_t base = exclusive_scan(total, wave_sum);
#pragma unroll
        for (int k = 0; k < kSortThreads / 64; ++k) {
            const uint32_t c = wave_count[k][threadIdx.x];
            wave_count[k][threadIdx.x] = base;
            base += c;
        }
        __syncthreads();
#pragma unroll
        for (int k = 0; k < kSortItems; ++k) {
            const int i = (w * kSortItems + k) * 64 + l;
            if (i < valid) {
                const uint32_t at = wave_count[w][(key[k] >> (8 * p)) & (kDigits - 1)] + rank[k];
                lk[at] = key[k];
                lp[at] = pos[k];
            }
        }
        __syncthreads();
#pragma unroll
        for (int k = 0; k < kSortItems; ++k) {
            const int i = (w * kSortItems + k) * 64 + l;
            if (i < valid) {
                key[k] = lk[i];
                pos[k] = lp[i];
            }
        }
        __syncthreads();
    }
#pragma unroll
    for (int k = 0; k < kSortItems; ++k) {
        const int i = (w * kSortItems + k) * 64 + l;
        if (i < valid) {
            sb.key[0][r * tokens + i] = key[k];
            sb.pos[0][r * tokens + i] = pos[k];
        }
    }
}

// Digit counts of each span of each replica (grid: spans x replicas).
__global__ void __launch_bounds__(kSortThreads) k_sort_count(Ids ids, SortBuf sb, int from, bool first, int64_t rows,
                                                             int64_t tokens, int64_t span, int shift) {
    __shared__ uint32_t c[kDigits];
    const int r = blockIdx.y;
    c[threadIdx.x] = 0;
    __syncthreads();
    const int64_t lo = blockIdx.x * span, hi = lo + span < tokens ? lo + span : tokens;
    for (int64_t i = lo + threadIdx.x; i < hi; i += kSortThreads) {
        const uint32_t k = first ? key_of(ids.p[r], ids.id_bytes, i, rows) : sb.key[from][r * tokens + i];
        atomicAdd(&c[(k >> shift) & (kDigits - 1)], 1u);
    }
    __syncthreads();
    sb.counts[(r * kMaxSpans + blockIdx.x) * kDigits + threadIdx.x] = c[threadIdx.x];
}

// Places the pairs of each span by a digit.
__global__ void __launch_bounds__(kSortThreads) k_sort_place(Ids ids, SortBuf sb, int from, bool first, int64_t rows,
                                                             int64_t tokens, int64_t span, int spans, int shift) {
    __shared__ uint32_t wave_count[kSortThreads / 64][kDigits];
    __shared__ uint32_t next[kDigits];  // where the span's next pair of each digit goes
    __shared__ uint32_t wave_sum[kSortThreads / 64];
    const int r = blockIdx.y, w = threadIdx.x >> 6, l = lane_id();
    {
        uint32_t total = 0, before = 0;
        const uint32_t* c = sb.counts + static_cast<int64_t>(r) * kMaxSpans * kDigits + threadIdx.x;
        for (int s = 0; s < spans; ++s) {
            const uint32_t x = c[s * kDigits];
            before += s < static_cast<int>(blockIdx.x) ? x : 0;
            total += x;
        }
        next[threadIdx.x] = exclusive_scan(total, wave_sum) + before;
    }
    const int64_t lo = blockIdx.x * span, hi = lo + span < tokens ? lo + span : tokens;
    for (int64_t t0 = lo; t0 < hi; t0 += kTile) {
        const int valid = static_cast<int>(hi - t0 < kTile ? hi - t0 : kTile);
        uint32_t key[kSortItems], pos[kSortItems], rank[kSortItems];
#pragma unroll
        for (int k = 0; k < kSortItems; ++k) {
            const int i = (w * kSortItems + k) * 64 + l;
            key[k] = pos[k] = 0;
            if (i < valid) {
                key[k] = first ? key_of(ids.p[r], ids.id_bytes, t0 + i, rows) : sb.key[from][r * tokens + t0 + i];
                pos[k] = first ? static_cast<uint32_t>(t0 + i) : sb.pos[from][r * tokens + t0 + i];
            }
        }
        for (int i = threadIdx.x; i < kDigits * (kSortThreads / 64); i += kSortThreads) (&wave_count[0][0])[i] = 0;
        __syncthreads();
        rank_tile(key, shift, valid, wave_count, rank);
        __syncthreads();
        uint32_t base = next[threadIdx.x];
#pragma unroll
        for (int k = 0; k < kSortThreads / 64; ++k) {
            const uint32_t c = wave_count[k][threadIdx.x];
            wave_count[k][threadIdx.x] = base;
            base += c;
        }
        next[threadIdx.x] = base;
        __syncthreads();
#pragma unroll
        for (int k = 0; k < kSortItems; ++k) {
            const int i = (w * kSortItems + k) * 64 + l;
            if (i < valid) {
                const int64_t at = r * tokens + wave_count[w][(key[k] >> shift) & (kDigits - 1)] + rank[k];
                sb.key[from ^ 1][at] = key[k];
                sb.pos[from ^ 1][at] = pos[k];
            }
        }
        __syncthreads();
    }
}

// ---- the sums ----------------------------------------------------------------
constexpr int kChunk = 32;      // pairs of the sorted list per wave
constexpr int kColumns = 256;   // columns per wave, 4 a lane
constexpr int kBatch = 8;       // rows of dy in flight per wave

struct GradArgs {
    const void* dy[DP_MAX_REPLICAS];
    float* acc[DP_MAX_REPLICAS];
    const uint32_t* key;  // [n][tokens], sorted
    const uint32_t* pos;
    float* part;          // [n][chunks][2][dim]: a chunk's first and last run where they cross its ends
    int64_t rows, dim, tokens, ld;
    int64_t chunks, slices, zero_rows;
    float scale;
    bool vec_dy, vec_acc;
};

// ACC of 4 columns (+)= scale * s.
template <bool kOver>
__device__ __forceinline__ void put(const GradArgs& a, float* acc, int64_t row, int64_t c, int valid, const float* s) {
    float v[4];
    const int64_t at = row * a.dim + c;
    if constexpr (!kOver) load_n<DP_F32, 4>(acc, at, valid, a.vec_acc, v);
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] = kOver ? a.scale * s[j] : v[j] + a.scale * s[j];
    store_n<DP_F32, 4>(acc, at, valid, a.vec_acc, v);
}

// Zeros in the rows [row0, row0 + zero_rows) that no token holds.
__device__ __forceinline__ void zero_rows(const GradArgs& a, float* acc, const uint32_t* key, int64_t row0) {
    const int l = lane_id();
    const int64_t mine = row0 + l;
    bool absent = false;
    if (l < a.zero_rows && mine < a.rows) {
        int64_t lo = 0, hi = a.tokens;  // first pair whose id is not below mine
        while (lo < hi) {
            const int64_t mid = (lo + hi) >> 1;
            if (key[mid] < mine) lo = mid + 1;
            else hi = mid;
        }
        absent = lo == a.tokens || key[lo] != mine;
    }
    uint64_t todo = __ballot(absent);
    const float zero[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    while (todo) {
        const int64_t row = row0 + __builtin_ctzll(todo);
        todo &= todo - 1;
        for (int64_t c = 4 * l; c < a.dim; c += kColumns)
            store_n<DP_F32, 4>(acc, row * a.dim + c, static_cast<int>(a.dim - c < 4 ? a.dim - c : 4), a.vec_acc, zero);
    }
}

// Grid: (chunks * slices + waves of zero_rows rows) x replicas, one wave each.
template <dp_dtype DT, bool kOver>
__global__ void __launch_bounds__(64) k_embed_sum(GradArgs a) {
    const int r = blockIdx.y, l = lane_id();
    const uint32_t* key = a.key + r * a.tokens;
    const uint32_t* pos = a.pos + r * a.tokens;
    float* acc = a.acc[r];
    const int64_t sums = a.chunks * a.slices;
    if (static_cast<int64_t>(blockIdx.x) >= sums) {
        if constexpr (kOver) zero_rows(a, acc, key, (blockIdx.x - sums) * a.zero_rows);
        return;
    }
    const int64_t chunk = blockIdx.x / a.slices, c = (blockIdx.x % a.slices) * kColumns + 4 * l;
    const int64_t left = a.dim - c;
    const int valid = left >= 4 ? 4 : left > 0 ? static_cast<int>(left) : 0;
    const int64_t i0 = chunk * kChunk;
    const int count = static_cast<int>(a.tokens - i0 < kChunk ? a.tokens - i0 : kChunk);
    // lane i < count: pair i; lane 62: the id before the chunk, lane 63: the one behind it
    const uint32_t none = 0xffffffffu;
    uint32_t k = none, p = 0;
    if (l < count) {
        k = key[i0 + l];
        p = pos[i0 + l];
    } else if (l == 62 && i0 > 0) {
        k = key[i0 - 1];
    } else if (l == 63 && i0 + count < a.tokens) {
        k = key[i0 + count];
    }
    const uint32_t before = __builtin_amdgcn_readlane(k, 62), behind = __builtin_amdgcn_readlane(k, 63);
    float* part = a.part + (r * a.chunks + chunk) * 2 * a.dim;
    const bool vec_part = a.dim % 4 == 0;
    float s[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    uint32_t run = __builtin_amdgcn_readlane(k, 0);
    bool head = run == before;  // the current run began in an earlier chunk
    for (int b = 0; b < count; b += kBatch) {
        float v[kBatch][4];
        uint32_t kk[kBatch];
#pragma unroll
        for (int j = 0; j < kBatch; ++j) {
            const int i = b + j < count ? b + j : count - 1;
            kk[j] = __builtin_amdgcn_readlane(k, i);
            const int64_t row = __builtin_amdgcn_readlane(p, i);
            // a batch past the chunk's end, or an id outside the table, reads no row
            const bool read = b + j < count && kk[j] < a.rows;
            load_n<DT, 4>(a.dy[r], row * a.ld + c, read ? valid : 0, a.vec_dy, v[j]);
        }
#pragma unroll
        for (int j = 0; j < kBatch; ++j) {
            if (b + j >= count) break;
            if (kk[j] != run) {
                if (run < a.rows) {
                    if (head) store_n<DP_F32, 4>(part, c, valid, vec_part, s);
                    else put<kOver>(a, acc, run, c, valid, s);
                }
                head = false;
                run = kk[j];
#pragma unroll
                for (int q = 0; q < 4; ++q) s[q] = 0.0f;
            }
#pragma unroll
            for (int q = 0; q < 4; ++q) s[q] += v[j][q];
        }
    }
    if (run < a.rows) {
        if (head) store_n<DP_F32, 4>(part, c, valid, vec_part, s);
        else if (run == behind) store_n<DP_F32, 4>(part + a.dim, c, valid, vec_part, s);
        else put<kOver>(a, acc, run, c, valid, s);
    }
}

// Finishes the runs that cross a chunk's end: the wave of the chunk where such
// a run begins adds its partials in chunk order (grid as the sums of k_embed_sum).
template <bool kOver>
__global__ void __launch_bounds__(64) k_embed_join(GradArgs a) {
    const int r = blockIdx.y, l = lane_id();
    const uint32_t* key = a.key + r * a.tokens;
    const int64_t chunk = blockIdx.x / a.slices, c = (blockIdx.x % a.slices) * kColumns + 4 * l;
    const int64_t i0 = chunk * kChunk, i1 = i0 + kChunk;
    if (i1 >= a.tokens) return;
    const uint32_t run = key[i1 - 1];
    if (run != key[i1] || run >= a.rows) return;
    if (i0 > 0 && key[i0 - 1] == run) return;  // began earlier
    // the run goes on through the chunks whose first id is its own: count them, 64 at a time
    int64_t n = 0;
    for (;;) {
        const int64_t i = (chunk + 1 + n + l) * kChunk;
        const uint64_t on = __ballot(i < a.tokens && key[i] == run);
        n += ~on == 0 ? 64 : __builtin_ctzll(~on);
        if (~on != 0) break;
    }
    const int64_t left = a.dim - c;
    const int valid = left >= 4 ? 4 : left > 0 ? static_cast<int>(left) : 0;
    const bool vec_part = a.dim % 4 == 0;
    const float* part = a.part + (r * a.chunks + chunk) * 2 * a.dim;
    float s[4];
    load_n<DP_F32, 4>(part + a.dim, c, valid, vec_part, s);
    for (int64_t b = 0; b < n; b += kBatch) {
        float v[kBatch][4];
#pragma unroll
        for (int j = 0; j < kBatch; ++j)
            load_n<DP_F32, 4>(part + (b + j + 1) * 2 * a.dim, c, b + j < n ? valid : 0, vec_part, v[j]);
#pragma unroll
        for (int j = 0; j < kBatch; ++j)
#pragma unroll
            for (int q = 0; q < 4; ++q) s[q] += v[j][q];
    }
    put<kOver>(a, a.acc[r], run, c, valid, s);
}

int64_t round256(int64_t x) { return (x + 255) & ~int64_t{255}; }
int64_t chunks_of(int64_t tokens) { return (tokens + kChunk - 1) / kChunk; }

int64_t slices_of(int64_t dim) { return (dim + kColumns - 1) / kColumns; }

// Rows of zeros per wave: about 64 KiB to write, a power of two of at most 64 rows.
int64_t zero_rows_per_wave(int64_t dim) {
    int64_t z = 64;
    while (z > 1 && z * dim > 16384) z >>= 1;
    return z;
}

int passes_of(int64_t rows) {
    int p = 1;
    while (p < 4 && (rows >> (8 * p)) != 0) ++p;  // the keys are 0 .. rows
    return p;
}

}  // namespace

hipError_t launch_embed(dp_dtype pdt, dp_dtype odt, const void* table, int64_t rows, int64_t dim, float scale,
                        int64_t tokens, const void* ids, int id_bytes, void* out, int64_t ld, bool vec,
                        hipStream_t stream) {
    if (tokens == 0) return hipSuccess;
    const dim3 grid(static_cast<unsigned>(tokens), static_cast<unsigned>((dim + kLookupSpan - 1) / kLookupSpan));
#define DP_GO(P, O)                                                                                              \
    if (pdt == P && odt == O)                                                                                    \
    hipLaunchKernelGGL((k_embed<P, O>), grid, dim3(64), 0, stream, table, rows, dim, scale, ids, id_bytes, out, ld, vec)
    DP_GO(DP_BF16, DP_BF16);
    DP_GO(DP_BF16, DP_F16);
    DP_GO(DP_BF16, DP_F32);
    DP_GO(DP_F16, DP_BF16);
    DP_GO(DP_F16, DP_F16);
    DP_GO(DP_F16, DP_F32);
#undef DP_GO
    return hipGetLastError();
}

size_t embed_workspace(int64_t dim, int64_t tokens, int n) {
    return static_cast<size_t>(4 * round256(4 * n * tokens) + round256(4 * int64_t{n} * kMaxSpans * kDigits) +
                               round256(8 * n * chunks_of(tokens) * dim));
}

int64_t embed_waves(const EmbedGrad& a) {
    const int64_t z = zero_rows_per_wave(a.dim);
    return chunks_of(a.tokens) * slices_of(a.dim) + (a.overwrite ? (a.rows + z - 1) / z : 0);
}

hipError_t launch_embed_grad(dp_dtype dt, const EmbedGrad& a, void* workspace, hipStream_t stream) {
    Ids ids{};
    GradArgs g{};
    SortBuf sb{};
    char* at = static_cast<char*>(workspace);
    for (int i = 0; i < 2; ++i) {
        sb.key[i] = reinterpret_cast<uint32_t*>(at);
        at += round256(4 * a.n * a.tokens);
        sb.pos[i] = reinterpret_cast<uint32_t*>(at);
        at += round256(4 * a.n * a.tokens);
    }
    sb.counts = reinterpret_cast<uint32_t*>(at);
    at += round256(4 * int64_t{a.n} * kMaxSpans * kDigits);
    g.part = reinterpret_cast<float*>(at);
    ids.id_bytes = a.id_bytes;
    for (int r = 0; r < a.n; ++r) {
        ids.p[r] = a.ids[r];
        g.dy[r] = a.dy[r];
        g.acc[r] = a.acc[r];
    }
    const int passes = passes_of(a.rows);
    int from = 0;
    if (a.tokens > 0 && a.tokens <= kTile) {
        hipLaunchKernelGGL(k_sort_small, dim3(a.n), dim3(kSortThreads), 0, stream, ids, sb, a.rows, a.tokens, passes);
    } else if (a.tokens > 0) {
        const int64_t tiles = (a.tokens + kTile - 1) / kTile;
        const int64_t span = (tiles + kMaxSpans - 1) / kMaxSpans * kTile;
        const int spans = static_cast<int>((a.tokens + span - 1) / span);
        for (int p = 0; p < passes; ++p) {
            hipLaunchKernelGGL(k_sort_count, dim3(spans, a.n), dim3(kSortThreads), 0, stream, ids, sb, from, p == 0,
                               a.rows, a.tokens, span, 8 * p);
            hipLaunchKernelGGL(k_sort_place, dim3(spans, a.n), dim3(kSortThreads), 0, stream, ids, sb, from, p == 0,
                               a.rows, a.tokens, span, spans, 8 * p);
            from ^= 1;
        }
    }
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    g.key = sb.key[from];
    g.pos = sb.pos[from];
    g.rows = a.rows;
    g.dim = a.dim;
    g.tokens = a.tokens;
    g.ld = a.ld;
    g.chunks = chunks_of(a.tokens);
    g.slices = slices_of(a.dim);
    g.scale = a.scale;
    g.vec_dy = a.vec_dy;
    g.vec_acc = a.vec_acc;
    g.zero_rows = zero_rows_per_wave(a.dim);
    const int64_t sums = g.chunks * g.slices, waves = embed_waves(a);
    if (waves == 0) return hipSuccess;
    const dim3 grid(static_cast<unsigned>(waves), static_cast<unsigned>(a.n));
#define DP_GO(D)                                                                                   \
    if (dt == D) {                                                                                 \
        if (a.overwrite) hipLaunchKernelGGL((k_embed_sum<D, true>), grid, dim3(64), 0, stream, g); \
        else hipLaunchKernelGGL((k_embed_sum<D, false>), grid, dim3(64), 0, stream, g);            \
    }
    DP_GO(DP_F32)
    DP_GO(DP_F16)
    DP_GO(DP_BF16)
#undef DP_GO
    e = hipGetLastError();
    if (e != hipSuccess || g.chunks < 2) return e;
    const dim3 jgrid(static_cast<unsigned>(sums), static_cast<unsigned>(a.n));
    if (a.overwrite) hipLaunchKernelGGL((k_embed_join<true>), jgrid, dim3(64), 0, stream, g);
    else hipLaunchKernelGGL((k_embed_join<false>), jgrid, dim3(64), 0, stream, g);
    return hipGetLastError();
}

}  // namespace dpk

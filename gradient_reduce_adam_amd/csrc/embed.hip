// gfx950 kernels of the embedding: the scaled lookup, and its gradient by
// sorted tokens.
//
// Lookup.  out[t] = scale * W[id_t]: a gather of rows, bound by HBM (the rows
// touched, once, and the output).  One wave64 workgroup moves up to 2048
// elements of one row, 8 per lane and access.  32768 rows of 4096 bf16 take 58
// us.
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
//    Lists of at most 16384 tokens are sorted in LDS by one workgroup a replica
//    in a single launch.
//  - The sorted list is cut into chunks of 64 pairs, 16 for each wave of a
//    workgroup.  A wave sums its pairs over 256 columns (4 a lane), adding rows of
//    dy in list order.  A run inside its 16 pairs is finished there; parts of
//    longer ones are added through LDS in order; and one that crosses a
//    chunk's end leaves a partial sum in the workspace, and a second launch
//    adds the partials of each such run in chunk order.  A token that fills the
//    whole batch is thus summed by all waves, and the order depends on nothing
//    but the list.
//  - When the gradient overwrites the accumulators, rows without a token have
//    to become zero: further workgroups of the sort's first launch clear the
//    tables meanwhile, so that the sort, which few CUs work on, costs nothing
//    beside them.
// 8 replicas of 4096 tokens and 50257 x 768 tables: cleared and sorted in 203 us
// (6.1 TB/s), summed in 22 us; a further micro-step sorts in 12 us and adds in 35.
// With 32 pairs a wave instead of 16 the 7B layout's table takes 4% more, with 16
// rows in flight instead of 8 both take 8% more (fewer waves fit).
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

template <dp_dtype PT, dp_dtype OT, bool kOnce>
__global__ void __launch_bounds__(64) k_embed(const void* table, int64_t rows, int64_t dim, float scale,
                                              const void* ids, int id_bytes, void* out, int64_t ld) {
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
        load_n<PT, 8>(table, src + c, valid, v[k]);
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const int64_t c = c0 + k * 512;
        const int64_t left = dim - c;
        const int valid = left >= 8 ? 8 : left > 0 ? static_cast<int>(left) : 0;
#pragma unroll
        for (int j = 0; j < 8; ++j) v[k][j] = ok ? v[k][j] * scale : 0.0f;
        store_n<OT, 8, kOnce>(out, t * ld + c, valid, v[k]);
    }
}

// ---- the sort ----------------------------------------------------------------
constexpr int kSortThreads = 1024;
constexpr int kSortWaves = kSortThreads / 64;
constexpr int kTileItems = 4;                     // pairs per thread that the launches over spans rank at a time
constexpr int kTile = kSortThreads * kTileItems;
constexpr int kMaxSpans = 64;
constexpr int kDigits = 256;
constexpr int kSmallSort = 16 * kSortThreads;     // longest list sorted by one workgroup

// The list of one replica during the sort, and the digit counts of its spans.
struct SortBuf {
    uint32_t* key[2];
    uint32_t* pos[2];
    uint32_t* counts;  // [n][kMaxSpans][kDigits]
};

struct Ids {
    const void* p[DP_MAX_REPLICAS];
    int32_t id_bytes, n;
};

// The sort key of token t: its id, or `rows` for an id outside the table (they
// sort behind every row and belong to none).
__device__ __forceinline__ uint32_t key_of(const void* ids, int id_bytes, int64_t t, int64_t rows) {
    const int64_t id = load_id(ids, id_bytes, t);
    return static_cast<uint32_t>(id >= 0 && id < rows ? id : rows);
}

__device__ __forceinline__ int lane_id() { return threadIdx.x & 63; }

// Of the lanes in `mask`, those that hold the same 8-bit digit as this one: a
// lane stays where its bit equals mine, mask & ~(lanes with the bit set ^ my bit).
__device__ __forceinline__ uint64_t same_digit(uint32_t d, uint64_t mask) {
    uint32_t lo = static_cast<uint32_t>(mask), hi = static_cast<uint32_t>(mask >> 32);
#pragma unroll
    for (int b = 0; b < 8; ++b) {
        const uint32_t mine = static_cast<uint32_t>(static_cast<int32_t>(d << (31 - b)) >> 31);
        const uint64_t m = __ballot(mine != 0);
        lo &= ~(static_cast<uint32_t>(m) ^ mine);
        hi &= ~(static_cast<uint32_t>(m >> 32) ^ mine);
    }
    return static_cast<uint64_t>(hi) << 32 | lo;
}

// The tables of every replica set to zero by further workgroups of the sort's
// first launch: `elements` floats each, `groups` workgroups a table of `span`
// floats each.  Tables that together fit the 256 MB of the last-level cache
// are cleared with ordinary stores, 64 KiB a workgroup: one of 154 MB, cleared
// again every step, takes 33 us with the sums of 4096 tokens, and 38 with
// streaming stores.  Beyond it (`once`) streaming stores, 32 KiB in a row by each
// wave, leave the caches to the sums: 100 us instead of 110 for 524 MB, and for
// 8 x 154 MB the sums behind the clearing take 22 us instead of 34.
struct Zeros {
    float* acc[DP_MAX_REPLICAS];
    int64_t elements, groups, span;
    int32_t n;
    bool once;
};
constexpr int kZeroQuads = 4, kZeroQuadsOnce = 32;  // 16-byte stores per thread
constexpr int64_t kZeroSpan = int64_t{4} * kZeroQuads * kSortThreads;
constexpr int64_t kZeroSpanOnce = int64_t{4} * kZeroQuadsOnce * kSortThreads;
constexpr int64_t kLastLevel = int64_t{256} << 20;

__device__ __forceinline__ void zero_table(const Zeros& z, int64_t group) {
    const f32x4 zero{0.0f, 0.0f, 0.0f, 0.0f};
    const int64_t i0 = group % z.groups * z.span;
    const int left = static_cast<int>(z.elements - i0 < z.span ? z.elements - i0 : z.span), tid = threadIdx.x;
    float* p = z.acc[group / z.groups] + i0;
    if (z.once && left == kZeroSpanOnce) {
#pragma unroll
        for (int k = 0; k < kZeroQuadsOnce; ++k)
            gstore_nt<f32x4, 4>(p, ((tid >> 6) * kZeroQuadsOnce + k) * 64 + (tid & 63), zero);
    } else if (left == kZeroSpan) {
#pragma unroll
        for (int k = 0; k < kZeroQuads; ++k) gstore<f32x4, 4>(p, k * kSortThreads + tid, zero);
    } else {
        for (int q = tid; q < left / 4; q += kSortThreads) gstore<f32x4, 4>(p, q, zero);
        if (tid < left % 4) gstore<float>(p, left / 4 * 4 + tid, 0.0f);
    }
}

// Counts of a tile's digits by wave, and scratch of the scan.
struct TileCounts {
    uint32_t wave[kSortWaves][kDigits];
    uint32_t sum[kDigits / 64];
};

// Where the pairs of one tile go by a digit.  Item k of lane l of wave w is pair
// (w * kItems + k) * 64 + l of the tile, so that waves hold consecutive pairs; the
// first `valid` exist.  A pair goes to first(its digit) + the pairs before it
// in the tile with the same digit: rank[k] is its rank within the wave, and
// c.wave holds, afterwards, the place of each wave's first pair of each digit.
// `place` (of the 256 threads of the first waves, one a digit) maps the
// tile's count of the digit to the place of its first pair.
template <int kItems, typename F>
__device__ __forceinline__ void rank_tile(const uint32_t (&key)[kItems], int shift, int valid, TileCounts& c,
                                          uint32_t (&rank)[kItems], F&& place) {
    const int w = threadIdx.x >> 6, l = lane_id();
    for (int i = threadIdx.x; i < kSortWaves * kDigits; i += kSortThreads) (&c.wave[0][0])[i] = 0;
    __syncthreads();
    volatile uint32_t* count = c.wave[w];
#pragma unroll
    for (int k = 0; k < kItems; ++k) {
        const bool in = (w * kItems + k) * 64 + l < valid;
        const uint32_t d = (key[k] >> shift) & (kDigits - 1);
        const uint64_t peers = same_digit(d, __ballot(in));
        if (in) {
            rank[k] = count[d] + __popcll(peers & ((uint64_t{1} << l) - 1));
            // the last of the peers moves the count on; all of them have read
            // it (a wave's LDS accesses keep their order)
            __builtin_amdgcn_wave_barrier();
            if ((peers >> l) == 1) count[d] = rank[k] + 1;
        }
        __builtin_amdgcn_wave_barrier();
    }
    __syncthreads();
    uint32_t total = 0;
    if (threadIdx.x < kDigits)
#pragma unroll
        for (int k = 0; k < kSortWaves; ++k) total += c.wave[k][threadIdx.x];
    uint32_t base = place(total);
    if (threadIdx.x < kDigits)
#pragma unroll
        for (int k = 0; k < kSortWaves; ++k) {
            const uint32_t n = c.wave[k][threadIdx.x];
            c.wave[k][threadIdx.x] = base;
            base += n;
        }
    __syncthreads();
}

// Exclusive sums over 256 values, one in each of the first 256 threads.
__device__ __forceinline__ uint32_t exclusive_scan(uint32_t x, uint32_t* wave_sum) {
    const int l = lane_id(), w = threadIdx.x >> 6;
    uint32_t s = x;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const uint32_t up = __shfl_up(s, d);
        if (l >= d) s += up;
    }
    if (l == 63 && threadIdx.x < kDigits) wave_sum[w] = s;
    __syncthreads();
    uint32_t base = 0;
#pragma unroll
    for (int k = 0; k < kDigits / 64; ++k) base += k < w ? wave_sum[k] : 0;
    __syncthreads();
    return base + s - x;
}

// The whole sort of a list of at most kItems * 1024 pairs, in LDS: one
// workgroup a replica, and those behind them for the zeros.
template <int kItems>
__global__ void __launch_bounds__(kSortThreads) k_sort_small(Ids ids, SortBuf sb, Zeros z, int64_t rows,
                                                             int64_t tokens, int passes) {
    __shared__ uint32_t lk[kItems * kSortThreads], lp[kItems * kSortThreads];
    __shared__ TileCounts c;
    if (static_cast<int>(blockIdx.x) >= ids.n) {
        zero_table(z, blockIdx.x - ids.n);
        return;
    }
    const int r = blockIdx.x, w = threadIdx.x >> 6, l = lane_id();
    const int valid = static_cast<int>(tokens);
    uint32_t key[kItems], pos[kItems], rank[kItems];
#pragma unroll
    for (int k = 0; k < kItems; ++k) {
        const int i = (w * kItems + k) * 64 + l;
        pos[k] = i;
        key[k] = i < valid ? key_of(ids.p[r], ids.id_bytes, i, rows) : 0;
    }
    for (int p = 0;; ++p) {
        rank_tile<kItems>(key, 8 * p, valid, c, rank, [&](uint32_t total) { return exclusive_scan(total, c.sum); });
        const bool last = p + 1 == passes;
#pragma unroll
        for (int k = 0; k < kItems; ++k) {
            if ((w * kItems + k) * 64 + l >= valid) continue;
            const uint32_t at = c.wave[w][(key[k] >> (8 * p)) & (kDigits - 1)] + rank[k];
            if (last) {
                sb.key[0][r * tokens + at] = key[k];
                sb.pos[0][r * tokens + at] = pos[k];
            } else {
                lk[at] = key[k];
                lp[at] = pos[k];
            }
        }
        if (last) break;
        __syncthreads();
#pragma unroll
        for (int k = 0; k < kItems; ++k) {
            const int i = (w * kItems + k) * 64 + l;
            if (i < valid) {
                key[k] = lk[i];
                pos[k] = lp[i];
            }
        }
    }
}

// Digit counts of each span of each replica (grid: spans x replicas), and
// workgroups behind those of the last replica for the zeros.
__global__ void __launch_bounds__(kSortThreads) k_sort_count(Ids ids, SortBuf sb, Zeros z, int from, bool first,
                                                             int64_t rows, int64_t tokens, int64_t span, int spans,
                                                             int shift) {
    __shared__ uint32_t c[kDigits];
    if (static_cast<int>(blockIdx.x) >= spans * ids.n) {
        zero_table(z, blockIdx.x - spans * ids.n);
        return;
    }
    const int r = blockIdx.x / spans, block = blockIdx.x % spans;
    if (threadIdx.x < kDigits) c[threadIdx.x] = 0;
    __syncthreads();
    const int64_t lo = block * span, hi = lo + span < tokens ? lo + span : tokens;
    for (int64_t i = lo + threadIdx.x; i < hi; i += kSortThreads) {
        const uint32_t k = first ? key_of(ids.p[r], ids.id_bytes, i, rows) : sb.key[from][r * tokens + i];
        atomicAdd(&c[(k >> shift) & (kDigits - 1)], 1u);
    }
    __syncthreads();
    if (threadIdx.x < kDigits) sb.counts[(r * kMaxSpans + block) * kDigits + threadIdx.x] = c[threadIdx.x];
}

// Places the pairs of each span by a digit.
__global__ void __launch_bounds__(kSortThreads) k_sort_place(Ids ids, SortBuf sb, int from, bool first, int64_t rows,
                                                             int64_t tokens, int64_t span, int spans, int shift) {
    __shared__ TileCounts c;
    const int r = blockIdx.y, w = threadIdx.x >> 6, l = lane_id();
    uint32_t next = 0;  // of a digit: where the span's next pair goes
    {
        uint32_t total = 0, before = 0;
        const uint32_t* n = sb.counts + static_cast<int64_t>(r) * kMaxSpans * kDigits + threadIdx.x;
        if (threadIdx.x < kDigits)
            for (int s = 0; s < spans; ++s) {
                const uint32_t x = n[s * kDigits];
                before += s < static_cast<int>(blockIdx.x) ? x : 0;
                total += x;
            }
        next = exclusive_scan(total, c.sum) + before;
    }
    const int64_t lo = blockIdx.x * span, hi = lo + span < tokens ? lo + span : tokens;
    for (int64_t t0 = lo; t0 < hi; t0 += kTile) {
        const int valid = static_cast<int>(hi - t0 < kTile ? hi - t0 : kTile);
        uint32_t key[kTileItems], pos[kTileItems], rank[kTileItems];
#pragma unroll
        for (int k = 0; k < kTileItems; ++k) {
            const int i = (w * kTileItems + k) * 64 + l;
            key[k] = pos[k] = 0;
            if (i < valid) {
                key[k] = first ? key_of(ids.p[r], ids.id_bytes, t0 + i, rows) : sb.key[from][r * tokens + t0 + i];
                pos[k] = first ? static_cast<uint32_t>(t0 + i) : sb.pos[from][r * tokens + t0 + i];
            }
        }
        rank_tile<kTileItems>(key, shift, valid, c, rank, [&](uint32_t total) {
            const uint32_t at = next;
            next += total;
            return at;
        });
#pragma unroll
        for (int k = 0; k < kTileItems; ++k) {
            if ((w * kTileItems + k) * 64 + l >= valid) continue;
            const int64_t at = r * tokens + c.wave[w][(key[k] >> shift) & (kDigits - 1)] + rank[k];
            sb.key[from ^ 1][at] = key[k];
            sb.pos[from ^ 1][at] = pos[k];
        }
        __syncthreads();
    }
}

// ---- the sums ----------------------------------------------------------------
constexpr int kSpan = 16;            // pairs of the sorted list per wave
constexpr int kSpans = 4;            // waves of a workgroup
constexpr int kChunk = kSpan * kSpans;
constexpr int kColumns = 256;        // columns per wave, 4 a lane
constexpr int kBatch = 8;            // rows in flight per wave

struct GradArgs {
    const void* dy[DP_MAX_REPLICAS];
    float* acc[DP_MAX_REPLICAS];
    const uint32_t* key;  // [n][tokens], sorted
    const uint32_t* pos;
    float* part;          // [n][chunks][2][dim]: a chunk's first and last run where they cross its ends
    int64_t rows, dim, tokens, ld;
    int64_t chunks, slices;
    float scale;
};

// The accumulator of 4 columns of a row, if the gradient is added to it.
template <bool kOver>
__device__ __forceinline__ Raw<DP_F32, 4> fetch(const GradArgs& a, const float* acc, int64_t row, int64_t c, int valid) {
    return load_raw<DP_F32, 4>(acc, row * a.dim + c, kOver ? 0 : valid, a.dim >= 4);
}
// ACC = scale * s, or what was fetched of it + scale * s.
template <bool kOver>
__device__ __forceinline__ void put(const GradArgs& a, float* acc, int64_t row, int64_t c, int valid, f32x4 s,
                                    Raw<DP_F32, 4> old) {
    float v[4];
    settle<DP_F32, 4>(old, valid, a.dim >= 4);
    expand<DP_F32, 4>(old, v);
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] = kOver ? a.scale * s[j] : v[j] + a.scale * s[j];
    store_n<DP_F32, 4>(acc, row * a.dim + c, valid, v);
}

// Grid: (chunks * slices) x replicas.  The four waves of a workgroup take 16 pairs
// each of one chunk, over the same columns.
template <dp_dtype DT, bool kOver>
__global__ void __launch_bounds__(64 * kSpans) k_embed_sum(GradArgs a) {
    __shared__ f32x4 heads[kSpans][64];  // sums of the waves' first runs, where they began in an earlier span
    __shared__ bool through[kSpans];     // such a run fills the span and goes on
    const int r = blockIdx.y, l = lane_id(), w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const uint32_t* key = a.key + r * a.tokens;
    const uint32_t* pos = a.pos + r * a.tokens;
    float* acc = a.acc[r];
    const int64_t chunk = blockIdx.x / a.slices, c = (blockIdx.x % a.slices) * kColumns + 4 * l;
    const int64_t width = a.dim - c;
    const int valid = width >= 4 ? 4 : width > 0 ? static_cast<int>(width) : 0;
    const int64_t i0 = chunk * kChunk + w * kSpan, left = a.tokens - i0;
    const int count = left >= kSpan ? kSpan : left > 0 ? static_cast<int>(left) : 0;
    // lane i < count: pair i; lane 62: the id before the span, lane 63: the one behind it
    const uint32_t none = 0xffffffffu;
    uint32_t k = none, p = 0;
    if (l < count) {
        k = key[i0 + l];
        p = pos[i0 + l];
    } else if (l == 62 && count > 0 && i0 > 0) {
        k = key[i0 - 1];
    } else if (l == 63 && count > 0 && i0 + count < a.tokens) {
        k = key[i0 + count];
    }
    const uint32_t before = __builtin_amdgcn_readlane(k, 62), behind = __builtin_amdgcn_readlane(k, 63);
    // bit i: pair i is the last of its run in this span
    const uint32_t after = __shfl_down(k, 1);
    const uint64_t ends = __ballot(l < count && (l == count - 1 || k != after));
    const uint32_t first = __builtin_amdgcn_readlane(k, 0), last = __builtin_amdgcn_readlane(k, count > 0 ? count - 1 : 0);
    const bool head = count > 0 && first == before && first < a.rows;  // the first run began earlier
    const bool open = count > 0 && last == behind && last < a.rows;    // the last run goes on
    f32x4 s{0.0f, 0.0f, 0.0f, 0.0f};
    bool at_head = head;
    for (int b = 0; b < count; b += kBatch) {
        Raw<DT, 4> v[kBatch];
        Raw<DP_F32, 4> old[kBatch];
        uint32_t kk[kBatch];
#pragma unroll
        for (int j = 0; j < kBatch; ++j) {
            const int i = b + j < count ? b + j : count - 1;
            kk[j] = __builtin_amdgcn_readlane(k, i);
            const int64_t row = __builtin_amdgcn_readlane(p, i);
            // a batch past the span's end, or an id outside the table, reads no row
            const bool read = b + j < count && kk[j] < a.rows;
            v[j] = load_raw<DT, 4>(a.dy[r], row * a.ld + c, read ? valid : 0, a.dim >= 4);
            // runs that lie inside the span are finished here
            const bool whole = (ends >> i & 1) && !(head && kk[j] == first) && !(open && kk[j] == last);
            old[j] = fetch<kOver>(a, acc, kk[j], c, read && whole ? valid : 0);
        }
#pragma unroll
        for (int j = 0; j < kBatch; ++j) {
            if (b + j >= count) break;
            float x[4];
            settle<DT, 4>(v[j], kk[j] < a.rows ? valid : 0, a.dim >= 4);
            expand<DT, 4>(v[j], x);
#pragma unroll
            for (int q = 0; q < 4; ++q) s[q] += x[q];
            if (!(ends >> (b + j) & 1)) continue;
            if (at_head) heads[w][l] = s;
            else if (b + j == count - 1 && open) break;  // s stays: the sum of the open run
            else if (kk[j] < a.rows) put<kOver>(a, acc, kk[j], c, valid, s, old[j]);
            at_head = false;
            s = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
        }
    }
    if (l == 0) through[w] = head && open && first == last;
    __syncthreads();
    // Runs over several spans: the wave where such a run begins adds the
    // following waves' parts in order; so does the first wave with a run that began
    // in an earlier chunk.
    const bool inner = head && w == 0, outer = open && !(head && first == last);
    float* part = a.part + (r * a.chunks + chunk) * 2 * a.dim;
    if (inner) {
        f32x4 t = heads[0][l];
        for (int v = 0; v + 1 < kSpans && through[v]; ++v) t += heads[v + 1][l];
        store_n<DP_F32, 4>(part, c, valid, reinterpret_cast<const float*>(&t));
    }
    if (outer) {
        bool on = true;
        for (int v = w + 1; v < kSpans && on; ++v) {
            s += heads[v][l];
            on = through[v];
        }
        if (on) store_n<DP_F32, 4>(part + a.dim, c, valid, reinterpret_cast<const float*>(&s));
        else put<kOver>(a, acc, last, c, valid, s, fetch<kOver>(a, acc, last, c, valid));
    }
}

// Finishes the runs that cross a chunk's end: the wave of the chunk where such
// a run begins adds its partials in chunk order (one wave per chunk and slice).
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
    const float* part = a.part + (r * a.chunks + chunk) * 2 * a.dim;
    f32x4 s;
    const Raw<DP_F32, 4> old = fetch<kOver>(a, a.acc[r], run, c, valid);
    load_n<DP_F32, 4>(part + a.dim, c, valid, reinterpret_cast<float*>(&s));
    for (int64_t b = 0; b < n; b += kBatch) {
        float v[kBatch][4];
#pragma unroll
        for (int j = 0; j < kBatch; ++j) load_n<DP_F32, 4>(part + (b + j + 1) * 2 * a.dim, c, b + j < n ? valid : 0, v[j]);
#pragma unroll
        for (int j = 0; j < kBatch; ++j)
#pragma unroll
            for (int q = 0; q < 4; ++q) s[q] += v[j][q];
    }
    put<kOver>(a, a.acc[r], run, c, valid, s, old);
}

int64_t round256(int64_t x) { return (x + 255) & ~int64_t{255}; }
int64_t chunks_of(int64_t tokens) { return (tokens + kChunk - 1) / kChunk; }

int64_t slices_of(int64_t dim) { return (dim + kColumns - 1) / kColumns; }

int passes_of(int64_t rows) {
    int p = 1;
    while (p < 4 && (rows >> (8 * p)) != 0) ++p;  // the keys are 0 .. rows
    return p;
}

}  // namespace

hipError_t launch_embed(dp_dtype pdt, dp_dtype odt, const void* table, int64_t rows, int64_t dim, float scale,
                        int64_t tokens, const void* ids, int id_bytes, void* out, int64_t ld, hipStream_t stream) {
    if (tokens == 0) return hipSuccess;
    const dim3 grid(static_cast<unsigned>(tokens), static_cast<unsigned>((dim + kLookupSpan - 1) / kLookupSpan));
    // An output beyond the 32 MiB of all L2 caches cannot wait there for its
    // reader, and stored past them it leaves them to the table's rows: 32768 x
    // 4096 bf16 takes 58 us instead of 81.  A smaller one stays for its reader.
    const bool once = tokens * dim * (odt == DP_F32 ? 4 : 2) > (int64_t{32} << 20);
#define DP_GO2(P, O, S) \
    hipLaunchKernelGGL((k_embed<P, O, S>), grid, dim3(64), 0, stream, table, rows, dim, scale, ids, id_bytes, out, ld)
#define DP_GO(P, O)                    \
    if (pdt == P && odt == O) {        \
        if (once) DP_GO2(P, O, true);  \
        else DP_GO2(P, O, false);      \
    }
    DP_GO(DP_BF16, DP_BF16)
    DP_GO(DP_BF16, DP_F16)
    DP_GO(DP_BF16, DP_F32)
    DP_GO(DP_F16, DP_BF16)
    DP_GO(DP_F16, DP_F16)
    DP_GO(DP_F16, DP_F32)
#undef DP_GO2
#undef DP_GO
    return hipGetLastError();
}

size_t embed_workspace(int64_t dim, int64_t tokens, int n) {
    return static_cast<size_t>(4 * round256(4 * n * tokens) + round256(4 * int64_t{n} * kMaxSpans * kDigits) +
                               round256(8 * n * chunks_of(tokens) * dim));
}

int64_t embed_waves(const EmbedGrad& a) {
    return chunks_of(a.tokens) * slices_of(a.dim);
}

int64_t embed_groups(const EmbedGrad& a) {
    return a.n * (kMaxSpans + (a.overwrite ? (a.rows * a.dim + kZeroSpan - 1) / kZeroSpan : 0));
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
    ids.n = a.tokens > 0 ? a.n : 0;
    Zeros z{};
    if (a.overwrite) {
        z.n = a.n;
        z.elements = a.rows * a.dim;
        z.once = 4 * z.elements * a.n > kLastLevel;
        z.span = z.once ? kZeroSpanOnce : kZeroSpan;
        z.groups = (z.elements + z.span - 1) / z.span;
        for (int r = 0; r < a.n; ++r) z.acc[r] = a.acc[r];
    }
    const int64_t zeros = z.groups * z.n;
    if (ids.n + zeros == 0) return hipSuccess;
    const int passes = passes_of(a.rows);
    int from = 0;
    if (a.tokens <= kSmallSort) {
        const dim3 sgrid(static_cast<unsigned>(ids.n + zeros));
#define DP_GO(K) \
    hipLaunchKernelGGL((k_sort_small<K>), sgrid, dim3(kSortThreads), 0, stream, ids, sb, z, a.rows, a.tokens, passes)
        if (a.tokens <= kSortThreads) DP_GO(1);
        else if (a.tokens <= 4 * kSortThreads) DP_GO(4);
        else if (a.tokens <= 8 * kSortThreads) DP_GO(8);
        else DP_GO(16);
#undef DP_GO
    } else {
        const int64_t tiles = (a.tokens + kTile - 1) / kTile;
        const int64_t span = (tiles + kMaxSpans - 1) / kMaxSpans * kTile;
        const int spans = static_cast<int>((a.tokens + span - 1) / span);
        for (int p = 0; p < passes; ++p) {
            const dim3 cgrid(static_cast<unsigned>(spans * a.n + (p == 0 ? zeros : 0)));
            hipLaunchKernelGGL(k_sort_count, cgrid, dim3(kSortThreads), 0, stream, ids, sb, z, from, p == 0, a.rows,
                               a.tokens, span, spans, 8 * p);
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
    if (g.chunks == 0) return hipSuccess;
    const dim3 grid(static_cast<unsigned>(embed_waves(a)), static_cast<unsigned>(a.n));
#define DP_GO(D)                                                                                   \
    if (dt == D) {                                                                                 \
        if (a.overwrite) hipLaunchKernelGGL((k_embed_sum<D, true>), grid, dim3(64 * kSpans), 0, stream, g); \
        else hipLaunchKernelGGL((k_embed_sum<D, false>), grid, dim3(64 * kSpans), 0, stream, g);            \
    }
    DP_GO(DP_F32)
    DP_GO(DP_F16)
    DP_GO(DP_BF16)
#undef DP_GO
    e = hipGetLastError();
    if (e != hipSuccess || g.chunks < 2) return e;
    if (a.overwrite) hipLaunchKernelGGL((k_embed_join<true>), grid, dim3(64), 0, stream, g);
    else hipLaunchKernelGGL((k_embed_join<false>), grid, dim3(64), 0, stream, g);
    return hipGetLastError();
}

}  // namespace dpk

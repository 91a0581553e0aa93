// gfx950 kernel of the distillation loss and its gradient, a workgroup for each row
// of logits.
//
// The gradient needs the sums over the whole row, so the row stays in registers
// between the two (50257 logits of 16 bits are 28 registers of 1024 threads) and
// is read from memory once: read, greatest logit, sums, gradient, write.  The
// teacher's list is gathered beside it into LDS, with a bit for each token of the list,
// by which the sums leave these tokens out of the rest.  Where the rest lies far below
// the row's greatest logit, it is summed again relative to its own greatest one (kFaint).
// The gradient is written as if no token were listed; then the listed ones and the
// label are written again.
// Memory bound: 16384 x 32000 bf16 logits with their gradient 390 to 405 us, 5.0 to 5.2 TB/s of
// what is read and written once (a large copy 4.9); losses alone, 4096 x 50257 binary32, 130 to
// 132 us, 5.9 TB/s (in both one row in 16 has the weight 0 and is not read).
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "dp_attention.h"
#include "dp_device.h"

namespace dpk {
namespace {

constexpr float kLog2e = 1.44269504088896340736f;
constexpr float kLn2 = 0.69314718055994530942f;
constexpr float kInf = __builtin_inff();
constexpr float kMost = 3.402823466e38f;

// Exponentials relative to the row's greatest logit are zero from 87 temperatures below
// it on, but the remainder's term, p' log(p' / q'), grows with this distance.  A sum of
// the tokens outside the list below kFaint is taken anew, relative to the greatest of
// them: above it, the terms that are lost, at most 2^18 of 2^-126, are less than 2^-44 of
// the sum.  So it is where the gradient's factor, others / sum, leaves binary32.
constexpr float kFaint = 0x1p-64f;

__device__ __forceinline__ float wave_max(float x) {
#pragma unroll
    for (int m = 1; m < 64; m <<= 1) x = fmaxf(x, __shfl_xor(x, m));
    return x;
}

// A value that all lanes have, in a scalar register.
__device__ __forceinline__ float uniform(float x) {
    return __builtin_bit_cast(float, __builtin_amdgcn_readfirstlane(__builtin_bit_cast(int, x)));
}

__device__ __forceinline__ float load_any(dp_dtype dt, const void* p, int64_t i) {
    return dt == DP_F32 ? load1<DP_F32>(p, i) : dt == DP_F16 ? load1<DP_F16>(p, i) : load1<DP_BF16>(p, i);
}
__device__ __forceinline__ int64_t load_id(int bytes, const void* p, int64_t i) {
    return bytes == 4 ? gload<int32_t>(p, i) : gload<int64_t>(p, i);
}

// One row's logits in pieces of 16 bytes at aligned addresses: piece i holds the
// logits kN i - shift + 0 .. kN - 1, those outside the row as -infinity.  A piece that
// the row's ends cut short is loaded from inside the row and moved into place when
// it is used (`settle`), so that no load lies behind a branch that waits for it.
// kTiny: a row shorter than a piece, element by element.
template <dp_dtype DT, bool kTiny>
struct Row {
    static constexpr int kN = DT == DP_F32 ? 4 : 8, kSize = 16 / kN;
    typedef Raw<DT, kN> Piece;
    const char* p;
    int shift, vocab, pieces;

    __device__ __forceinline__ Row(const void* logits, int64_t row, int64_t ld, int64_t v) {
        p = static_cast<const char*>(logits) + row * ld * kSize;
        shift = kTiny ? 0 : static_cast<int>(reinterpret_cast<uintptr_t>(p) / kSize % kN);
        vocab = static_cast<int>(v);
        pieces = (vocab + shift + kN - 1) / kN;
    }
    // -infinity in every element of a word
    static constexpr unsigned int kNone = DT == DP_F32 ? 0xff800000u : DT == DP_F16 ? 0xfc00fc00u : 0xff80ff80u;
    __device__ __forceinline__ Piece load(int i) const {  // past the last piece: that one
        Piece q;
        if constexpr (kTiny) {
            float x[kN];
#pragma unroll
            for (int j = 0; j < kN; ++j) x[j] = j < vocab ? load1<DT>(p, j) : -kInf;
#pragma unroll
            for (int j = 0; j < 4; ++j)
                q.w[j] = DT == DP_F32 ? __builtin_bit_cast(unsigned int, x[j * kN / 4])
                                      : pack2<DT == DP_F32 ? DP_BF16 : DT>(x[j * kN / 4], x[j * kN / 4 + kN / 8]);
        } else {
            int at = (i < pieces ? i : pieces - 1) * kN - shift;
            at = at < 0 ? 0 : at > vocab - kN ? vocab - kN : at;
            const u32x4 v = gload<u32x4, kSize>(p + static_cast<int64_t>(at) * kSize, 0);
#pragma unroll
            for (int j = 0; j < 4; ++j) q.w[j] = v[j];
        }
        return q;
    }
    __device__ __forceinline__ void settle(int i, Piece& q) const {
        if (i > 0 && i < pieces - 1) return;
        const int at = i * kN - shift;
        if (kTiny || i >= pieces) {
            if (i >= pieces)
#pragma unroll
                for (int j = 0; j < 4; ++j) q.w[j] = kNone;
            return;
        }
        // by how many elements the piece was loaded too late (the first one) or too early
        const int up = at < 0 ? -at : 0, down = at > vocab - kN ? at - (vocab - kN) : 0;
        constexpr int kWord = DT == DP_F32 ? 1 : 2;  // elements
        unsigned int* w = q.w;
        if (down & (2 * kWord)) w[0] = w[2], w[1] = w[3], w[2] = w[3] = kNone;
        if (down & kWord) w[0] = w[1], w[1] = w[2], w[2] = w[3], w[3] = kNone;
        if (up & (2 * kWord)) w[3] = w[1], w[2] = w[0], w[0] = w[1] = kNone;
        if (up & kWord) w[3] = w[2], w[2] = w[1], w[1] = w[0], w[0] = kNone;
        if constexpr (kWord == 2) {
            if (down & 1)
#pragma unroll
                for (int j = 0; j < 4; ++j) w[j] = __builtin_amdgcn_alignbit(j < 3 ? w[j + 1] : kNone, w[j], 16);
            if (up & 1)
#pragma unroll
                for (int j = 3; j >= 0; --j) w[j] = __builtin_amdgcn_alignbit(w[j], j > 0 ? w[j - 1] : kNone, 16);
        }
    }
    __device__ __forceinline__ void store(void* out, int i, const float* x) const {
        const int at = i * kN - shift;
        if (at >= 0 && at + kN <= vocab) {
            store_n<DT, kN, true>(out, at, kN, x);
        } else {
#pragma unroll
            for (int j = 0; j < kN; ++j)
                if (at + j >= 0 && at + j < vocab) store1<DT>(out, at + j, x[j]);
        }
    }
};

constexpr int kStream = 0, kTinyRow = -1;

// kKept pieces of a row in a thread's registers; kStream: the row is read piece by
// piece, once for the sums, which follow each thread's greatest logit, and once for
// the gradient; kTinyRow: one piece, read element by element.
template <dp_dtype DT, int kThreads, int kKept>
__global__ void __launch_bounds__(kThreads) k_distill(DistillArgs a, dp_dtype teacher_dt) {
    using R = Row<DT, kKept == kTinyRow>;
    constexpr int kPieces = kKept == kTinyRow ? 1 : kKept;
    constexpr int kN = R::kN, kWaves = kThreads / 64, kSums = 5;
    // Rows with a CU of their own wait for the exponentials, so the gradient takes those of
    // the sums from registers, as far as they fit: 61 x 50257 bf16 11.0 us, without 12.9.
    constexpr bool kHold = kThreads == 1024 && kPieces > 0 && kPieces <= 7;
    extern __shared__ unsigned int dyn[];
    __shared__ float tops[2][kWaves], sums[kSums][kWaves];
    const int K = a.top, tid = threadIdx.x;
    int* const ids = reinterpret_cast<int*>(dyn);                   // -1: not in the list
    float* const teacher = reinterpret_cast<float*>(dyn + K);       // y / tau, then p
    float* const student = reinterpret_cast<float*>(dyn + 2 * K);   // the logit
    unsigned int* const bits = dyn + 3 * K;                         // of token v at v + shift

    // What does not depend on anything is asked for first, together: a row of few
    // rows waits for memory twice, not five times.
    const int64_t t = blockIdx.x;
    const bool rest = a.total != nullptr;
    const float weight = a.weight ? gload<float>(a.weight, t) : 1.0f;
    const float total = rest ? gload<float>(a.total, t) : 0.0f;
    int64_t y_label = -1;
    if (a.hard != 0.0f && a.labels) y_label = load_id(a.id_bytes, a.labels, t);
    const float heat = 1.0f / a.temperature;
    float list = -kInf;
    for (int k = tid; k < K; k += kThreads) {
        const int64_t id = load_id(a.id_bytes, a.ids, t * a.ld_ids + k);
        const float y = load_any(teacher_dt, a.teacher, t * a.ld_teacher + k) * heat;
        const bool there = id >= 0 && id < a.vocab;
        ids[k] = there ? static_cast<int>(id) : -1;
        teacher[k] = there ? y : -kInf;
        list = fmaxf(list, there ? y : -kInf);
    }
    const R row(a.logits, t, a.ld, a.vocab);
    char* const out = a.dlogits ? static_cast<char*>(a.dlogits) + t * a.ld_dlogits * R::kSize : nullptr;
    if (weight == 0.0f) {
        if (a.loss && tid == 0) gstore<float>(a.loss, t, 0.0f);
        float x[kN];
#pragma unroll
        for (int j = 0; j < kN; ++j) x[j] = 0.0f;
        if (out)
            for (int i = tid; i < row.pieces; i += kThreads) row.store(out, i, x);
        return;
    }

    // 1. the row, its logits of the list, and the greatest of both
    typename R::Piece kept[kPieces > 0 ? kPieces : 1];
#pragma unroll
    for (int k = 0; k < kPieces; ++k)
        if (k * kThreads < row.pieces) kept[k] = row.load(k * kThreads + tid);
    const int label = y_label >= 0 && y_label < a.vocab ? static_cast<int>(y_label) : -1;
    const float target = label >= 0 ? load1<DT>(row.p, label) : 0.0f;
    for (int k = tid; k < K; k += kThreads) student[k] = ids[k] >= 0 ? load1<DT>(row.p, ids[k]) : 0.0f;
    const auto each = [&](auto&& use) {  // use(piece, its logits, its place in the registers)
        if constexpr (kKept != kStream) {
#pragma unroll
            for (int k = 0; k < kPieces; ++k) {
                if (k * kThreads < row.pieces) {
                    float x[kN];
                    expand<DT, kN>(kept[k], x);
                    use(k * kThreads + tid, x, k);
                }
            }
        } else {
            constexpr int kAhead = 4;  // pieces on their way together
            for (int i = 0; i < row.pieces; i += kAhead * kThreads) {
                typename R::Piece q[kAhead];
#pragma unroll
                for (int k = 0; k < kAhead; ++k) q[k] = row.load(i + k * kThreads + tid);
#pragma unroll
                for (int k = 0; k < kAhead; ++k) {
                    float x[kN];
                    row.settle(i + k * kThreads + tid, q[k]);
                    expand<DT, kN>(q[k], x);
                    use(i + k * kThreads + tid, x, 0);
                }
            }
        }
    };
    // The same for the few rows whose remainder is faint: from memory again, in little code.
    const auto walk = [&](auto&& use) {
#pragma unroll 1
        for (int i = tid; i < row.pieces; i += kThreads) {
            typename R::Piece q = row.load(i);
            float x[kN];
            row.settle(i, q);
            expand<DT, kN>(q, x);
            use(i, x);
        }
    };
    for (int i = tid; i < (row.vocab + row.shift + 31) / 32; i += kThreads) bits[i] = 0;
    bool twice = false;
    const auto mark = [&]() {
        for (int k = tid; k < K; k += kThreads)
            if (ids[k] >= 0) {
                const int at = ids[k] + row.shift;
                twice |= (atomicOr(&bits[at >> 5], 1u << (at & 31)) >> (at & 31) & 1) != 0;
            }
    };
    // Exponentials are 2^(z c - peak), peak = top c as rounded: a row's reference, which
    // log_all and the label's term take it for, so its rounding cancels.
    const bool both = a.hard != 0.0f && a.temperature != 1.0f, square = a.temperature == 2.0f;
    const float c = kLog2e * heat;
    float held[kHold ? kPieces : 1][kN];
    float s[kSums] = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f};
    // Which elements of piece i are tokens of the list.
    const auto listed_of = [&](int i) { return bits[(i < row.pieces ? i : 0) * kN >> 5] >> (i * kN & 31); };
    // A piece's part of the sums of the row at both temperatures, and of the tokens
    // outside the list.  At 2 the exponential without the temperature is the square.
    const auto add = [&](int i, const float* x, float peak, float peak1, float* e) {
#pragma unroll
        for (int j = 0; j < kN; ++j) {
            e[j] = __builtin_amdgcn_exp2f(__builtin_fmaf(x[j], c, -peak));
            s[0] += e[j];
        }
        if (rest) {
            const unsigned int listed = listed_of(i);
#pragma unroll
            for (int j = 0; j < kN; ++j) s[1] += listed >> j & 1 ? 0.0f : e[j];
        }
        if (both) {
            if (square) {
#pragma unroll
                for (int j = 0; j < kN; ++j) s[2] = __builtin_fmaf(e[j], e[j], s[2]);
            } else {
#pragma unroll
                for (int j = 0; j < kN; ++j) s[2] += __builtin_amdgcn_exp2f(__builtin_fmaf(x[j], kLog2e, -peak1));
            }
        }
    };
    float top = -kInf, own = -kInf, own1 = -kInf;  // own: the thread's reference while it streams
    if constexpr (kKept == kStream) {
        if (rest) {
            __syncthreads();
            mark();
            __syncthreads();
        }
        each([&](int i, const float* x, int) {
            float high = x[0];
#pragma unroll
            for (int j = 1; j < kN; ++j) high = fmaxf(high, x[j]);
            if (high > top) {
                top = high;
                const float peak = top * c, peak1 = square ? 2.0f * peak : top * kLog2e;
                const float less = __builtin_amdgcn_exp2f(own - peak);
                s[0] *= less;
                s[1] *= less;
                s[2] *= __builtin_amdgcn_exp2f(own1 - peak1);
                own = peak;
                own1 = peak1;
            }
            // nothing but -infinity yet: any reference gives zeros
            float e[kN];
            add(i, x, own == -kInf ? 0.0f : own, own1 == -kInf ? 0.0f : own1, e);
        });
    } else {
#pragma unroll
        for (int k = 0; k < kPieces; ++k)
            if (k * kThreads < row.pieces && (k == 0 || (k + 1) * kThreads >= row.pieces)) row.settle(k * kThreads + tid, kept[k]);
        each([&](int, const float* x, int) {
#pragma unroll
            for (int j = 0; j < kN; ++j) top = fmaxf(top, x[j]);
        });
    }
    top = wave_max(top);
    list = wave_max(list);
    if ((tid & 63) == 0) {
        tops[0][tid >> 6] = top;
        tops[1][tid >> 6] = list;
    }
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kWaves; ++w) {
        top = fmaxf(top, tops[0][w]);
        list = fmaxf(list, tops[1][w]);
    }
    if (kKept != kStream || !rest) mark();
    twice = __syncthreads_or(twice);

    // 2. the sums, and those of the list's probabilities and of their products with
    // log p / q
    const float peak = uniform(top * c), peak1 = uniform(square ? 2.0f * peak : top * kLog2e);
    const auto plain = [&](float z, float e) { return square ? e * e : __builtin_amdgcn_exp2f(__builtin_fmaf(z, kLog2e, -peak1)); };
    const float base = uniform(rest ? total : list == -kInf ? 0.0f : list);
    if constexpr (kKept == kStream) {
        const float less = __builtin_amdgcn_exp2f(own - peak), less1 = __builtin_amdgcn_exp2f(own1 - peak1);
        s[0] *= less;
        s[1] *= less;
        s[2] *= less1;
    } else {
        each([&](int i, const float* x, int k) {
            float e[kN];
            add(i, x, peak, peak1, kHold ? held[k] : e);
        });
    }
    for (int k = tid; k < K; k += kThreads) {
        if (ids[k] < 0) continue;
        const float y = teacher[k] - base, p = __builtin_amdgcn_exp2f(y * kLog2e);
        teacher[k] = p;
        s[3] += p;
        if (p > 0.0f) s[4] += p * (y - kLn2 * __builtin_fmaf(student[k], c, -peak));
    }
#pragma unroll
    for (int n = 0; n < kSums; ++n) {
        s[n] = wave_sum(s[n]);
        if ((tid & 63) == 0) sums[n][tid >> 6] = s[n];
    }
    __syncthreads();
#pragma unroll
    for (int n = 0; n < kSums; ++n) {
        s[n] = 0.0f;
#pragma unroll
        for (int w = 0; w < kWaves; ++w) s[n] += sums[n][w];
        s[n] = uniform(s[n]);
    }
    if (!both) s[2] = s[0];

    const float log_all = kLn2 * __builtin_amdgcn_logf(s[0]);
    const float factor = a.scale * weight, soft = factor * a.soft * a.temperature;
    float kl = 0.0f, mass = 0.0f, others = 0.0f, norm = 1.0f;  // norm: of the list's p
    float low = peak;  // the reference of s[1]
    bool faint = false;
    if (rest) {
        others = 1.0f - s[3];
        faint = others > 0.0f && (s[1] < kFaint || !(fabsf(soft * (others / s[1])) <= kMost));
        if (faint) {
            float high = -kInf;
            walk([&](int i, const float* x) {
                const unsigned int listed = listed_of(i);
#pragma unroll
                for (int j = 0; j < kN; ++j) high = listed >> j & 1 ? high : fmaxf(high, x[j]);
            });
            high = wave_max(high);
            if ((tid & 63) == 0) tops[0][tid >> 6] = high;
            __syncthreads();
#pragma unroll
            for (int w = 0; w < kWaves; ++w) high = fmaxf(high, tops[0][w]);
            low = uniform(high * c);
            float sum = 0.0f;
            if (high != -kInf)  // else there is no such token, or none that the student gives anything to
                walk([&](int i, const float* x) {
                    const unsigned int listed = listed_of(i);
#pragma unroll
                    for (int j = 0; j < kN; ++j)
                        sum += listed >> j & 1 ? 0.0f : __builtin_amdgcn_exp2f(__builtin_fmaf(x[j], c, -low));
                });
            sum = wave_sum(sum);
            if ((tid & 63) == 0) sums[0][tid >> 6] = sum;
            __syncthreads();
            s[1] = 0.0f;
#pragma unroll
            for (int w = 0; w < kWaves; ++w) s[1] += sums[0][w];
            s[1] = uniform(s[1]);
        }
        if (!(others > 0.0f) || s[1] == 0.0f) others = s[3] != s[3] ? s[3] : 0.0f;
        kl = s[4] + s[3] * log_all;
        if (others > 0.0f)
            kl += others * (kLn2 * __builtin_amdgcn_logf(others) - (kLn2 * (__builtin_amdgcn_logf(s[1]) + (low - peak)) - log_all));
        mass = s[3] + others;
    } else if (s[3] != 0.0f) {  // a list; one of nothing but NaN, too, whose maximum is -infinity
        norm = 1.0f / s[3];
        kl = s[4] * norm - kLn2 * __builtin_amdgcn_logf(s[3]) + log_all;
        mass = s[3] != s[3] ? s[3] : 1.0f;
    }
    const float ce = kLn2 * (__builtin_amdgcn_logf(s[2]) - __builtin_fmaf(target, both ? kLog2e : c, both ? -peak1 : -peak));
    if (a.loss && tid == 0)
        gstore<float>(a.loss, t, a.soft * a.temperature * a.temperature * kl + (label >= 0 ? a.hard * ce : 0.0f));
    if (!out) return;
    __syncthreads();  // in place: every logit of the list and the label's are read

    // 3. the gradient of the tokens outside the list, then of the others
    const float hard = uniform(label >= 0 ? factor * a.hard / s[2] : 0.0f);
    const float in = uniform(soft * (mass / s[0])), share = uniform(others > 0.0f ? soft * (others / s[1]) : 0.0f);
    faint = faint && others > 0.0f;  // then what the remainder takes is written with its own reference
    const float over = uniform(faint ? in : in - share);
    if (faint) walk([&](int i, const float* x) {
        float g[kN];
#pragma unroll
        for (int j = 0; j < kN; ++j) {
            const float e = __builtin_amdgcn_exp2f(__builtin_fmaf(x[j], c, -peak));
            g[j] = __builtin_fmaf(both ? plain(x[j], e) : e, hard, e * in);
            g[j] -= share * __builtin_amdgcn_exp2f(__builtin_fmaf(x[j], c, -low));
        }
        row.store(out, i, g);
    });
    else each([&](int i, const float* x, int k) {
        float g[kN];
        const auto power = [&](int j) { return kHold ? held[k][j] : __builtin_amdgcn_exp2f(__builtin_fmaf(x[j], c, -peak)); };
        if (both && square) {  // e over + e^2 hard
#pragma unroll
            for (int j = 0; j < kN; ++j) {
                const float e = power(j);
                g[j] = e * __builtin_fmaf(e, hard, over);
            }
        } else {
#pragma unroll
            for (int j = 0; j < kN; ++j) g[j] = power(j) * (both ? over : over + hard);
            if (both) {
#pragma unroll
                for (int j = 0; j < kN; ++j) g[j] = __builtin_fmaf(plain(x[j], 0.0f), hard, g[j]);
            }
        }
        if (i < row.pieces) row.store(out, i, g);
    });
    __syncthreads();
    const auto again = [&](int id, float z, float p, float coefficient, bool remainder) {
        const float e = __builtin_amdgcn_exp2f(__builtin_fmaf(z, c, -peak));
        float g = e * coefficient - soft * p;
        if (remainder) g -= share * __builtin_amdgcn_exp2f(__builtin_fmaf(z, c, -low));
        const float e1 = both ? plain(z, e) : e;
        g += e1 * hard;
        if (id == label) g -= factor * a.hard;
        store1<DT>(out, id, g);
    };
    for (int k = tid; k < K; k += kThreads) {
        if (ids[k] < 0) continue;
        float p = teacher[k] * norm;
        if (twice) {  // the first of a token's places in the list writes for all of them
            bool earlier = false;
            p = 0.0f;
            for (int i = 0; i < K; ++i)
                if (ids[i] == ids[k]) {
                    earlier |= i < k;
                    p += teacher[i] * norm;
                }
            if (earlier) continue;
        }
        again(ids[k], student[k], p, in, false);
    }
    if (tid == 0 && label >= 0) {
        const int at = label + row.shift;
        if (!(bits[at >> 5] >> (at & 31) & 1)) again(label, target, 0.0f, over, faint);
    }
}

template <dp_dtype DT, int kThreads, int kKept>
hipError_t go(const DistillArgs& a, dp_dtype teacher_dt, hipStream_t stream) {
    const size_t lds = 12 * static_cast<size_t>(a.top) + 4 * static_cast<size_t>((a.vocab + 8 + 31) / 32);
    hipLaunchKernelGGL((k_distill<DT, kThreads, kKept>), dim3(static_cast<unsigned>(a.tokens)), dim3(kThreads), lds, stream,
                       a, teacher_dt);
    return hipGetLastError();
}

// The smallest number of registers that holds a row.  Many rows hide each other's
// waits, so small workgroups, of which three or four are on a CU at once, take them:
// 16384 x 32000 bf16 logits with their gradient 390 us by 512 threads a row, 398 by 256,
// 446 to 680 by 1024.  Up to one row a CU, a row has all threads that a workgroup can have.
// Many rows' losses alone need no row twice and are streamed: 4096 x 50257 in binary32 139
// us by 1024 threads a row and 163 by 256, from registers 187; 16384 x 32000 bf16 302, 207
// and 214.
template <dp_dtype DT>
hipError_t launch_row(const DistillArgs& a, dp_dtype teacher_dt, hipStream_t stream) {
    constexpr int kN = DT == DP_F32 ? 4 : 8;
    if (a.vocab < kN) return go<DT, 64, kTinyRow>(a, teacher_dt, stream);
    const int64_t pieces = (a.vocab + kN - 1 + kN - 1) / kN;  // at any alignment
    if (a.tokens > 256) {
        if (pieces <= 256 * 4) return go<DT, 256, 4>(a, teacher_dt, stream);
        if (!a.dlogits) return pieces <= 1024 * 8 ? go<DT, 256, kStream>(a, teacher_dt, stream) : go<DT, 1024, kStream>(a, teacher_dt, stream);
        if (pieces <= 256 * 8) return go<DT, 256, 8>(a, teacher_dt, stream);
        if (pieces <= 512 * 8) return go<DT, 512, 8>(a, teacher_dt, stream);
        if (pieces <= 512 * 13) return go<DT, 512, 13>(a, teacher_dt, stream);
    }
    if (pieces <= 1024 * 2) return go<DT, 1024, 2>(a, teacher_dt, stream);
    if (pieces <= 1024 * 7) return go<DT, 1024, 7>(a, teacher_dt, stream);
    if (pieces <= 1024 * 13) return go<DT, 1024, 13>(a, teacher_dt, stream);
    if (pieces <= 1024 * 16) return go<DT, 1024, 16>(a, teacher_dt, stream);
    return go<DT, 1024, kStream>(a, teacher_dt, stream);
}

}  // namespace

hipError_t launch_distill(dp_dtype dt, dp_dtype teacher_dt, const DistillArgs& a, hipStream_t stream) {
    if (a.tokens == 0) return hipSuccess;
    if (dt == DP_F32) return launch_row<DP_F32>(a, teacher_dt, stream);
    if (dt == DP_F16) return launch_row<DP_F16>(a, teacher_dt, stream);
    return launch_row<DP_BF16>(a, teacher_dt, stream);
}

}  // namespace dpk

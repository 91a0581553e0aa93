// Device helpers of the layer operators: element types, rows read and written
// in vectors, reductions over a wave.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "dpstep.h"

namespace dpk {

#define DP_GLOBAL __attribute__((address_space(1)))

typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef unsigned int u32x2 __attribute__((ext_vector_type(2)));
typedef unsigned int u32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));

// Global memory in units of V at the alignment A: vectors may lie at any
// element (unaligned access is on for compute, so a vector at 2-byte alignment is
// still one instruction).
template <typename V, int A>
struct Loose {
    typedef V type __attribute__((aligned(A)));
};
template <typename V, int A = sizeof(V)>
__device__ __forceinline__ V gload(const void* p, int64_t i) {
    return ((const DP_GLOBAL typename Loose<V, A>::type*)p)[i];
}
template <typename V, int A = sizeof(V)>
__device__ __forceinline__ void gstore(void* p, int64_t i, V x) {
    ((DP_GLOBAL typename Loose<V, A>::type*)p)[i] = x;
}
template <typename V, int A = sizeof(V)>
__device__ __forceinline__ void gstore_nt(void* p, int64_t i, V x) {
    __builtin_nontemporal_store(x, ((DP_GLOBAL typename Loose<V, A>::type*)p) + i);
}

// Two binary32 values as two 16-bit elements in one word and back (to nearest
// even; one conversion instruction each way).
template <dp_dtype DT>
__device__ __forceinline__ unsigned int pack2(float a, float b) {
    if constexpr (DT == DP_BF16) {
        return __builtin_bit_cast(unsigned int, __builtin_convertvector((f32x2{a, b}), bf16x2));
    } else {
        return __builtin_bit_cast(unsigned int, __builtin_convertvector((f32x2{a, b}), f16x2));
    }
}
template <dp_dtype DT>
__device__ __forceinline__ void unpack2(unsigned int u, float* o) {
    if constexpr (DT == DP_BF16) {
        o[0] = __builtin_bit_cast(float, u << 16);
        o[1] = __builtin_bit_cast(float, u & 0xffff0000u);
    } else {
        const f16x2 h = __builtin_bit_cast(f16x2, u);
        o[0] = static_cast<float>(h[0]);
        o[1] = static_cast<float>(h[1]);
    }
}

template <dp_dtype DT>
__device__ __forceinline__ float load1(const void* p, int64_t i) {
    if constexpr (DT == DP_F32) return gload<float>(p, i);
    if constexpr (DT == DP_F16) return static_cast<float>(gload<_Float16>(p, i));
    return __builtin_bit_cast(float, static_cast<unsigned int>(gload<unsigned short>(p, i)) << 16);
}
template <dp_dtype DT>
__device__ __forceinline__ void store1(void* p, int64_t i, float x) {
    if constexpr (DT == DP_F32) {
        gstore<float>(p, i, x);
    } else {
        gstore<unsigned short>(p, i, static_cast<unsigned short>(pack2<DT>(x, 0.0f)));
    }
}

// The sum of a wave's 64 values, in every lane, in a fixed order: within rows of
// 16 lanes by shifts of 1, 2, 4 and 8, then over the rows (data-parallel moves
// folded into the additions; a butterfly through LDS costs ten times as long).
template <int kCtrl, int kRows>
__device__ __forceinline__ float moved(float x) {
    return __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, x), kCtrl, kRows, 0xf, true));
}
__device__ __forceinline__ float wave_sum(float x) {
    x += moved<0x111, 0xf>(x);
    x += moved<0x112, 0xf>(x);
    x += moved<0x114, 0xf>(x);
    x += moved<0x118, 0xf>(x);
    x += moved<0x142, 0xa>(x);  // the last lane of rows 0 and 2 into rows 1 and 3
    x += moved<0x143, 0xc>(x);  // lane 31 into the upper half
    return __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, x), 63));
}

// N (4 or 8) consecutive elements from element i of p, of which the first
// `valid` exist (the others come back as zero, or are not written); a whole
// vector goes in one or two accesses.
template <dp_dtype DT, int N>
__device__ __forceinline__ void load_n(const void* p, int64_t i, int valid, float* o) {
    if (valid >= N) {
        if constexpr (DT == DP_F32) {
#pragma unroll
            for (int k = 0; k < N / 4; ++k) {
                const f32x4 v = gload<f32x4, 4>(static_cast<const float*>(p) + i, k);
#pragma unroll
                for (int j = 0; j < 4; ++j) o[4 * k + j] = v[j];
            }
        } else if constexpr (N == 8) {
            const u32x4 v = gload<u32x4, 2>(static_cast<const unsigned short*>(p) + i, 0);
#pragma unroll
            for (int j = 0; j < 4; ++j) unpack2<DT>(v[j], o + 2 * j);
        } else {
            const u32x2 v = gload<u32x2, 2>(static_cast<const unsigned short*>(p) + i, 0);
#pragma unroll
            for (int j = 0; j < 2; ++j) unpack2<DT>(v[j], o + 2 * j);
        }
        return;
    }
#pragma unroll
    for (int j = 0; j < N; ++j) o[j] = j < valid ? load1<DT>(p, i + j) : 0.0f;
}
// kOnce: the data is not read again soon, so it need not stay in the caches.
template <dp_dtype DT, int N, bool kOnce = false>
__device__ __forceinline__ void store_n(void* p, int64_t i, int valid, const float* x) {
    const auto put = [](auto* at, int64_t k, auto v) {
        constexpr int kAlign = sizeof(*at);
        if constexpr (kOnce) gstore_nt<decltype(v), kAlign>(at, k, v);
        else gstore<decltype(v), kAlign>(at, k, v);
    };
    if (valid >= N) {
        if constexpr (DT == DP_F32) {
#pragma unroll
            for (int k = 0; k < N / 4; ++k)
                put(static_cast<float*>(p) + i, k, f32x4{x[4 * k], x[4 * k + 1], x[4 * k + 2], x[4 * k + 3]});
        } else if constexpr (N == 8) {
            put(static_cast<unsigned short*>(p) + i, 0,
                u32x4{pack2<DT>(x[0], x[1]), pack2<DT>(x[2], x[3]), pack2<DT>(x[4], x[5]), pack2<DT>(x[6], x[7])});
        } else {
            put(static_cast<unsigned short*>(p) + i, 0, u32x2{pack2<DT>(x[0], x[1]), pack2<DT>(x[2], x[3])});
        }
        return;
    }
#pragma unroll
    for (int j = 0; j < N; ++j)
        if (j < valid) store1<DT>(p, i + j, x[j]);
}

// VW (4 or 8) elements as they lie in memory.
template <dp_dtype DT, int VW>
struct Raw {
    static constexpr int kWords = VW * (DT == DP_F32 ? 4 : 2) / 4;
    unsigned int w[kWords];
};

// A lane's piece of a row, loaded ahead of its use: elements i .. i + VW - 1 of p,
// of which the first `valid` belong to the row.  A piece that the row's end cuts
// short is loaded whole from VW - valid elements earlier (`whole`: the row has
// that many), and `settle` moves its elements into place when they are used, so
// that no lane waits for its loads where they are issued.
template <dp_dtype DT, int VW>
__device__ __forceinline__ Raw<DT, VW> load_raw(const void* p, int64_t i, int valid, bool whole) {
    constexpr int kWords = Raw<DT, VW>::kWords;
    constexpr int kSize = DT == DP_F32 ? 4 : 2;
    Raw<DT, VW> q;
#pragma unroll
    for (int k = 0; k < kWords; ++k) q.w[k] = 0;
    if (valid <= 0) return q;
    if (whole) {
        const char* at = static_cast<const char*>(p) + (i - (VW - valid)) * kSize;
        if constexpr (kWords == 2) {
            const u32x2 v = gload<u32x2, kSize>(at, 0);
            q.w[0] = v[0];
            q.w[1] = v[1];
        } else {
#pragma unroll
            for (int k = 0; k < kWords / 4; ++k) {
                const u32x4 v = gload<u32x4, kSize>(at, k);
#pragma unroll
                for (int j = 0; j < 4; ++j) q.w[4 * k + j] = v[j];
            }
        }
    } else if constexpr (DT == DP_F32) {
#pragma unroll
        for (int j = 0; j < VW; ++j) q.w[j] = j < valid ? gload<unsigned int>(p, i + j) : 0u;
    } else {
#pragma unroll
        for (int j = 0; j < VW / 2; ++j) {
            const unsigned int lo = 2 * j < valid ? gload<unsigned short>(p, i + 2 * j) : 0u;
            const unsigned int hi = 2 * j + 1 < valid ? gload<unsigned short>(p, i + 2 * j + 1) : 0u;
            q.w[j] = lo | hi << 16;
        }
    }
    return q;
}
template <dp_dtype DT, int VW>
__device__ __forceinline__ void settle(Raw<DT, VW>& q, int valid, bool whole) {
    if (!whole || valid <= 0 || valid >= VW) return;
    constexpr int kWords = Raw<DT, VW>::kWords;
#pragma unroll
    for (int s = 0; s < VW - 1; ++s) {
        if (s >= VW - valid) break;  // one element down, VW - valid times
#pragma unroll
        for (int k = 0; k < kWords; ++k) {
            const unsigned int up = k + 1 < kWords ? q.w[k + 1] : 0u;
            q.w[k] = DT == DP_F32 ? up : __builtin_amdgcn_alignbit(up, q.w[k], 16);
        }
    }
}

template <dp_dtype DT, int VW>
__device__ __forceinline__ void expand(const Raw<DT, VW>& q, float* o) {
    if constexpr (DT == DP_F32) {
#pragma unroll
        for (int j = 0; j < VW; ++j) o[j] = __builtin_bit_cast(float, q.w[j]);
    } else {
#pragma unroll
        for (int j = 0; j < VW / 2; ++j) unpack2<DT>(q.w[j], o + 2 * j);
    }
}

}  // namespace dpk

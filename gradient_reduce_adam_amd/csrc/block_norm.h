// What the forward and the backward of the block norms share: rows in
// registers, reductions over a row, the choices of a launch.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "dp_device.h"
#include "dp_layers.h"

namespace dpk {

// Threads of a workgroup whose rows are held by nt threads each.
constexpr int block_of(int nt) { return nt < 256 ? 256 : nt; }

// Scratch of row_sum: 4 floats a wave for each of two turns, taken in
// alternation, so that one barrier a reduction is enough.
constexpr int sum_scratch(int nt) { return nt > 64 ? 2 * 4 * (block_of(nt) / 64) : 1; }

// Sums of K <= 4 values over the NT threads of a row, the same in each of them.
template <int NT, int K>
__device__ __forceinline__ void row_sum(float (&v)[K], float* lds, int& turn) {
#pragma unroll
    for (int k = 0; k < K; ++k) v[k] = wave_sum(v[k]);
    if constexpr (NT > 64) {
        constexpr int kWaves = NT / 64;  // of a row
        float* at = lds + turn * (block_of(NT) / 64) * 4;
        turn ^= 1;
        if ((threadIdx.x & 63) == 0)
#pragma unroll
            for (int k = 0; k < K; ++k) at[(threadIdx.x >> 6) * 4 + k] = v[k];
        __syncthreads();
        at += threadIdx.x / NT * kWaves * 4;
#pragma unroll
        for (int k = 0; k < K; ++k) {
            v[k] = 0.0f;
#pragma unroll
            for (int w = 0; w < kWaves; ++w) v[k] += at[w * 4 + k];
        }
    }
}

struct Weights {
    const void *post_w, *post_b, *gate, *pre_w, *pre_b;  // null: none
};

// The weights of this thread's columns stay packed in registers over all rows.
template <dp_dtype PT, int NV, int VW>
struct Column {
    Raw<PT, VW> q[NV];
    __device__ __forceinline__ void load(const void* p, int c0, int step, int dim) {
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const int left = dim - (c0 + k * step);
            const int valid = !p || left <= 0 ? 0 : left < VW ? left : VW;
            q[k] = load_raw<PT, VW>(p, c0 + k * step, valid, dim >= VW);
            settle<PT, VW>(q[k], valid, dim >= VW);
        }
    }
};

template <int VW>
__device__ __forceinline__ int valid_of(int dim, int c) {
    return dim - c >= VW ? VW : dim - c > 0 ? dim - c : 0;
}

// How a row is held: nt threads with nv vectors of vw elements each.
struct Shape {
    int nt, nv, vw;
};

inline Weights weights_of(const BlockNorm& b) {
    Weights w{};
    w.post_w = b.weight[0];
    w.post_b = b.weight[1];
    w.gate = b.weight[2];
    w.pre_w = b.weight[3];
    w.pre_b = b.weight[4];
    return w;
}


// Calls GO with the compile-time choices of a call: row type, weight type,
// mean, biases, post norm.  Centred norms take the form with biases whether or not
// they have any (an absent one reads as zero).
#define DP_KINDS(GO)                                                        \
    do {                                                                    \
        if (dt == DP_F32 && pdt == DP_BF16) DP_KINDS2(GO, DP_F32, DP_BF16)  \
        else if (dt == DP_F32) DP_KINDS2(GO, DP_F32, DP_F16)                \
        else if (dt == DP_F16) DP_KINDS2(GO, DP_F16, DP_F16)                \
        else DP_KINDS2(GO, DP_BF16, DP_BF16)                                \
    } while (0)
#define DP_KINDS2(GO, D, P)                                   \
    {                                                         \
        if (b.centered && post) GO(D, P, true, true, true);   \
        else if (b.centered) GO(D, P, true, true, false);     \
        else if (b.bias && post) GO(D, P, false, true, true); \
        else if (b.bias) GO(D, P, false, true, false);        \
        else if (post) GO(D, P, false, false, true);          \
        else GO(D, P, false, false, false);                   \
    }

}  // namespace dpk

// gfx950 kernels of the 8-bit activation format: rows to e4m3 codes with one
// power-of-two scale for 32 channels, and back.
//
// The scale of a group is 2^e with e the smallest power under which the
// largest finite magnitude is at most 448: with that magnitude 1.m * 2^k,
// e = k - 8 for 1.m <= 1.75, else k - 7, taken from the bits without a
// logarithm.  Multiplying by 2^-e is exact, so the only rounding is the
// conversion's, to nearest even.  Both kernels are bound by HBM (the row in its own
// type, one byte an element, and a byte for 32): a lane moves 16 consecutive
// elements, two lanes share a group.  Packing and unpacking 16384 x 11008 bf16
// takes 206 us together, 5.3 TB/s; with 8 elements a lane 5 to 8% more, and
// loads or stores that pass the caches by cost up to 14%.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "dp_device.h"
#include "dp_layers.h"

namespace dpk {
namespace {

constexpr int kThreads = 256;
constexpr int kSpan = 16;  // elements per thread: half a group

struct PackArgs {
    const void* in;
    const unsigned char* codes_in;
    const unsigned char* scales_in;
    void* out;
    unsigned char* codes;
    unsigned char* scales;
    int64_t tokens, dim, ld, ld_codes, ld_scales;
};

// The row and first column of this thread's span.  Spans are numbered along
// the rows, an even number of them in each (whole groups); a workgroup takes
// 256 consecutive ones.
__device__ __forceinline__ bool span_of(const PackArgs& a, int64_t& row, int64_t& c) {
    const uint32_t spans = static_cast<uint32_t>((a.dim + DPL_GROUP - 1) / DPL_GROUP) * (DPL_GROUP / kSpan);
    const int64_t first = static_cast<int64_t>(blockIdx.x) * kThreads;
    const int64_t row0 = first / spans;
    const uint32_t i = static_cast<uint32_t>(first - row0 * spans) + threadIdx.x;
    const uint32_t down = i / spans;
    row = row0 + down;
    c = static_cast<int64_t>(i - down * spans) * kSpan;
    return row < a.tokens;
}

template <dp_dtype DT>
__global__ void __launch_bounds__(kThreads) k_pack(PackArgs a) {
    int64_t row, c;
    const bool in = span_of(a, row, c);
    const int64_t left = in ? a.dim - c : 0;
    const int valid = left >= kSpan ? kSpan : left > 0 ? static_cast<int>(left) : 0;
    float v[kSpan];
    load_n<DT, 8>(a.in, row * a.ld + c, valid, v);
    load_n<DT, 8>(a.in, row * a.ld + c + 8, valid - 8, v + 8);
    float top = 0.0f;
#pragma unroll
    for (int j = 0; j < kSpan; ++j) {
        const float m = __builtin_fabsf(v[j]);
        if (m < __builtin_inff()) {
            if constexpr (DT == DP_F16) v[j] = __builtin_fminf(__builtin_fmaxf(v[j], -61440.0f), 61440.0f);
            top = __builtin_fmaxf(top, __builtin_fabsf(v[j]));
        }
    }
    top = __builtin_fmaxf(top, __shfl_xor(top, 1));  // the other half of the group
    const unsigned int bits = __builtin_bit_cast(unsigned int, top);
    int e = static_cast<int>(bits >> 23) - 135 + ((bits & 0x7fffffu) > 0x600000u ? 1 : 0);
    e = e < -117 ? -117 : e > 119 ? 119 : e;
    const float unit = __builtin_bit_cast(float, static_cast<unsigned int>(127 - e) << 23);
    u32x4 q;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        float f[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float x = v[4 * k + j] * unit;
            // values beyond 448 (a group at the scales' limit) are limited to it; no number becomes NaN
            const float lim = __builtin_fminf(__builtin_fmaxf(x, -448.0f), 448.0f);
            f[j] = __builtin_fabsf(v[4 * k + j]) < __builtin_inff() ? lim : __builtin_nanf("");
        }
        int w = __builtin_amdgcn_cvt_pk_fp8_f32(f[0], f[1], 0, false);
        w = __builtin_amdgcn_cvt_pk_fp8_f32(f[2], f[3], w, true);
        q[k] = static_cast<unsigned int>(w);
    }
    if (!in) return;
    unsigned char* out = a.codes + row * a.ld_codes + c;
    if (valid == kSpan) {
        gstore<u32x4, 1>(out, 0, q);
    } else {
#pragma unroll
        for (int j = 0; j < kSpan; ++j)
            if (j < valid) gstore<unsigned char>(out, j, static_cast<unsigned char>(q[j / 4] >> (8 * (j % 4))));
    }
    if ((threadIdx.x & 1) == 0)
        gstore<unsigned char>(a.scales, row * a.ld_scales + c / DPL_GROUP, static_cast<unsigned char>(e + 127));
}

template <dp_dtype DT>
__global__ void __launch_bounds__(kThreads) k_unpack(PackArgs a) {
    int64_t row, c;
    if (!span_of(a, row, c)) return;
    const int64_t left = a.dim - c;
    const int valid = left >= kSpan ? kSpan : left > 0 ? static_cast<int>(left) : 0;
    if (valid == 0) return;
    const unsigned char* in = a.codes_in + row * a.ld_codes + c;
    u32x4 q{0, 0, 0, 0};
    if (valid == kSpan) {
        q = gload<u32x4, 1>(in, 0);
    } else {
#pragma unroll
        for (int j = 0; j < kSpan; ++j)
            if (j < valid) q[j / 4] |= static_cast<unsigned int>(gload<unsigned char>(in, j)) << (8 * (j % 4));
    }
    const unsigned int byte = gload<unsigned char>(a.scales_in, row * a.ld_scales + c / DPL_GROUP);
    const float unit = __builtin_bit_cast(float, byte << 23);
    float v[kSpan];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const f32x2 lo = __builtin_amdgcn_cvt_pk_f32_fp8(static_cast<int>(q[k]), false);
        const f32x2 hi = __builtin_amdgcn_cvt_pk_f32_fp8(static_cast<int>(q[k]), true);
        v[4 * k] = lo[0] * unit;
        v[4 * k + 1] = lo[1] * unit;
        v[4 * k + 2] = hi[0] * unit;
        v[4 * k + 3] = hi[1] * unit;
    }
    store_n<DT, 8>(a.out, row * a.ld + c, valid, v);
    store_n<DT, 8>(a.out, row * a.ld + c + 8, valid - 8, v + 8);
}

dim3 grid_of(int64_t tokens, int64_t dim) {
    const int64_t spans = (dim + DPL_GROUP - 1) / DPL_GROUP * (DPL_GROUP / kSpan) * tokens;
    return dim3(static_cast<unsigned>((spans + kThreads - 1) / kThreads));
}

}  // namespace

hipError_t launch_pack(dp_dtype dt, int64_t tokens, int64_t dim, const void* x, int64_t ld, void* codes,
                       int64_t ld_codes, void* scales, int64_t ld_scales, hipStream_t stream) {
    if (tokens == 0) return hipSuccess;
    PackArgs a{};
    a.in = x;
    a.codes = static_cast<unsigned char*>(codes);
    a.scales = static_cast<unsigned char*>(scales);
    a.tokens = tokens;
    a.dim = dim;
    a.ld = ld;
    a.ld_codes = ld_codes;
    a.ld_scales = ld_scales;
    const dim3 grid = grid_of(tokens, dim);
    if (dt == DP_F32) hipLaunchKernelGGL((k_pack<DP_F32>), grid, dim3(kThreads), 0, stream, a);
    if (dt == DP_F16) hipLaunchKernelGGL((k_pack<DP_F16>), grid, dim3(kThreads), 0, stream, a);
    if (dt == DP_BF16) hipLaunchKernelGGL((k_pack<DP_BF16>), grid, dim3(kThreads), 0, stream, a);
    return hipGetLastError();
}

hipError_t launch_unpack(dp_dtype dt, int64_t tokens, int64_t dim, const void* codes, int64_t ld_codes,
                         const void* scales, int64_t ld_scales, void* x, int64_t ld, hipStream_t stream) {
    if (tokens == 0) return hipSuccess;
    PackArgs a{};
    a.codes_in = static_cast<const unsigned char*>(codes);
    a.scales_in = static_cast<const unsigned char*>(scales);
    a.out = x;
    a.tokens = tokens;
    a.dim = dim;
    a.ld = ld;
    a.ld_codes = ld_codes;
    a.ld_scales = ld_scales;
    const dim3 grid = grid_of(tokens, dim);
    if (dt == DP_F32) hipLaunchKernelGGL((k_unpack<DP_F32>), grid, dim3(kThreads), 0, stream, a);
    if (dt == DP_F16) hipLaunchKernelGGL((k_unpack<DP_F16>), grid, dim3(kThreads), 0, stream, a);
    if (dt == DP_BF16) hipLaunchKernelGGL((k_unpack<DP_BF16>), grid, dim3(kThreads), 0, stream, a);
    return hipGetLastError();
}

}  // namespace dpk

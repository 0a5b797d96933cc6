// Device helpers of the kernels that quantize fp32 values eight columns to a lane: a 1x128 tile is 16 lanes, one DPP row.
#pragma once
#include "ffn_math.h"

__device__ __forceinline__ void unpack8(uint4 v, float (&f)[8]) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int p = 0; p < 4; p++) {
        f[2 * p] = fg_bf16_lo(w[p]);
        f[2 * p + 1] = fg_bf16_hi(w[p]);
    }
}

__device__ __forceinline__ float absmax8(const float (&f)[8]) {
    float m = 0.0f;
#pragma unroll
    for (int e = 0; e < 8; e++) m = __builtin_fmaxf(m, __builtin_fabsf(f[e]));
    return m;
}

template <bool SMALL>
__device__ __forceinline__ uint2 quant8(const float (&f)[8], float s) {
    const fg_divisor d = fg_divisor_of(s);
    return make_uint2(fg_quant4<SMALL>(f[0], f[1], f[2], f[3], d), fg_quant4<SMALL>(f[4], f[5], f[6], f[7], d));
}

// Sum over the four lanes l % 16 + 16 i: each row swap leaves the two partners' values in its two results.
__device__ __forceinline__ float rows_sum(float v) {
    const auto a = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    const float m = __uint_as_float(a[0]) + __uint_as_float(a[1]);
    const auto b = __builtin_amdgcn_permlane32_swap(__float_as_uint(m), __float_as_uint(m), false, false);
    return __uint_as_float(b[0]) + __uint_as_float(b[1]);
}

// 16-byte slot of piece `piece` of column c in an LDS image [128 columns][128 rows] of codes: pieces are XORed with the
// column's chunk of eight, and column pairs are swapped for the upper chunks, so that the 64 dwords a wave writes at once
// lie in 64 banks.
__device__ __forceinline__ int t_slot(int c, int piece) { return ((c ^ ((c >> 6) & 1)) * 8 + (piece ^ ((c >> 3) & 7))); }

// Device helpers of the feed-forward operators: activation functions in fp32 and the quantization rule on
// fp32 values.
#pragma once
#include "common.h"
#include "fp8fg_ffn.h"

// 1 / (1 + exp(-z)) from the hardware's 2^x and reciprocal, each within one unit in the last place. The
// product z * log2(e) is rounded, which makes a relative error of |z| 2^-24 in exp(-z): below 2^-20 wherever
// the sigmoid differs from 0 and 1 by more than e^-16. exp(-z) overflows to infinity for z < -88 and the
// reciprocal is then 0, the limit.
__device__ __forceinline__ float fg_sigmoid(float z) {
    return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(z * -1.44269504f));
}

// GELU in its tanh form is z * sigmoid(2 u), u = sqrt(2 / pi) (z + 0.044715 z^3); the argument is computed
// from z clamped to +-32, where the sigmoid has long reached 0 or 1, so that its square stays finite.
__device__ __forceinline__ float fg_gelu_sigmoid(float z, float& z2) {
    const float c = __builtin_fminf(__builtin_fmaxf(z, -32.0f), 32.0f);
    z2 = c * c;
    return fg_sigmoid(c * __builtin_fmaf(z2, 0.0713548163f, 1.59576912f));   // 2 sqrt(2/pi) (1 + 0.044715 z^2)
}

template <int ACT>
__device__ __forceinline__ float fg_act_value(float z) {
    if constexpr (ACT == FG_ACT_RELU) return __builtin_elementwise_maximum(z, 0.0f);      // a NaN stays one
    if constexpr (ACT == FG_ACT_SILU) return z * fg_sigmoid(z);
    if constexpr (ACT == FG_ACT_GELU_TANH) {
        // without the clamp: where z^2 overflows, the sigmoid's argument is infinite and it 0 or 1 all the same.
        // The constants are those of fg_gelu_sigmoid times -log2(e).
        const float e = __builtin_amdgcn_exp2f(z * __builtin_fmaf(z * z, -0.102943242f, -2.30220819f));
        return z * __builtin_amdgcn_rcpf(1.0f + e);
    }
    return z;
}

// act(z) and act'(z) together. With k the sigmoid: silu' = k + a (1 - k), gelu' = k + a (1 - k) 2 u'. For
// z far below 0, a = z k is -0 and the slope 0; far above, 1 - k is 0 and the slope 1.
template <int ACT>
__device__ __forceinline__ void fg_act_both(float z, float& a, float& slope) {
    if constexpr (ACT == FG_ACT_RELU) {
        a = fg_act_value<FG_ACT_RELU>(z);
        slope = z <= 0.0f ? 0.0f : 1.0f;
    } else if constexpr (ACT == FG_ACT_SILU) {
        const float k = fg_sigmoid(z);
        a = z * k;
        slope = __builtin_fmaf(a, 1.0f - k, k);
    } else if constexpr (ACT == FG_ACT_GELU_TANH) {
        float z2;
        const float k = fg_gelu_sigmoid(z, z2);
        a = z * k;
        slope = __builtin_fmaf(a * (1.0f - k), __builtin_fmaf(z2, 0.214064449f, 1.59576912f), k);
    } else {
        a = z;
        slope = 1.0f;
    }
}

__device__ __forceinline__ float fg_act_any(int act, float z) {
    switch (act) {   // uniform over the launch
        case FG_ACT_RELU: return fg_act_value<FG_ACT_RELU>(z);
        case FG_ACT_GELU_TANH: return fg_act_value<FG_ACT_GELU_TANH>(z);
        case FG_ACT_SILU: return fg_act_value<FG_ACT_SILU>(z);
        default: return z;
    }
}

// Scales of N groups of fp32 values from their max-abs: as fg_scale_from_amax_bits, whose corrected product equals
// the correctly rounded amax / 448 while its remainder is exact; below 2^-80 (rare: one branch for all the groups) the
// division itself. A max-abs that overflowed counts as the largest finite one: the codes of the infinite values are
// then NaN (inf - inf in fg_quot_arg), and the scale stays a number. Call with the whole wave active.
template <int N>
__device__ __forceinline__ void fg_scales_from_amax(const float (&amax)[N], int pow2, float (&s)[N]) {
    const float c = 0x1.24924ap-9f;                     // RN(1/448)
    float least = amax[0];
#pragma unroll
    for (int i = 0; i < N; i++) {
        const float m = __builtin_fminf(amax[i], 0x1.fffffep127f), q0 = m * c;
        s[i] = __builtin_fmaf(__builtin_fmaf(-q0, 448.0f, m), c, q0);
        least = __builtin_fminf(least, amax[i]);
    }
    if (__builtin_amdgcn_ballot_w64(least < 0x1p-80f) != 0) {
#pragma unroll
        for (int i = 0; i < N; i++) {
            const float q = amax[i] / 448.0f;
            if (amax[i] < 0x1p-80f) s[i] = amax[i] == 0.0f ? 1.0f : q < 1.17549435e-38f ? 1.17549435e-38f : q;
        }
    }
    if (pow2) {
#pragma unroll
        for (int i = 0; i < N; i++) {
            const uint32_t u = __float_as_uint(s[i]);
            s[i] = __uint_as_float((u & 0x007FFFFFu) ? (u & 0x7F800000u) + 0x00800000u : u);
        }
    }
}
__device__ __forceinline__ float fg_scale_from_amax(float amax, int pow2) {
    const float m[1] = {amax};
    float s[1];
    fg_scales_from_amax(m, pow2, s);
    return s[0];
}

// The divisor of a group whose values are quantized from fp32: the reciprocal refined once is within a unit in the
// last place, and the corrected quotient (fg_quot_arg) is then off by at most 2^-22 of one before its rounding. A
// quotient that is a tie between two codes is exact, and a power-of-2 scale's too, so one form serves both modes.
// The remainder has up to 48 bits here: it is exact for scales from 2^-80 on (quotients that encode to a code other
// than 0 are at least 2^-10), and smaller scales are moved up by 2^64 with their values.
__device__ __forceinline__ fg_divisor fg_divisor_of(float s) {
    const float r = __builtin_amdgcn_rcpf(s);
    return fg_divisor{s, __builtin_fmaf(__builtin_fmaf(-s, r, 1.0f), r, r)};
}
__device__ __forceinline__ bool fg_small_scale(float s) { return s < 0x1p-80f; }

// Four fp32 values by the divisor of their group -> four E4M3 codes in a dword. SMALL: the scale may be below 2^-80.
template <bool SMALL>
__device__ __forceinline__ uint32_t fg_quant4(float a, float b, float c, float e, const fg_divisor& d) {
    const uint32_t q = fg_cvt2q<FG_Q_FAST, true>(c, e, d, fg_cvt2q<FG_Q_FAST, false>(a, b, d, 0));
    if constexpr (!SMALL) return q;
    const fg_divisor m = fg_divisor_shifted(d);
    const uint32_t t = fg_cvt2q<FG_Q_TINY, true>(c, e, m, fg_cvt2q<FG_Q_TINY, false>(a, b, m, 0));
    return fg_small_scale(d.s) ? t : q;
}
// `small` is uniform over the wave.
__device__ __forceinline__ uint32_t fg_quant4(float a, float b, float c, float e, const fg_divisor& d, bool small) {
    return small ? fg_quant4<true>(a, b, c, e, d) : fg_quant4<false>(a, b, c, e, d);
}
__device__ __forceinline__ bool fg_any_small(float s) { return __builtin_amdgcn_ballot_w64(fg_small_scale(s)) != 0; }

// Max across the 16 lanes of a DPP row, of values that are not negative: their bits order like them, and the integer
// max takes its DPP operand as it is (the float one would first quiet NaNs, an instruction more a step).
__device__ __forceinline__ float fg_row16_max(float f) {
    uint32_t v = __float_as_uint(f);
#define FG_STEP(ctrl)                                                                             \
    {                                                                                             \
        const uint32_t o = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, ctrl, 0xF, 0xF, false); \
        v = o > v ? o : v;                                                                        \
    }
    FG_STEP(0x128)
    FG_STEP(0x124)
    FG_STEP(0x4E)
    FG_STEP(0xB1)
#undef FG_STEP
    return __uint_as_float(v);
}

__device__ __forceinline__ uint32_t fg_bf16_bits(float f) { return (uint32_t)__builtin_bit_cast(unsigned short, (__bf16)f); }

// Element i of an array of f32 or bf16.
__device__ __forceinline__ float fg_load_elem(const void* p, int64_t i, int bf16) {
    return bf16 ? __uint_as_float((uint32_t)((const uint16_t*)p)[i] << 16) : ((const float*)p)[i];
}

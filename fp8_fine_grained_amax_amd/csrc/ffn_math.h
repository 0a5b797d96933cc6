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
    if constexpr (ACT == FG_ACT_RELU) return __builtin_fmaxf(z, 0.0f);
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
        a = __builtin_fmaxf(z, 0.0f);
        slope = z > 0.0f ? 1.0f : 0.0f;
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

// Scale of a group of fp32 values from their max-abs: as fg_scale_from_amax_bits, whose corrected product
// equals the correctly rounded amax / 448 while its remainder is exact; below 2^-80 the division itself.
__device__ __forceinline__ float fg_scale_from_amax(float amax, int pow2) {
    const float c = 0x1.24924ap-9f;                     // RN(1/448)
    const float q0 = amax * c;
    float s = __builtin_fmaf(__builtin_fmaf(-q0, 448.0f, amax), c, q0);
    if (amax < 0x1p-80f) s = amax / 448.0f;
    s = s < 1.17549435e-38f ? 1.17549435e-38f : s;
    if (pow2) {
        const uint32_t u = __float_as_uint(s);
        s = __uint_as_float((u & 0x007FFFFFu) ? (u & 0x7F800000u) + 0x00800000u : u);
    }
    return amax == 0.0f ? 1.0f : s;
}

// Quotient forms for fp32 values, as in common.h: the remainder of the corrected quotient has up to 48 bits
// here, so it is exact for scales from 2^-80 on (quotients that encode to a code other than 0 are at least
// 2^-10), and smaller scales are moved up by 2^64 with their values.
__device__ __forceinline__ bool fg_small_scale(float s) { return s < 0x1p-80f; }

// The form of a wave whose lanes hold the scales s: uniform. Call with the whole wave active.
__device__ __forceinline__ int fg_quot_form(float s, int pow2) {
    if (pow2) return FG_Q_POW2;
    return __builtin_amdgcn_ballot_w64(fg_small_scale(s)) == 0 ? FG_Q_FAST : FG_Q_TINY;
}

// Four fp32 values by the divisors of their groups -> four E4M3 codes in a dword. FORM is the wave's; under
// FG_Q_TINY each lane takes the form of its own scale.
template <int FORM>
__device__ __forceinline__ uint32_t fg_quant4(float a, float b, float c, float e, const fg_divisor& d) {
    if constexpr (FORM == FG_Q_TINY) {
        if (!fg_small_scale(d.s)) return fg_quant4<FG_Q_FAST>(a, b, c, e, d);
        const fg_divisor m = fg_divisor_shifted(d);
        return fg_cvt2q<FG_Q_TINY, true>(c, e, m, fg_cvt2q<FG_Q_TINY, false>(a, b, m, 0));
    } else {
        return fg_cvt2q<FORM, true>(c, e, d, fg_cvt2q<FORM, false>(a, b, d, 0));
    }
}
__device__ __forceinline__ uint32_t fg_quant4_any(int form, float a, float b, float c, float e, const fg_divisor& d) {
    if (form == FG_Q_POW2) return fg_quant4<FG_Q_POW2>(a, b, c, e, d);
    if (form == FG_Q_FAST) return fg_quant4<FG_Q_FAST>(a, b, c, e, d);
    return fg_quant4<FG_Q_TINY>(a, b, c, e, d);
}

// Max across the 16 lanes of a DPP row.
__device__ __forceinline__ float fg_row16_max(float v) {
#define FG_STEP(ctrl) v = __builtin_fmaxf(v, __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), ctrl, 0xF, 0xF, false)))
    FG_STEP(0x128);
    FG_STEP(0x124);
    FG_STEP(0x4E);
    FG_STEP(0xB1);
#undef FG_STEP
    return v;
}

__device__ __forceinline__ uint32_t fg_bf16_bits(float f) { return (uint32_t)__builtin_bit_cast(unsigned short, (__bf16)f); }

// Element i of an array of f32 or bf16.
__device__ __forceinline__ float fg_load_elem(const void* p, int64_t i, int bf16) {
    return bf16 ? __uint_as_float((uint32_t)((const uint16_t*)p)[i] << 16) : ((const float*)p)[i];
}

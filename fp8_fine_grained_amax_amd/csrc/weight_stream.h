// Weight streaming for products with few tokens (gfx950), shared by the Linear of few rows and the mixture of experts.
//
// With few tokens a product reads its weights once and does little with them: it is bound by the rate at which
// weight codes stream from HBM, not by the matrix cores. So no tile is staged in LDS: a wave keeps 16-row weight
// tiles of one 128-deep K block as MFMA operands in registers, loads them a few K blocks ahead, and the waves
// of a workgroup split the contraction and join their sums through LDS in a fixed order. An MFMA takes weight
// rows as its first operand and tokens as its second, so lane l ends with token l % 16 and four consecutive
// weight rows.
//
// Loads and operands: an MFMA operand has row l % 16 and the bytes [16 g, 16 g + 16) and [64 + 16 g, + 16) of its 128,
// g = l / 16, in lane l. Loaded like that, every lane of a quad reads another row, which a compute unit serves at a
// third of its rate (L2-resident rows: 9.4 TB/s over the card, against 29 with quads that read 64 contiguous
// bytes; from HBM 3.9 to 5.2 against 5.1 to 5.8). So lane l loads row l / 4 and the bytes of g = l % 4, and the
// registers are turned to operands by an exchange over the LDS crossbar (ds_bpermute, eight an operand).
#pragma once
#include "ffn_math.h"

namespace {

enum { SRC_BF16 = 0, SRC_F32 = 1, SRC_ROWS = 2, SRC_OPERAND = 3 };   // values to quantize; codes in rows; codes as operands
constexpr int BK = FG_GROUP;

// A lane's place in a load of a 16-row tile, and the byte address (4 x lane) that an operand lane takes its bytes from.
__device__ __forceinline__ int load_row(int lane) { return lane >> 2; }
__device__ __forceinline__ int load_group(int lane) { return lane & 3; }
__device__ __forceinline__ int operand_source(int lane) { return 4 * (4 * (lane & 15) + (lane >> 4)); }

__device__ __forceinline__ v8i to_operand(const v4i& lo, const v4i& hi, int source) {
    v8i r;
#pragma unroll
    for (int i = 0; i < 4; i++) {
        r[i] = __builtin_amdgcn_ds_bpermute(source, lo[i]);
        r[4 + i] = __builtin_amdgcn_ds_bpermute(source, hi[i]);
    }
    return r;
}

// Hidden values in the workspace: the 32 values of each lane group g of a row's 128 are eight fours, and four j of
// all groups lie next to each other, so that the loads of a quad are contiguous there too. Position of the four
// that begins at k (a multiple of 4).
__device__ __forceinline__ int hidden_at(int k) { return ((k >> 6) * 4 + ((k >> 2) & 3)) * 16 + ((k >> 4) & 3) * 4; }

// One token tile of one K block as it is loaded: this lane's 32 values of its row's 128. `row` is the load row's.
template <int SRC>
struct ActRegs;
template <>
struct ActRegs<SRC_BF16> {
    uint4 v[4];
    __device__ __forceinline__ void load(const uint16_t* row, int64_t k, int lane) {
        const uint16_t* p = row + k + 16 * load_group(lane);
#pragma unroll
        for (int i = 0; i < 4; i++) v[i] = *reinterpret_cast<const uint4*>(p + (i >> 1) * 64 + (i & 1) * 8);
    }
    __device__ __forceinline__ void get(float (&f)[32]) const {
#pragma unroll
        for (int i = 0; i < 4; i++) {
            const uint32_t w[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
#pragma unroll
            for (int j = 0; j < 4; j++) {
                f[8 * i + 2 * j] = fg_bf16_lo(w[j]);
                f[8 * i + 2 * j + 1] = fg_bf16_hi(w[j]);
            }
        }
    }
};
template <>
struct ActRegs<SRC_F32> {
    v4f v[8];
    __device__ __forceinline__ void load(const float* row, int64_t k, int lane) {
        const float* p = row + k + 4 * load_group(lane);
#pragma unroll
        for (int i = 0; i < 8; i++) v[i] = *reinterpret_cast<const v4f*>(p + 16 * i);
    }
    __device__ __forceinline__ void get(float (&f)[32]) const {
#pragma unroll
        for (int i = 0; i < 32; i++) f[i] = v[i >> 2][i & 3];
    }
};
template <>
struct ActRegs<SRC_ROWS> {
    v4i lo, hi;
    float s;          // of the operand's row
    __device__ __forceinline__ void load(const uint8_t* row, const float* scale, int64_t k, int lane) {
        const uint8_t* p = row + k + 16 * load_group(lane);
        lo = *reinterpret_cast<const v4i*>(p);
        hi = *reinterpret_cast<const v4i*>(p + 64);
        s = *scale;
    }
};

// Codes that this library laid out as operands: a tile's block is 2 KB, the first halves of all lanes and then the
// second ones, and its 16 scales.
template <>
struct ActRegs<SRC_OPERAND> {
    v4i lo, hi;
    float s;
    __device__ __forceinline__ void load(const uint8_t* codes, const float* scales, int64_t block, int lane) {
        const uint8_t* p = codes + block * 2048 + 16 * lane;
        lo = *reinterpret_cast<const v4i*>(p);
        hi = *reinterpret_cast<const v4i*>(p + 1024);
        s = scales[block * 16 + (lane & 15)];
    }
};
// Where the codes k .. k + 7 (k a multiple of 8) of a tile's row go in its block.
__device__ __forceinline__ int operand_at(int row, int k) {
    const int c = k >> 4;
    return (c >> 2) * 1024 + (row + 16 * (c & 3)) * 16 + (k & 8);
}

// Max over the quad that holds one row (quad_perm [1,0,3,2], [2,3,0,1]).
__device__ __forceinline__ float quad_max(float v) {
    v = __builtin_fmaxf(v, __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), 0xB1, 0xF, 0xF, false)));
    return __builtin_fmaxf(v, __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), 0x4E, 0xF, 0xF, false)));
}

// The MFMA operand of a token tile and the scale of the lane's operand row; fp32 and bf16 values are quantized
// 1x128 here, as loaded.
template <int SRC>
__device__ __forceinline__ v8i act_operand(const ActRegs<SRC>& r, int pow2, int source, float& s) {
    if constexpr (SRC == SRC_OPERAND) {
        s = r.s;
        return v8i{r.lo.x, r.lo.y, r.lo.z, r.lo.w, r.hi.x, r.hi.y, r.hi.z, r.hi.w};
    } else if constexpr (SRC == SRC_ROWS) {
        s = r.s;
        return to_operand(r.lo, r.hi, source);
    } else {
        float f[32];
        r.get(f);
        float m = 0.0f;
#pragma unroll
        for (int i = 0; i < 32; i++) m = __builtin_fmaxf(m, __builtin_fabsf(f[i]));
        const float own = fg_scale_from_amax(quad_max(m), pow2);
        const fg_divisor d = fg_divisor_of(own);
        const bool small = fg_any_small(own);
        v4i c[2];
        if (!small) {
#pragma unroll
            for (int i = 0; i < 8; i++) c[i >> 2][i & 3] = (int)fg_quant4<false>(f[4 * i], f[4 * i + 1], f[4 * i + 2], f[4 * i + 3], d);
        } else {
#pragma unroll
            for (int i = 0; i < 8; i++) c[i >> 2][i & 3] = (int)fg_quant4<true>(f[4 * i], f[4 * i + 1], f[4 * i + 2], f[4 * i + 3], d);
        }
        s = __int_as_float(__builtin_amdgcn_ds_bpermute(source, __float_as_int(own)));
        return to_operand(c[0], c[1], source);
    }
}

// One K block as loaded: RT weight tiles of 16 rows, their block scales (RT / SG tiles share one) and NT token
// tiles.
template <int RT, int SG, int NT, int SRC>
struct StepRegs {
    v4i w[RT][2];
    float ws[SG];
    ActRegs<SRC> x[NT];
};

// Not a non-temporal load: the two halves of a line come from two instructions, and only a cached line is fetched once.
__device__ __forceinline__ v4i load_weight(const uint8_t* p) { return *reinterpret_cast<const v4i*>(p); }

typedef __bf16 v2bf __attribute__((ext_vector_type(2)));
typedef __bf16 v8bf __attribute__((ext_vector_type(8)));

// A lane's 32 codes as the bf16 values they stand for (exact), for four 32-deep bf16 MFMAs.
struct WideOperand {
    v8bf v[4];
    __device__ __forceinline__ explicit WideOperand(const v8i& q) {
#pragma unroll
        for (int i = 0; i < 8; i++) {
            const v2bf lo = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(q[i], 1.0f, false);
            const v2bf hi = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(q[i], 1.0f, true);
            v[i >> 1][4 * (i & 1)] = lo[0];
            v[i >> 1][4 * (i & 1) + 1] = lo[1];
            v[i >> 1][4 * (i & 1) + 2] = hi[0];
            v[i >> 1][4 * (i & 1) + 3] = hi[1];
        }
    }
};

// acc += sW sX P_b for every tile of a step; `tiles` has a bit for each token tile that holds a token in use.
// EXACT: P_b by bf16 MFMAs. The FP8 MFMAs align the 32 products of a chunk and cut off what falls below, 1.5e-5 of
// the block's sum; that moves about one in 2000 of the values that are quantized next over a border between two
// codes (a mixture's output 2.7e-3 off instead of the 1.7e-3 of its own rounding). The bf16 ones sum exactly to fp32
// (1e-8), and the matrix cores have the time: 0.2 of a weight stream's.
template <int RT, int SG, int NT, int SRC, bool EXACT>
__device__ __forceinline__ void consume(const StepRegs<RT, SG, NT, SRC>& b, int pow2, int tiles, int source,
                                        v4f (&acc)[RT][NT]) {
    v8i w[RT];
#pragma unroll
    for (int r = 0; r < RT; r++) w[r] = to_operand(b.w[r][0], b.w[r][1], source);
    if constexpr (EXACT) {
        v8i x[NT];
        float s[NT];
#pragma unroll
        for (int t = 0; t < NT; t++) x[t] = act_operand<SRC>(b.x[t], pow2, source, s[t]);
#pragma unroll
        for (int r = 0; r < RT; r++) {
            const WideOperand wr(w[r]);
#pragma unroll
            for (int t = 0; t < NT; t++) {
                if (NT > 1 && !((tiles >> t) & 1)) continue;
                const WideOperand xt(x[t]);
                v4f part = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int i = 0; i < 4; i++) part = __builtin_amdgcn_mfma_f32_16x16x32_bf16(wr.v[i], xt.v[i], part, 0, 0, 0);
                const float f = s[t] * b.ws[r * SG / RT];
#pragma unroll
                for (int q = 0; q < 4; q++) acc[r][t][q] = __builtin_fmaf(part[q], f, acc[r][t][q]);
            }
        }
    } else {
#pragma unroll
        for (int t = 0; t < NT; t++) {
            if (NT > 1 && !((tiles >> t) & 1)) continue;
            float s;
            const v8i x = act_operand<SRC>(b.x[t], pow2, source, s);
#pragma unroll
            for (int r = 0; r < RT; r++) {
                const v4f part = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(w[r], x, v4f{0.f, 0.f, 0.f, 0.f}, 0, 0, 0, 127, 0, 127);
                const float f = s * b.ws[r * SG / RT];
#pragma unroll
                for (int q = 0; q < 4; q++) acc[r][t][q] = __builtin_fmaf(part[q], f, acc[r][t][q]);
            }
        }
    }
}

// A zero that the compiler takes for a lane's own value: a load at a uniform address plus this stays a vector
// load, whose wait counts only the loads before it. (Scalar loads return out of order, so waiting for one waits
// for all that were issued ahead.)
__device__ __forceinline__ int lane_zero() {
    int z = 0;
    asm("" : "+v"(z));
    return z;
}

// Runs steps [k0, k1) with DEPTH steps' loads in flight. load(buffer) loads the next step (and, past the end, the
// last one again: every pass of the loop issues the same loads, so that the waits can count them); use(buffer)
// is called for the steps in order.
template <int DEPTH, class Regs, class Load, class Use>
__device__ __forceinline__ void stream_steps(int k0, int k1, Load&& load, Use&& use) {
    Regs buf[DEPTH];
    if (k0 >= k1) return;
    // The order of the loads is kept by scheduling fences: a wait for one counts the ones behind it.
#pragma unroll
    for (int i = 0; i < DEPTH; i++) {
        load(buf[i]);
        __builtin_amdgcn_sched_barrier(0);
    }
    for (int k = k0; k < k1; k += DEPTH) {
#pragma unroll
        for (int i = 0; i < DEPTH; i++) {
            if (k + i < k1) use(buf[i]);
            __builtin_amdgcn_sched_barrier(0);
            load(buf[i]);
            __builtin_amdgcn_sched_barrier(0);
        }
    }
}

}  // namespace

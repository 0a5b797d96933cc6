// Activation functions whose input is kept as an FP8 checkpoint, and their backward pass from it (gfx950).
//
// Both kernels are elementwise with maxima over tiles: HBM-bound by their bytes, and close to it by their
// VALU work (three to five quantizations of every element besides the activation), so every tensor is read
// and written once and the values stay in registers between the maxima and the codes.
#include "ffn_launch.h"
#include "ffn_math.h"
#include "host_util.h"

namespace {

template <int ACT>
struct ActTag {
    static constexpr int value = ACT;
};

template <class Fn>
hipError_t by_act(int act, Fn&& fn) {
    switch (act) {
        case FG_ACT_RELU: return fn(ActTag<FG_ACT_RELU>{});
        case FG_ACT_GELU_TANH: return fn(ActTag<FG_ACT_GELU_TANH>{});
        case FG_ACT_SILU: return fn(ActTag<FG_ACT_SILU>{});
        default: return fn(ActTag<FG_ACT_NONE>{});
    }
}

__device__ __forceinline__ void unpack8(uint4 v, float (&f)[8]) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int p = 0; p < 4; p++) {
        f[2 * p] = fg_bf16_lo(w[p]);
        f[2 * p + 1] = fg_bf16_hi(w[p]);
    }
}

__device__ __forceinline__ uint32_t absmax8_bits(uint4 v) {
    return fg_pk_max_u16(fg_pk_max_u16(v.x & 0x7FFF7FFFu, v.y & 0x7FFF7FFFu),
                         fg_pk_max_u16(v.z & 0x7FFF7FFFu, v.w & 0x7FFF7FFFu));
}

__device__ __forceinline__ float absmax8(const float (&f)[8]) {
    float m = 0.0f;
#pragma unroll
    for (int e = 0; e < 8; e++) m = __builtin_fmaxf(m, __builtin_fabsf(f[e]));
    return m;
}

__device__ __forceinline__ uint2 quant8(const float (&f)[8], float s, int pow2) {
    const fg_divisor d = fg_make_divisor(s, pow2);
    const int form = fg_quot_form(s, pow2);
    return make_uint2(fg_quant4_any(form, f[0], f[1], f[2], f[3], d), fg_quant4_any(form, f[4], f[5], f[6], f[7], d));
}

// ------------------------------------------------------------------------------------------------
// Forward. As in the 1x128 quantizer: a tile of z is 256 B = 16 lanes x 16 B, one DPP row, and a 256-thread
// workgroup covers 16 rows of one 128-column group per slot. The checkpoint's codes come from the bf16 bits
// of z (bit for bit the quantizer's), a from the same registers.
// ------------------------------------------------------------------------------------------------
template <int ACT, bool GATED, int UNROLL>
__global__ __launch_bounds__(256) void fg_act_fwd_kernel(const uint16_t* __restrict__ z, int64_t rows, int64_t F,
                                                         int64_t ld, int pow2, uint8_t* __restrict__ zq,
                                                         float* __restrict__ sz, uint8_t* __restrict__ aq,
                                                         float* __restrict__ sa) {
    constexpr int Z = GATED ? 2 : 1;
    const int lane16 = threadIdx.x & 15, slot = threadIdx.x >> 4;
    const uint32_t ng = (uint32_t)(F / FG_GROUP);
    const int64_t g = blockIdx.x % ng;
    const int64_t r_base = (int64_t)(blockIdx.x / ng) * (16 * UNROLL) + slot;
    const int64_t col = g * FG_GROUP + lane16 * 8;

    uint4 v[UNROLL][Z];
#pragma unroll
    for (int u = 0; u < UNROLL; u++) {
        const int64_t r = r_base + 16 * u;
#pragma unroll
        for (int h = 0; h < Z; h++)
            v[u][h] = r < rows ? *reinterpret_cast<const uint4*>(z + r * ld + h * F + col) : make_uint4(0, 0, 0, 0);
    }
#pragma unroll
    for (int u = 0; u < UNROLL; u++) {
        const int64_t r = r_base + 16 * u;
        uint2 zc[Z];
        float zs[Z];
#pragma unroll
        for (int h = 0; h < Z; h++) {
            zs[h] = fg_scale_from_amax_bits(fg_max_halves(fg_row16_max_pk(absmax8_bits(v[u][h]))), pow2);
            zc[h] = fg_quant8_any(v[u][h], fg_make_divisor(zs[h], pow2), pow2);
        }
        float a[8];
        unpack8(v[u][0], a);
#pragma unroll
        for (int e = 0; e < 8; e++) a[e] = fg_act_value<ACT>(a[e]);
        if constexpr (GATED) {
            float up[8];
            unpack8(v[u][1], up);
#pragma unroll
            for (int e = 0; e < 8; e++) a[e] *= up[e];
        }
        const float as = fg_scale_from_amax(fg_row16_max(absmax8(a)), pow2);
        const uint2 ac = quant8(a, as, pow2);
        if (r < rows) {
#pragma unroll
            for (int h = 0; h < Z; h++) *reinterpret_cast<uint2*>(zq + r * (Z * F) + h * F + col) = zc[h];
            *reinterpret_cast<uint2*>(aq + r * F + col) = ac;
            if (lane16 == 0) {
#pragma unroll
                for (int h = 0; h < Z; h++) sz[(h * (int64_t)ng + g) * rows + r] = zs[h];
                sa[g * rows + r] = as;
            }
        }
    }
}

// ------------------------------------------------------------------------------------------------
// Backward. A 512-thread workgroup owns 128 rows x 128 columns of da: thread t holds rows 4 (t / 16) + i
// (i = 0..3) of the 8-column chunk t % 16, so a DPP row of 16 lanes holds a whole 1x128 tile (its maximum
// takes four DPP steps), and a column's maximum is 4 registers, two lane exchanges and an 8-wave exchange
// through LDS. The codes along the columns leave at once, 128 contiguous bytes a row; those along the rows go
// through an LDS image [128 columns][128 rows], whose 16 B pieces are XORed with the column's chunk and whose
// column pairs are swapped for the upper chunks, so that the 64 dwords a wave writes at once lie in 64 banks.
// dz and a are computed once and stay in registers (up to 96 a thread) for the maxima and both codes.
// ------------------------------------------------------------------------------------------------
constexpr int kBwdThreads = 512, kBwdWaves = kBwdThreads / 64;

// Physical column and piece of the transposed image.
__device__ __forceinline__ int t_slot(int c, int piece) { return ((c ^ ((c >> 6) & 1)) * 8 + (piece ^ ((c >> 3) & 7))); }

template <int ACT, bool GATED>
__global__ __launch_bounds__(kBwdThreads) void fg_act_bwd_kernel(FgActBwd p) {
    constexpr int Z = GATED ? 2 : 1;            // halves of dz
    constexpr int V = Z + 1;                    // values with column tiles: dz, a
    extern __shared__ __attribute__((aligned(16))) uint8_t smem[];
    uint4* image = reinterpret_cast<uint4*>(smem);                              // [V][128 * 8]
    float* colmax = reinterpret_cast<float*>(smem + V * 16384);                 // [V][kBwdWaves][128]
    float* colsum = colmax + V * kBwdWaves * 128;                               // [Z][kBwdWaves][128]
    float* col_s = colsum + Z * kBwdWaves * 128;                                // [V][128] scales, then reciprocals
    float* col_r = col_s + V * 128;
    __shared__ int small_w[8];                  // per wave of the column scales: one below 2^-80

    const int t = threadIdx.x, lane = t & 63, wave = t >> 6;
    const int chunk = t & 15, rgrp = t >> 4;
    const int64_t F = p.F, W = Z * F, rows = p.rows;
    const int64_t row_blocks = (rows + FG_GROUP - 1) / FG_GROUP;
    const int64_t br = blockIdx.x % row_blocks, g = blockIdx.x / row_blocks;
    const int64_t r0 = br * FG_GROUP + 4 * rgrp;
    const int64_t col = g * FG_GROUP + chunk * 8;
    const int64_t gstep = F / FG_GROUP;

    float dz[Z][4][8], a[4][8];
    uint2 zc[4][Z];
    float zs[4][Z];
    uint4 d0[4], d1[4];
#pragma unroll
    for (int i = 0; i < 4; i++) {
        const int64_t r = r0 + i;
        const bool ok = r < rows;
#pragma unroll
        for (int h = 0; h < Z; h++) {
            zc[i][h] = ok ? *reinterpret_cast<const uint2*>(p.zq + r * W + h * F + col) : make_uint2(0, 0);
            zs[i][h] = ok ? p.sz[(h * gstep + g) * rows + r] : 0.0f;
        }
        if (p.da_bf16) {
            d0[i] = ok ? *reinterpret_cast<const uint4*>((const uint16_t*)p.da + r * p.ld_da + col) : make_uint4(0, 0, 0, 0);
        } else {
            const float* d = (const float*)p.da + r * p.ld_da + col;
            d0[i] = ok ? *reinterpret_cast<const uint4*>(d) : make_uint4(0, 0, 0, 0);
            d1[i] = ok ? *reinterpret_cast<const uint4*>(d + 4) : make_uint4(0, 0, 0, 0);
        }
    }
#pragma unroll
    for (int i = 0; i < 4; i++) {
        float da[8], zv[Z][8];
        if (p.da_bf16) {
            unpack8(d0[i], da);
        } else {
            const uint32_t w[8] = {d0[i].x, d0[i].y, d0[i].z, d0[i].w, d1[i].x, d1[i].y, d1[i].z, d1[i].w};
#pragma unroll
            for (int e = 0; e < 8; e++) da[e] = __uint_as_float(w[e]);
        }
#pragma unroll
        for (int h = 0; h < Z; h++) {
            const auto f0 = __builtin_amdgcn_cvt_pk_f32_fp8((int)zc[i][h].x, false), f1 = __builtin_amdgcn_cvt_pk_f32_fp8((int)zc[i][h].x, true);
            const auto f2 = __builtin_amdgcn_cvt_pk_f32_fp8((int)zc[i][h].y, false), f3 = __builtin_amdgcn_cvt_pk_f32_fp8((int)zc[i][h].y, true);
            const float f[8] = {f0[0], f0[1], f1[0], f1[1], f2[0], f2[1], f3[0], f3[1]};
#pragma unroll
            for (int e = 0; e < 8; e++) zv[h][e] = f[e] * zs[i][h];
        }
#pragma unroll
        for (int e = 0; e < 8; e++) {
            float act, slope;
            fg_act_both<ACT>(zv[0][e], act, slope);
            if constexpr (GATED) {
                dz[0][i][e] = da[e] * zv[1][e] * slope;
                dz[1][i][e] = da[e] * act;
                a[i][e] = act * zv[1][e];
            } else {
                dz[0][i][e] = da[e] * slope;
                a[i][e] = act;
            }
        }
    }

    // tiles along the columns
#pragma unroll
    for (int h = 0; h < Z; h++) {
        float s_row[4];
#pragma unroll
        for (int i = 0; i < 4; i++) {
            s_row[i] = fg_scale_from_amax(fg_row16_max(absmax8(dz[h][i])), p.pow2);
            const uint2 c = quant8(dz[h][i], s_row[i], p.pow2);
            if (r0 + i < rows) *reinterpret_cast<uint2*>(p.dzq_cols + (r0 + i) * W + h * F + col) = c;
        }
#pragma unroll
        for (int i = 0; i < 4; i++)
            if (chunk == i && r0 + i < rows) p.sdz_cols[(h * gstep + g) * rows + r0 + i] = s_row[i];
    }

    // column maxima and sums of this wave's 16 rows
    const bool want_dz = p.dzq_rows != nullptr, want_a = p.aq_rows != nullptr, want_b = p.dbias != nullptr;
    if (!want_dz && !want_a && !want_b) return;
#pragma unroll
    for (int v = 0; v < V; v++) {
        if (v < Z ? !want_dz : !want_a) continue;
#pragma unroll
        for (int e = 0; e < 8; e++) {
            float m = 0.0f;
#pragma unroll
            for (int i = 0; i < 4; i++) m = __builtin_fmaxf(m, __builtin_fabsf(v < Z ? dz[v < Z ? v : 0][i][e] : a[i][e]));
            m = __builtin_fmaxf(m, __shfl_xor(m, 16));
            m = __builtin_fmaxf(m, __shfl_xor(m, 32));
            if (lane < 16) colmax[(v * kBwdWaves + wave) * 128 + chunk * 8 + e] = m;
        }
    }
    if (want_b) {
#pragma unroll
        for (int h = 0; h < Z; h++)
#pragma unroll
            for (int e = 0; e < 8; e++) {
                float s = (dz[h][0][e] + dz[h][1][e]) + (dz[h][2][e] + dz[h][3][e]);
                s += __shfl_xor(s, 16);
                s += __shfl_xor(s, 32);
                if (lane < 16) colsum[(h * kBwdWaves + wave) * 128 + chunk * 8 + e] = s;
            }
    }
    __syncthreads();
    if (want_b && t < Z * 128) {
        const int h = t >> 7, c = t & 127;
        float s = 0.0f;
#pragma unroll
        for (int w = 0; w < kBwdWaves; w++) s += colsum[(h * kBwdWaves + w) * 128 + c];
        float* out = row_blocks == 1 ? p.dbias : p.partial + br * W;
        out[h * F + g * FG_GROUP + c] = s;
    }
    if (!want_dz && !want_a) return;
    // one scale and reciprocal per column
    if (t < V * 128) {
        const int v = t >> 7, c = t & 127;
        if (v < Z ? want_dz : want_a) {
            float m = 0.0f;
#pragma unroll
            for (int w = 0; w < kBwdWaves; w++) m = __builtin_fmaxf(m, colmax[(v * kBwdWaves + w) * 128 + c]);
            const float s = fg_scale_from_amax(m, p.pow2);
            const fg_divisor d = fg_make_divisor(s, p.pow2);
            col_s[t] = d.s;
            col_r[t] = d.r;
            const uint64_t small = __builtin_amdgcn_ballot_w64(fg_small_scale(s));
            if (lane == 0) small_w[wave] = small != 0;
            if (v < Z) p.sdz_rows[br * W + v * F + g * FG_GROUP + c] = s;
            else p.sa_rows[br * F + g * FG_GROUP + c] = s;
        }
    }
    __syncthreads();
#pragma unroll
    for (int v = 0; v < V; v++) {
        if (v < Z ? !want_dz : !want_a) continue;
        const int form = p.pow2 ? FG_Q_POW2 : (small_w[2 * v] | small_w[2 * v + 1]) ? FG_Q_TINY : FG_Q_FAST;
        uint32_t* img = reinterpret_cast<uint32_t*>(image + v * 1024);
#pragma unroll
        for (int e = 0; e < 8; e++) {
            const int c = chunk * 8 + e;
            const fg_divisor d{col_s[v * 128 + c], col_r[v * 128 + c]};
            float f[4];
#pragma unroll
            for (int i = 0; i < 4; i++) f[i] = v < Z ? dz[v < Z ? v : 0][i][e] : a[i][e];
            img[t_slot(c, rgrp >> 2) * 4 + (rgrp & 3)] = fg_quant4_any(form, f[0], f[1], f[2], f[3], d);
        }
    }
    __syncthreads();
#pragma unroll
    for (int v = 0; v < V; v++) {
        if (v < Z ? !want_dz : !want_a) continue;
        uint8_t* out = v < Z ? p.dzq_rows + v * F * rows : p.aq_rows;
#pragma unroll
        for (int k = 0; k < 1024 / kBwdThreads; k++) {
            const int id = t + kBwdThreads * k, c = id >> 3, piece = id & 7;
            *reinterpret_cast<uint4*>(out + (g * FG_GROUP + c) * rows + br * FG_GROUP + 16 * piece) =
                image[v * 1024 + t_slot(c, piece)];
        }
    }
}

// Sum of the row blocks' partial bias gradients: 64 columns a workgroup, the blocks dealt to 4 waves in turn
// and the waves' sums added in order.
__global__ __launch_bounds__(256) void fg_bias_sum_kernel(const float* __restrict__ partial, int64_t blocks, int64_t W,
                                                          float* __restrict__ dbias) {
    __shared__ float sums[4][64];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int64_t c = (int64_t)blockIdx.x * 64 + lane;
    float s = 0.0f;
    for (int64_t b = wave; b < blocks; b += 4) s += partial[b * W + c];
    sums[wave][lane] = s;
    __syncthreads();
    if (wave == 0) dbias[c] = (sums[0][lane] + sums[1][lane]) + (sums[2][lane] + sums[3][lane]);
}

template <int ACT, bool GATED>
hipError_t launch_bwd(const FgActBwd& p, unsigned grid, hipStream_t stream) {
    constexpr int Z = GATED ? 2 : 1, V = Z + 1;
    constexpr int bytes = V * 16384 + (V + Z) * kBwdWaves * 128 * 4 + 2 * V * 128 * 4;
    auto kern = fg_act_bwd_kernel<ACT, GATED>;
    static std::atomic<uint64_t> lds_limit_set{0};
    const hipError_t e = fg_set_lds_limit_once((const void*)kern, bytes, lds_limit_set);
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(kern, dim3(grid), dim3(kBwdThreads), bytes, stream, p);
    return hipGetLastError();
}

}  // namespace

hipError_t fg_launch_act_fwd(const uint16_t* z, int64_t rows, int64_t F, int64_t ld, int act, int gated, int pow2,
                             uint8_t* zq, float* sz, uint8_t* aq, float* sa, hipStream_t stream) {
    constexpr int UNROLL = 2;
    const unsigned grid = (unsigned)((F / FG_GROUP) * ((rows + 16 * UNROLL - 1) / (16 * UNROLL)));
    return by_act(act, [&](auto tag) {
        constexpr int ACT = decltype(tag)::value;
        if (gated)
            hipLaunchKernelGGL((fg_act_fwd_kernel<ACT, true, UNROLL>), dim3(grid), dim3(256), 0, stream, z, rows, F, ld,
                               pow2, zq, sz, aq, sa);
        else
            hipLaunchKernelGGL((fg_act_fwd_kernel<ACT, false, UNROLL>), dim3(grid), dim3(256), 0, stream, z, rows, F, ld,
                               pow2, zq, sz, aq, sa);
        return hipGetLastError();
    });
}

// Rows of the bias gradient's partial sums: one per 128 rows, none where a single block writes the result.
int64_t fg_act_bwd_partial_rows(int64_t rows) {
    const int64_t blocks = (rows + FG_GROUP - 1) / FG_GROUP;
    return blocks > 1 ? blocks : 0;
}

hipError_t fg_launch_act_bwd(const FgActBwd& p, hipStream_t stream) {
    const int64_t blocks = (p.rows + FG_GROUP - 1) / FG_GROUP, W = (p.gated ? 2 : 1) * p.F;
    if (blocks > 0) {
        const unsigned grid = (unsigned)(blocks * (p.F / FG_GROUP));
        const hipError_t e = by_act(p.act, [&](auto tag) {
            constexpr int ACT = decltype(tag)::value;
            return p.gated ? launch_bwd<ACT, true>(p, grid, stream) : launch_bwd<ACT, false>(p, grid, stream);
        });
        if (e != hipSuccess) return e;
    }
    if (p.dbias && blocks != 1) {   // no rows: sums of nothing
        hipLaunchKernelGGL(fg_bias_sum_kernel, dim3((unsigned)(W / 64)), dim3(256), 0, stream, p.partial, blocks, W, p.dbias);
        return hipGetLastError();
    }
    return hipSuccess;
}

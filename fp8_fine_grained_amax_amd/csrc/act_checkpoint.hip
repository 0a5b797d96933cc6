// Activation functions whose input is kept as an FP8 checkpoint, and their backward pass from it (gfx950).
//
// Both kernels are elementwise with maxima over tiles: HBM-bound by their bytes, and close to it by their
// VALU work (three to five quantizations of every element besides the activation), so every tensor is read
// and written once and the values stay in registers between the maxima and the codes.
#include "ffn_launch.h"
#include "ffn_math.h"
#include "host_util.h"

#include <algorithm>
#include <type_traits>

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

// ------------------------------------------------------------------------------------------------
// Forward. As in the 1x128 quantizer: a tile of z is 256 B = 16 lanes x 16 B, one DPP row, and a 256-thread
// workgroup covers 16 rows of one 128-column group per slot. The checkpoint's codes come from the bf16 bits
// of z (bit for bit the quantizer's), a from the same registers. Bound by HBM: 4096 rows, F = 18432, gated SiLU, 102.5 us
// for 536 MB (5.2 TB/s; a copy of 2 GiB runs at 4.7). Two slots a thread keep 64 bytes of gated loads in flight. 7 rows of
// F = 2048 take 4.0 us, all latency.
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
        const uint2 ac = fg_any_small(as) ? quant8<true>(a, as) : quant8<false>(a, as);
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
// takes four DPP steps); a column's maximum is 4 registers, then the 32 row groups' through LDS. The codes along the
// columns leave at once, 128 contiguous bytes a row; those along the rows go through an LDS image [128 columns][128
// rows] (in the place of the maxima), whose 16 B pieces are XORed with the column's chunk and whose column pairs are
// swapped for the upper chunks, so that the 64 dwords a wave writes at once lie in 64 banks.
//
// dz and a are computed once and stay in registers (96 a thread when gated) for the maxima and both codes. The work is
// bound by the VALU as much as by HBM (about 70 operations an element of da when gated, 13 of them the activation's and
// 18 the five quotients'), so the two have to overlap: a gated launch's one workgroup a CU loads its next tile's inputs
// while it quantizes this one; the others leave registers enough for a second workgroup.
// Addresses are a wave-uniform base and a 32-bit lane offset (the host bounds widths and strides for it).
// Measured: gated SiLU, 4096 x 18432, FP32 da, every output but the bias gradient: 195 us for 847 MB (4.3 TB/s; 326 without
// the tile ahead, with the maxima in DPP steps across rows and 64-bit offsets); GELU, 8192 x 7168, bf16 da, every output:
// 83 to 86 us with the sum below for 360 MB. One tile alone takes 7.3 us with every output (2.9 for the identity and the
// column codes), 16 of them 8.2 to 9.1: with few tiles the time is a workgroup's own work. A gated launch's 257th tile is
// a second one for its CU: 256 tiles 14.6 us, 257 19.3, 512 26.5.
// ------------------------------------------------------------------------------------------------
constexpr int kBwdThreads = 512, kBwdWaves = kBwdThreads / 64;

// 16-byte slot of a column's piece in the transposed image.
__device__ __forceinline__ int t_slot(int c, int piece) { return ((c ^ ((c >> 6) & 1)) * 8 + (piece ^ ((c >> 3) & 7))); }

// FULL: rows is a multiple of 128. Otherwise no tiling along the rows is asked for, and rows past the end count as
// zeros of da.
template <int ACT, bool GATED, bool FULL>
__global__ __launch_bounds__(kBwdThreads, GATED ? 2 : 4) void fg_act_bwd_kernel(FgActBwd p) {
    constexpr int Z = GATED ? 2 : 1;            // halves of dz
    constexpr int V = Z + 1;                    // values with column tiles: dz, a
    constexpr bool AHEAD = GATED;               // inputs loaded a tile ahead
    extern __shared__ __attribute__((aligned(16))) uint8_t smem[];
    uint4* image = reinterpret_cast<uint4*>(smem);                              // [V][128 * 8]
    float* colmax = reinterpret_cast<float*>(smem);                             // [V][32][128], before the image
    float* colsum = reinterpret_cast<float*>(smem + V * 16384);                 // [Z][kBwdWaves][128]
    float* col_s = colsum + Z * kBwdWaves * 128;                                // [V][128] scales, then reciprocals
    float* col_r = col_s + V * 128;
    __shared__ int small_w[8];                  // per wave of the column scales: one below 2^-80

    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t F = p.F, W = Z * F, rows = p.rows;
    const uint32_t row_blocks = (uint32_t)((rows + FG_GROUP - 1) / FG_GROUP);
    const int64_t gstep = F / FG_GROUP;
    const uint32_t tiles = row_blocks * (uint32_t)gstep;
    const bool want_dz = FULL && p.dzq_rows != nullptr, want_a = FULL && p.aq_rows != nullptr, want_b = p.dbias != nullptr;

    // a thread's four rows of inputs as loaded
    v2i in_z[4][Z];
    float in_s[4][Z];
    v4i in_d[4][2];
    auto load = [&](uint32_t tile, int chunk, int rgrp) __attribute__((always_inline)) {
        const int64_t g = tile / row_blocks, r0 = (int64_t)(tile % row_blocks) * FG_GROUP;
        const uint32_t W32 = (uint32_t)W, ld32 = (uint32_t)p.ld_da;
        // rows past the end: the last one again
        const int last = FULL ? 0 : (int)(rows - 1 - r0 < 127 ? rows - 1 - r0 : 127);
        auto row = [&](int i) { return FULL ? 4 * rgrp : (4 * rgrp + i < last ? 4 * rgrp + i : last); };
#pragma unroll
        for (int i = 0; i < 4; i++)
#pragma unroll
            for (int h = 0; h < Z; h++) {
                const uint8_t* z = p.zq + (r0 + (FULL ? i : 0)) * W + h * F + g * FG_GROUP;
                in_z[i][h] = *reinterpret_cast<const v2i*>(z + ((uint32_t)row(i) * W32 + 8 * chunk));
                const float* s = p.sz + (h * gstep + g) * rows + r0 + (FULL ? i : 0);
                in_s[i][h] = s[(uint32_t)row(i)];
            }
        if (p.da_bf16) {
#pragma unroll
            for (int i = 0; i < 4; i++) {
                const uint16_t* d = (const uint16_t*)p.da + (r0 + (FULL ? i : 0)) * p.ld_da + g * FG_GROUP;
                in_d[i][0] = *reinterpret_cast<const v4i*>(d + ((uint32_t)row(i) * ld32 + 8 * chunk));
                in_d[i][1] = v4i{0, 0, 0, 0};
            }
        } else {
#pragma unroll
            for (int i = 0; i < 4; i++) {
                const float* d = (const float*)p.da + (r0 + (FULL ? i : 0)) * p.ld_da + g * FG_GROUP;
                const uint32_t off = (uint32_t)row(i) * ld32 + 8 * chunk;
                in_d[i][0] = *reinterpret_cast<const v4i*>(d + off);
                in_d[i][1] = *reinterpret_cast<const v4i*>(d + off + 4);
            }
        }
    };

    if constexpr (AHEAD) load(blockIdx.x, threadIdx.x & 15, threadIdx.x >> 4);
    for (uint32_t tile = blockIdx.x; tile < tiles; tile += gridDim.x) {
        // The thread's place, hidden from the compiler so that it does not keep the addresses that follow from it in
        // registers from tile to tile (they would spill).
        int t = threadIdx.x;
        asm volatile("" : "+v"(t));
        const int lane = t & 63, chunk = t & 15, rgrp = t >> 4;
        const int64_t br = tile % row_blocks, g = tile / row_blocks;
        const int64_t r0 = br * FG_GROUP + 4 * rgrp;

        if constexpr (!AHEAD) load(tile, chunk, rgrp);
        float v[V][4][8];                        // v[h < Z]: dz; v[Z]: a, which begins as da
        if (p.da_bf16) {
#pragma unroll
            for (int i = 0; i < 4; i++) unpack8(make_uint4(in_d[i][0].x, in_d[i][0].y, in_d[i][0].z, in_d[i][0].w), v[Z][i]);
        } else {
#pragma unroll
            for (int i = 0; i < 4; i++) {
#pragma unroll
                for (int e = 0; e < 8; e++) v[Z][i][e] = __int_as_float(in_d[i][e >> 2][e & 3]);
            }
        }
        if constexpr (!FULL) {
#pragma unroll
            for (int i = 0; i < 4; i++)
#pragma unroll
                for (int e = 0; e < 8; e++) v[Z][i][e] = r0 + i < rows ? v[Z][i][e] : 0.0f;
        }
#pragma unroll
        for (int i = 0; i < 4; i++) {
            float zv[Z][8];
#pragma unroll
            for (int h = 0; h < Z; h++) {
                const auto f0 = __builtin_amdgcn_cvt_pk_f32_fp8((int)in_z[i][h].x, false), f1 = __builtin_amdgcn_cvt_pk_f32_fp8((int)in_z[i][h].x, true);
                const auto f2 = __builtin_amdgcn_cvt_pk_f32_fp8((int)in_z[i][h].y, false), f3 = __builtin_amdgcn_cvt_pk_f32_fp8((int)in_z[i][h].y, true);
                const float f[8] = {f0[0], f0[1], f1[0], f1[1], f2[0], f2[1], f3[0], f3[1]};
#pragma unroll
                for (int e = 0; e < 8; e++) zv[h][e] = f[e] * in_s[i][h];
            }
#pragma unroll
            for (int e = 0; e < 8; e++) {
                const float da = v[Z][i][e];
                float act, slope;
                fg_act_both<ACT>(zv[0][e], act, slope);
                if constexpr (GATED) {
                    v[0][i][e] = da * zv[1][e] * slope;
                    v[1][i][e] = da * act;
                    v[Z][i][e] = act * zv[1][e];
                } else {
                    v[0][i][e] = da * slope;
                    v[Z][i][e] = act;
                }
            }
            __builtin_amdgcn_sched_barrier(0);
        }
        // the next tile's inputs (past the last tile, this one's again) come in while this one is quantized
        if constexpr (AHEAD) load(tile + gridDim.x < tiles ? tile + gridDim.x : tile, chunk, rgrp);
        __builtin_amdgcn_sched_barrier(0);

        // tiles along the columns
#pragma unroll
        for (int h = 0; h < Z; h++) {
            float m[4], s[4];
#pragma unroll
            for (int i = 0; i < 4; i++) m[i] = fg_row16_max(absmax8(v[h][i]));
            fg_scales_from_amax(m, p.pow2, s);
            uint2 c[4];
            if (!fg_any_small(__builtin_fminf(__builtin_fminf(s[0], s[1]), __builtin_fminf(s[2], s[3])))) {
#pragma unroll
                for (int i = 0; i < 4; i++) c[i] = quant8<false>(v[h][i], s[i]);
            } else {
#pragma unroll
                for (int i = 0; i < 4; i++) c[i] = quant8<true>(v[h][i], s[i]);
            }
#pragma unroll
            for (int i = 0; i < 4; i++) {
                uint8_t* out = p.dzq_cols + (br * FG_GROUP + i) * W + h * F + g * FG_GROUP;
                if (FULL || r0 + i < rows) *reinterpret_cast<uint2*>(out + (4 * (uint32_t)rgrp * (uint32_t)W + 8 * chunk)) = c[i];
            }
            const float own = chunk & 2 ? (chunk & 1 ? s[3] : s[2]) : (chunk & 1 ? s[1] : s[0]);   // lane i of 16: row i's
            float* out_s = p.sdz_cols + (h * gstep + g) * rows + br * FG_GROUP;
            if (chunk < 4 && (FULL || r0 + chunk < rows)) out_s[4 * (uint32_t)rgrp + chunk] = own;
            __builtin_amdgcn_sched_barrier(0);
        }
        if (!want_dz && !want_a && !want_b) continue;

        // column maxima of the thread's four rows, and column sums of its wave's 16
#pragma unroll
        for (int k = 0; k < V; k++) {
            if (k < Z ? !want_dz : !want_a) continue;
            float m[8];
#pragma unroll
            for (int e = 0; e < 8; e++) {
                m[e] = 0.0f;
#pragma unroll
                for (int i = 0; i < 4; i++) m[e] = __builtin_fmaxf(m[e], __builtin_fabsf(v[k][i][e]));
            }
            v4f* out = reinterpret_cast<v4f*>(colmax + (k * 32 + rgrp) * 128 + chunk * 8);
            out[0] = v4f{m[0], m[1], m[2], m[3]};
            out[1] = v4f{m[4], m[5], m[6], m[7]};
            __builtin_amdgcn_sched_barrier(0);
        }
        if (want_b) {
#pragma unroll
            for (int h = 0; h < Z; h++)
#pragma unroll
                for (int e = 0; e < 8; e++) {
                    const float s = rows_sum((v[h][0][e] + v[h][1][e]) + (v[h][2][e] + v[h][3][e]));
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
        if (!want_dz && !want_a) {
            __syncthreads();                    // the sums are read before the next tile's are written
            continue;
        }
        // one scale and reciprocal per column
        if (t < V * 128) {
            const int k = t >> 7, c = t & 127;
            if (k < Z ? want_dz : want_a) {
                float m = 0.0f;
#pragma unroll
                for (int w = 0; w < 32; w++) m = __builtin_fmaxf(m, colmax[(k * 32 + w) * 128 + c]);
                const float s = fg_scale_from_amax(m, p.pow2);
                const fg_divisor d = fg_divisor_of(s);
                col_s[t] = d.s;
                col_r[t] = d.r;
                const bool small = fg_any_small(s);
                if (lane == 0) small_w[wave] = small;
                if (k < Z) p.sdz_rows[br * W + k * F + g * FG_GROUP + c] = s;
                else p.sa_rows[br * F + g * FG_GROUP + c] = s;
            }
        }
        __syncthreads();
#pragma unroll
        for (int k = 0; k < V; k++) {
            if (k < Z ? !want_dz : !want_a) continue;
            // dword rgrp of column c = 8 chunk + e, at t_slot: swapping column pairs moves the even columns up by one
            // column (128 bytes) and the odd ones down
            uint8_t* even = smem + k * 16384 + chunk * 1024 + ((rgrp >> 2) ^ (chunk & 7)) * 16 + (rgrp & 3) * 4;
            uint8_t* odd = even - (chunk >> 3) * 128;
            even += (chunk >> 3) * 128;
            auto quant_columns = [&](auto small) {
#pragma unroll
                for (int e0 = 0; e0 < 8; e0 += 4) {
                    const v4f s = *reinterpret_cast<const v4f*>(col_s + k * 128 + chunk * 8 + e0);
                    const v4f r = *reinterpret_cast<const v4f*>(col_r + k * 128 + chunk * 8 + e0);
#pragma unroll
                    for (int e = 0; e < 4; e++) {
                        const fg_divisor d{s[e], r[e]};
                        *reinterpret_cast<uint32_t*>((e & 1 ? odd : even) + (e0 + e) * 128) =
                            fg_quant4<decltype(small)::value>(v[k][0][e0 + e], v[k][1][e0 + e], v[k][2][e0 + e], v[k][3][e0 + e], d);
                    }
                    __builtin_amdgcn_sched_barrier(0);      // the columns' divisors not all at once
                }
            };
            if (small_w[2 * k] | small_w[2 * k + 1]) quant_columns(std::true_type{});
            else quant_columns(std::false_type{});
        }
        __syncthreads();
#pragma unroll
        for (int k = 0; k < V; k++) {
            if (k < Z ? !want_dz : !want_a) continue;
#pragma unroll
            for (int j = 0; j < 1024 / kBwdThreads; j++) {
                uint8_t* out = (k < Z ? p.dzq_rows + k * F * rows : p.aq_rows) + (g * FG_GROUP + 64 * j) * rows + br * FG_GROUP;
                const int c = t >> 3, piece = t & 7;
                *reinterpret_cast<uint4*>(out + ((uint32_t)c * (uint32_t)rows + 16 * piece)) = image[k * 1024 + t_slot(64 * j + c, piece)];
            }
        }
        __syncthreads();                        // the image is read before the next tile's maxima take its place
    }
}

// Sum of the row blocks' partial bias gradients: 64 columns a workgroup, the blocks dealt to 16 waves in turn (four
// loads of each in flight) and the waves' sums added in order, so that the result depends on the sizes only, which atomics
// would not give. 64 blocks of 7168 columns: 4.7 us, mostly the launch.
constexpr int kSumWaves = 16;
__global__ __launch_bounds__(kSumWaves * 64) void fg_bias_sum_kernel(const float* __restrict__ partial, int64_t blocks, int64_t W,
                                                                    float* __restrict__ dbias) {
    __shared__ float sums[kSumWaves][64];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int64_t c = (int64_t)blockIdx.x * 64 + lane;
    float s = 0.0f;
    for (int64_t b = wave; b < blocks; b += 4 * kSumWaves) {
        float v[4];
#pragma unroll
        for (int i = 0; i < 4; i++) v[i] = b + i * kSumWaves < blocks ? partial[(b + i * kSumWaves) * W + c] : 0.0f;
#pragma unroll
        for (int i = 0; i < 4; i++) s += v[i];
    }
    sums[wave][lane] = s;
    __syncthreads();
    if (wave == 0) {
        s = 0.0f;
#pragma unroll
        for (int w = 0; w < kSumWaves; w++) s += sums[w][lane];
        dbias[c] = s;
    }
}

template <int ACT, bool GATED, bool FULL>
hipError_t launch_bwd(const FgActBwd& p, unsigned tiles, hipStream_t stream) {
    constexpr int Z = GATED ? 2 : 1, V = Z + 1;
    constexpr int bytes = V * 16384 + Z * kBwdWaves * 128 * 4 + 2 * V * 128 * 4;
    auto kern = fg_act_bwd_kernel<ACT, GATED, FULL>;
    static std::atomic<uint64_t> lds_limit_set{0};
    const hipError_t e = fg_set_lds_limit_once((const void*)kern, bytes, lds_limit_set);
    if (e != hipSuccess) return e;
    const unsigned grid = GATED ? std::min(tiles, (unsigned)fg_device_cus()) : tiles;
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
        const unsigned tiles = (unsigned)(blocks * (p.F / FG_GROUP));
        const hipError_t e = by_act(p.act, [&](auto tag) {
            constexpr int ACT = decltype(tag)::value;
            if (p.rows % FG_GROUP == 0)
                return p.gated ? launch_bwd<ACT, true, true>(p, tiles, stream) : launch_bwd<ACT, false, true>(p, tiles, stream);
            return p.gated ? launch_bwd<ACT, true, false>(p, tiles, stream) : launch_bwd<ACT, false, false>(p, tiles, stream);
        });
        if (e != hipSuccess) return e;
    }
    if (p.dbias && blocks != 1) {   // no rows: sums of nothing
        hipLaunchKernelGGL(fg_bias_sum_kernel, dim3((unsigned)(W / 64)), dim3(kSumWaves * 64), 0, stream, p.partial, blocks, W, p.dbias);
        return hipGetLastError();
    }
    return hipSuccess;
}

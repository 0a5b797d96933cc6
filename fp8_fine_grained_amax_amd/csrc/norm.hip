// Layer and RMS norm whose output leaves as FP8 tiles, and their backward pass (gfx950). Both are bound by HBM.
//
// A row's threads hold it in registers, eight neighbouring columns a thread and group, so a 1x128 tile is 16 lanes (one
// DPP row). With tiles along the columns only, one kernel reads x once for statistics, tiles and output. Tiles along the rows
// need the statistics of 128 rows, which no workgroup holds: there one kernel makes the statistics, and a second one reads x
// again in 128 x 128 blocks and writes both tilings. (Columns' tiles in the first kernel and rows' tiles in the second write
// the same bytes, but with the first kernel's scales scattered and its sums waited for twice: 4096 x 7168 bf16 43.0 us
// against 36.4, 4096 x 18432 f32 155 against 147.)
//
// y is (x gamma) rstd, in this order: the product of two bf16 numbers is exact in FP32, so RMS of bf16 x and gamma rounds once
// before the codes, whose borders such products often lie on. rstd's power of two goes to x first, which rounds nothing and keeps
// x gamma from overflowing where y does not.
#include "host_util.h"
#include "tile8.h"
#include "train_launch.h"

#include <algorithm>
#include <type_traits>

namespace {

// Element i of an array of f32 or bf16: with a uniform i, a uniform address to which a lane adds its 32-bit offset.
__device__ __forceinline__ const void* at_elem(const void* p, int64_t i, int bf16) { return (const char*)p + (i << (bf16 ? 1 : 2)); }

// Eight elements of f32 or bf16 as loaded.
struct Raw8 {
    uint4 a, b;
    __device__ __forceinline__ void load(const void* p, uint32_t i, int bf16) {
        if (bf16) {
            a = *reinterpret_cast<const uint4*>((const uint16_t*)p + i);
        } else {
            a = *reinterpret_cast<const uint4*>((const float*)p + i);
            b = *reinterpret_cast<const uint4*>((const float*)p + i + 4);
        }
    }
    // Hides that these are the values loaded, so that what was computed from them is computed again and not kept.
    __device__ __forceinline__ void hide() {
        asm volatile("" : "+v"(a.x), "+v"(a.y), "+v"(a.z), "+v"(a.w), "+v"(b.x), "+v"(b.y), "+v"(b.z), "+v"(b.w));
    }
    __device__ __forceinline__ void get(float (&f)[8], int bf16) const {
        if (bf16) {
            unpack8(a, f);
        } else {
            const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
            for (int e = 0; e < 8; e++) f[e] = __uint_as_float(w[e]);
        }
    }
};

__device__ __forceinline__ void store8(void* p, uint32_t i, const float (&f)[8], int bf16) {
    if (bf16) {
        uint32_t w[4];
#pragma unroll
        for (int e = 0; e < 4; e++) w[e] = fg_bf16_bits(f[2 * e]) | (fg_bf16_bits(f[2 * e + 1]) << 16);
        *reinterpret_cast<uint4*>((uint16_t*)p + i) = make_uint4(w[0], w[1], w[2], w[3]);
    } else {
        float* o = (float*)p + i;
        *reinterpret_cast<float4*>(o) = make_float4(f[0], f[1], f[2], f[3]);
        *reinterpret_cast<float4*>(o + 4) = make_float4(f[4], f[5], f[6], f[7]);
    }
}

typedef float v4f_at4 __attribute__((ext_vector_type(4), aligned(4)));      // the scales' buffer is aligned to its elements only

// Sum over the 16 lanes of a DPP row, in all of them (row_ror 8 and 4, quad_perm [2,3,0,1] and [1,0,3,2]).
__device__ __forceinline__ float row16_sum(float v) {
#define FG_STEP(ctrl) v += __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), ctrl, 0xF, 0xF, false));
    FG_STEP(0x128)
    FG_STEP(0x124)
    FG_STEP(0x4E)
    FG_STEP(0xB1)
#undef FG_STEP
    return v;
}
// Sum over a DPP row's lanes l % LANES, in all of them.
template <int LANES>
__device__ __forceinline__ float lanes_sum(float v) {
    if constexpr (LANES <= 8) v += __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), 0x128, 0xF, 0xF, false));
    if constexpr (LANES <= 4) v += __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), 0x124, 0xF, 0xF, false));
    return v;
}
__device__ __forceinline__ float wave_sum(float v) { return rows_sum(row16_sum(v)); }

// y's parts: ((x - mean) power gamma) rest, where power rest is rstd, power a power of two, and rest in [1, 2), so that the first three
// factors are as large as y at most. (x - mean) power is one operation, rounded as x - mean is, as long as mean power is in range: where it
// would not be (a constant row and a tiny eps), power is less and rest more. A rstd of NaN makes rest NaN; zero or denormal it is not.
template <bool LAYER>
struct Normed {
    float power, shift, rest;
    __device__ __forceinline__ void set(float mean, float rstd) {
        uint32_t e = __float_as_uint(rstd) >> 23 & 255;
        if constexpr (LAYER) {
            const uint32_t most = 380 - (__float_as_uint(mean) >> 23 & 255);       // the product below 2^128
            e = e < most ? e : most;
        }
        power = __uint_as_float(e << 23);
        shift = LAYER ? -mean * power : 0.0f;
        rest = rstd * __uint_as_float((254 - e) << 23);
    }
    __device__ __forceinline__ float gained(float x, float gamma) const {
        return (LAYER ? __builtin_fmaf(x, power, shift) : x * power) * gamma;
    }
};

constexpr int kMaxWaves = 16;
// Threads of a workgroup whose threads hold U groups of eight columns each: with more groups a thread needs more registers
// than 16 waves leave it.
constexpr int max_waves(int u) { return u == 1 ? 16 : 12; }

// The place of a workgroup's threads: `waves` to a row, so blockDim / (64 waves) rows at a time. Group u of thread t of a row
// holds the columns 8 (t + 64 waves u) .. + 7.
struct Place {
    int wave, lane, group, groups, first, t, span, chunks;       // first: of the row's waves; chunks: a row's eights
    __device__ __forceinline__ Place(int waves, int64_t cols) {
        wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
        lane = threadIdx.x & 63;
        group = wave / waves;
        first = group * waves;
        groups = (int)(blockDim.x >> 6) / waves;
        t = (int)threadIdx.x - first * 64;
        span = 64 * waves;
        chunks = (int)(cols / 8);
    }
    // Whether group u of U begins behind the row's end: only the last one can (the host takes no more waves than that needs).
    template <int U>
    __device__ __forceinline__ bool past(int u) const { return u + 1 == U && t + u * span >= chunks; }
    template <int U>
    __device__ __forceinline__ int wave_cols(int w) const {      // columns of the row's wave w
        int n = 0;
#pragma unroll
        for (int u = 0; u < U; u++) {
            const int left = chunks - w * 64 - u * span;
            n += 8 * (left < 0 ? 0 : left > 64 ? 64 : left);
        }
        return n;
    }
};

// ------------------------------------------------------------------------------------------------
// Forward: the statistics, and with TILES the columns' tiles and the output. U groups of eight columns a thread, the next row's
// loaded while this one is worked on. With TILES a workgroup's rows follow one another, so that the scales it writes (rows
// contiguous) meet in lines of its own L2; without, rows are dealt in turn, so that the last ones are those that the Infinity
// Cache still holds when the second kernel begins with them.
//
// 4096 x 7168 bf16, columns' tiles: RMS 22.5 us, 4.0 TB/s (a copy of x takes 21 us; with x from HBM 24.5), layer 28, with beta 27.4 to 32;
// without its loads or its stores RMS takes 18 to 20, so HBM, sums and quantization overlap and none of them alone bounds it.
// 4096 x 18432 f32: 85 us, 4.5 TB/s; there HBM does.
//
// FEW rows: a thread has as few groups as 16 waves a row allow, and gamma and beta in registers; a call's time is the latency
// of its loads (one row of 1024: 2.3 us). Many: two groups (three past 16384 columns), so that what a row costs besides its elements
// (sums, joins) is shared by more of them, and gamma and beta in LDS.
// ------------------------------------------------------------------------------------------------
template <int U, bool XB, bool LAYER, bool FEW, bool TILES>
__global__ __launch_bounds__(64 * (FEW ? max_waves(U) : 16)) void fg_norm_kernel(FgNorm p, int waves, int64_t rows_each) {
    __shared__ float part[2][kMaxWaves][2];         // a row's waves: sum, and sum of squares about the wave's mean
    extern __shared__ __attribute__((aligned(16))) float weights[];    // gamma, then beta
    const Place at(waves, p.cols);
    const int64_t row0 = (int64_t)blockIdx.x * (TILES ? rows_each : at.groups), step = (int64_t)at.groups * (TILES ? 1 : gridDim.x);
    const int64_t end = TILES && row0 + rows_each < p.rows ? row0 + rows_each : p.rows;
    const float n = (float)p.cols;

    Raw8 next[U];
    auto load = [&](int64_t row) {
        row = row < end ? row : end - 1;
#pragma unroll
        for (int u = 0; u < U; u++)
            if (!at.past<U>(u)) next[u].load(at_elem(p.x, row * p.ld, XB), 8 * (at.t + u * at.span), XB);
    };
    load(row0 + at.group);
    float gamma[FEW ? U : 1][8], beta[FEW ? U : 1][8];
    auto weight = [&](const void* from, int c, float (&f)[8]) {
        Raw8 w;
        w.load(from, 8 * c, p.w_bf16);
        w.get(f, p.w_bf16);
    };
    if constexpr (TILES && FEW) {
#pragma unroll
        for (int u = 0; u < U; u++) {
            if (at.past<U>(u)) continue;
            weight(p.gamma, at.t + u * at.span, gamma[u]);
            if (p.beta) weight(p.beta, at.t + u * at.span, beta[u]);
        }
    } else if constexpr (TILES) {
        for (int c = threadIdx.x; c < at.chunks; c += (int)blockDim.x) {
            weight(p.gamma, c, gamma[0]);
            store8(weights, 8 * c, gamma[0], 0);
            if (p.beta) {
                weight(p.beta, c, beta[0]);
                store8(weights + p.cols, 8 * c, beta[0], 0);
            }
        }
        __syncthreads();
    }
    float* scales[U];                               // of the lane's tiles, row 0
#pragma unroll
    for (int u = 0; u < U; u++) scales[u] = p.s_cols + (int64_t)((at.t + u * at.span) >> 4) * p.rows;
    int parity = 0;
    for (int64_t base = row0; base < end; base += step, parity ^= 1) {
        const int64_t row = base + at.group;
        float v[U][8];
#pragma unroll
        for (int u = 0; u < U; u++) next[u].get(v[u], XB);
        load(row + step);

        float sum = 0.0f, mean = 0.0f, square = 0.0f;
        if constexpr (LAYER) {
#pragma unroll
            for (int u = 0; u < U; u++) {
                if (at.past<U>(u)) continue;
#pragma unroll
                for (int e = 0; e < 8; e++) sum += v[u][e];
            }
            sum = wave_sum(sum);
            const int own = at.wave_cols<U>(at.wave - at.first);
            mean = own ? sum / (float)own : 0.0f;
        }
#pragma unroll
        for (int u = 0; u < U; u++) {
            if (at.past<U>(u)) continue;
#pragma unroll
            for (int e = 0; e < 8; e++) {
                const float d = LAYER ? v[u][e] - mean : v[u][e];
                square = __builtin_fmaf(d, d, square);
            }
        }
        square = wave_sum(square);
        if (waves > 1) {
            if (at.lane == 0) {
                part[parity][at.wave][0] = sum;
                part[parity][at.wave][1] = square;
            }
            __syncthreads();
            // each DPP row joins the waves' parts, one a lane
            const int w = at.lane & 15;
            const bool there = w < waves;
            square = there ? part[parity][at.first + w][1] : 0.0f;
            if constexpr (LAYER) {                  // about the row's mean instead of the wave's
                const float s = there ? part[parity][at.first + w][0] : 0.0f;
                mean = row16_sum(s) / n;
                const float cols = (float)at.wave_cols<U>(w), d = there && cols > 0.0f ? s / cols - mean : 0.0f;
                square = __builtin_fmaf(cols * d, d, square);
            }
            square = row16_sum(square);
        }
        if (row >= end) continue;
        const float var = square / n;
        // a row that is not finite, or whose squares overflow, is NaN throughout (RMS would make its finite values zeros)
        const float rstd = var < __builtin_inff() ? 1.0f / __builtin_sqrtf(var + p.eps) : __builtin_nanf("");
        if (at.t == 0) {
            if (LAYER && p.mean) p.mean[row] = mean;
            if (p.rstd) p.rstd[row] = rstd;
        }
        if constexpr (!TILES) continue;
        float top[U], s[U];
        Normed<LAYER> normed;
        normed.set(mean, rstd);
#pragma unroll
        for (int u = 0; u < U; u++) {
            const int c = at.t + u * at.span;
            top[u] = 1.0f;                          // past the end: nothing, and no small scale
            if (at.past<U>(u)) continue;            // whole DPP rows: cols is a multiple of 128
            if constexpr (!FEW) {
                const v4f a = *reinterpret_cast<const v4f*>(weights + 8 * c), b = *reinterpret_cast<const v4f*>(weights + 8 * c + 4);
#pragma unroll
                for (int e = 0; e < 4; e++) gamma[0][e] = a[e], gamma[0][4 + e] = b[e];
                if (p.beta) {
                    const float* from = weights + (int)p.cols + 8 * c;
                    const v4f d = *reinterpret_cast<const v4f*>(from), f = *reinterpret_cast<const v4f*>(from + 4);
#pragma unroll
                    for (int e = 0; e < 4; e++) beta[0][e] = d[e], beta[0][4 + e] = f[e];
                }
            }
#pragma unroll
            for (int e = 0; e < 8; e++) v[u][e] = normed.gained(v[u][e], gamma[FEW ? u : 0][e]);
            if (p.beta) {
#pragma unroll
                for (int e = 0; e < 8; e++) v[u][e] = __builtin_fmaf(v[u][e], normed.rest, beta[FEW ? u : 0][e]);
            } else {
#pragma unroll
                for (int e = 0; e < 8; e++) v[u][e] *= normed.rest;
            }
            top[u] = fg_row16_max(absmax8(v[u]));
        }
        fg_scales_from_amax(top, p.pow2, s);
        float least = s[0];
#pragma unroll
        for (int u = 1; u < U; u++) least = __builtin_fminf(least, s[u]);
        const bool small = fg_any_small(least);
        uint8_t* out = p.q_cols + row * p.cols;
#pragma unroll
        for (int u = 0; u < U; u++) {
            const int c = at.t + u * at.span;
            if (at.past<U>(u)) continue;
            const uint2 q = small ? quant8<true>(v[u], s[u]) : quant8<false>(v[u], s[u]);
            *reinterpret_cast<uint2*>(out + 8 * (uint32_t)c) = q;
            if ((at.t & 15) == 0) scales[u][row] = s[u];       // the span is a multiple of 64
        }
        if (p.y) {
#pragma unroll
            for (int u = 0; u < U; u++)
                if (!at.past<U>(u)) store8(p.y + row * p.cols, 8 * (at.t + u * at.span), v[u], 1);
        }
    }
}

// ------------------------------------------------------------------------------------------------
// Forward, both tilings and the output: a 512-thread workgroup takes 128 rows x 128 columns and reads x again (from the Infinity
// Cache where it fits, hence the last rows first), with the statistics of the kernel above. Thread t holds rows 4 (t / 16) + i
// of the eight columns t % 16: a row's tile is a DPP row, while the columns' maxima and codes go through LDS. HBM bounds it: 4096
// x 7168 bf16 23.2 us, x from the cache, 117 MB in all; 4096 x 18432 f32 75.7 us, 453 MB, 6.0 TB/s. The statistics before it: 10.6
// and 73.0 us (5.5 and 4.1 TB/s).
// ------------------------------------------------------------------------------------------------
template <bool LAYER>
__global__ __launch_bounds__(512) void fg_norm_tiles_kernel(FgNorm p) {
    __shared__ __attribute__((aligned(16))) uint8_t smem[16384];       // maxima [32][128], then codes [128 columns][128 rows]
    __shared__ float col_s[128], col_r[128];
    __shared__ int small_w[2];
    float* colmax = reinterpret_cast<float*>(smem);
    const int tid = threadIdx.x, lane = tid & 63, chunk = tid & 15, rgrp = tid >> 4;
    const uint32_t blocks = (uint32_t)(p.cols / FG_GROUP);
    const int64_t g = blockIdx.x % blocks, br = (gridDim.x - 1 - blockIdx.x) / blocks;
    const int64_t r0 = br * FG_GROUP + 4 * rgrp, col = g * FG_GROUP + 8 * chunk;

    Raw8 raw[4], w;
#pragma unroll
    for (int i = 0; i < 4; i++) raw[i].load(at_elem(p.x, (r0 + i) * p.ld, p.x_bf16), (uint32_t)col, p.x_bf16);
    float gamma[8], beta[8], y[4][8];
    Normed<LAYER> normed[4];
#pragma unroll
    for (int i = 0; i < 4; i++) normed[i].set(LAYER ? p.mean[r0 + i] : 0.0f, p.rstd[r0 + i]);
    w.load(p.gamma, col, p.w_bf16);
    w.get(gamma, p.w_bf16);
    if (p.beta) {
        w.load(p.beta, col, p.w_bf16);
        w.get(beta, p.w_bf16);
    }
#pragma unroll
    for (int i = 0; i < 4; i++) {
        raw[i].get(y[i], p.x_bf16);
#pragma unroll
        for (int e = 0; e < 8; e++) {
            const float t = normed[i].gained(y[i][e], gamma[e]);
            y[i][e] = p.beta ? __builtin_fmaf(t, normed[i].rest, beta[e]) : t * normed[i].rest;
        }
    }
    float top[4], s[4], m[8];
#pragma unroll
    for (int i = 0; i < 4; i++) top[i] = fg_row16_max(absmax8(y[i]));
    fg_scales_from_amax(top, p.pow2, s);
    const bool small = fg_any_small(__builtin_fminf(__builtin_fminf(s[0], s[1]), __builtin_fminf(s[2], s[3])));
#pragma unroll
    for (int i = 0; i < 4; i++) {
        const uint2 q = small ? quant8<true>(y[i], s[i]) : quant8<false>(y[i], s[i]);
        *reinterpret_cast<uint2*>(p.q_cols + (r0 + i) * p.cols + col) = q;
        if (p.y) store8(p.y + (r0 + i) * p.cols, (uint32_t)col, y[i], 1);
    }
    if (chunk == 0) *reinterpret_cast<v4f_at4*>(p.s_cols + g * p.rows + r0) = v4f_at4{s[0], s[1], s[2], s[3]};
#pragma unroll
    for (int e = 0; e < 8; e++) {
        m[e] = 0.0f;
#pragma unroll
        for (int i = 0; i < 4; i++) m[e] = __builtin_fmaxf(m[e], __builtin_fabsf(y[i][e]));
    }
    v4f* out = reinterpret_cast<v4f*>(colmax + rgrp * 128 + chunk * 8);
    out[0] = v4f{m[0], m[1], m[2], m[3]};
    out[1] = v4f{m[4], m[5], m[6], m[7]};
    __syncthreads();
    if (tid < 128) {
        float most = 0.0f;
#pragma unroll
        for (int r = 0; r < 32; r++) most = __builtin_fmaxf(most, colmax[r * 128 + tid]);
        const float scale = fg_scale_from_amax(most, p.pow2);
        const fg_divisor d = fg_divisor_of(scale);
        col_s[tid] = d.s;
        col_r[tid] = d.r;
        const bool tiny = fg_any_small(scale);
        if (lane == 0) small_w[tid >> 6] = tiny;
        p.s_rows[br * p.cols + g * FG_GROUP + tid] = scale;
    }
    __syncthreads();
    uint8_t* even = smem + chunk * 1024 + ((rgrp >> 2) ^ (chunk & 7)) * 16 + (rgrp & 3) * 4;
    uint8_t* odd = even - (chunk >> 3) * 128;
    even += (chunk >> 3) * 128;
    auto quant_columns = [&](auto small) {
#pragma unroll
        for (int e = 0; e < 8; e++) {
            const fg_divisor d{col_s[chunk * 8 + e], col_r[chunk * 8 + e]};
            *reinterpret_cast<uint32_t*>((e & 1 ? odd : even) + e * 128) =
                fg_quant4<decltype(small)::value>(y[0][e], y[1][e], y[2][e], y[3][e], d);
        }
    };
    if (small_w[0] | small_w[1]) quant_columns(std::true_type{});
    else quant_columns(std::false_type{});
    __syncthreads();
    const uint4* image = reinterpret_cast<const uint4*>(smem);
#pragma unroll
    for (int j = 0; j < 2; j++) {
        const int c = 64 * j + (tid >> 3), piece = tid & 7;
        *reinterpret_cast<uint4*>(p.q_rows + (g * FG_GROUP + c) * p.rows + br * FG_GROUP + 16 * piece) = image[t_slot(c, piece)];
    }
}

// ------------------------------------------------------------------------------------------------
// Backward. The threads of a row as in the forward kernel with few rows; a workgroup's rows follow one another, and each thread
// adds up its own columns' dy xhat and dy over them. The groups of a workgroup join in LDS, the workgroups in a second launch:
// no atomics, so that the result depends on the sizes only.
//
// HBM bounds it: x, dy and the residual's gradient are read once and dx is written (inputs bf16, f32, bf16; dx bf16). Up to
// 8192 columns the next row is loaded while this one is worked on: 4096 x 7168 62 us, 4.7 TB/s; 16384 x 2048 68 us, 4.9 TB/s
// (a copy reaches 4.7 to 5.2). With two and three groups a thread the registers do not hold a second row: 4096 x 12288 122 us,
// 4.1 TB/s, 4096 x 18432 179 us, 4.2 TB/s. (With the same inputs again and again, part of which the Infinity Cache then holds,
// 58, 58, 108 and 160 us.) The second launch takes 2.5 to 5 us. Few rows are bound by latency, so they take one
// launch, in which other workgroups read x and dy once more for the columns' sums.
// ------------------------------------------------------------------------------------------------
// Columns of a workgroup that sums them by itself. 64 and 128: 256 x 1024 f32 5.3 and 6.4 us, 512 x 1024 7.0 and 9.9, 64 x 18432
// 11.2 and 8.8; 32 the first as 64, the last 12.3.
constexpr int kSlab = 64;
// A workgroup's columns of dgamma and dbeta, whole: kSlab / 8 lanes to a row, so 512 / kSlab rows of a wave at a time.
template <bool LAYER>
__device__ __forceinline__ void sum_columns(const FgNormBwd& p, int block, float (*sums)[kMaxWaves][kSlab]) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, waves = (int)(blockDim.x >> 6);
    constexpr int LANES = kSlab / 8, ROWS = 64 / LANES;
    const int64_t col = (int64_t)block * kSlab + 8 * (lane % LANES), step = ROWS * waves;
    float dg[8] = {}, db[8] = {};
    constexpr int AT_ONCE = 4;
    for (int64_t r0 = ROWS * wave + lane / LANES; r0 < p.rows; r0 += AT_ONCE * step) {
        Raw8 rx[AT_ONCE], rd[AT_ONCE];
        float rstd[AT_ONCE], mean[AT_ONCE];
#pragma unroll
        for (int i = 0; i < AT_ONCE; i++) {
            const int64_t row = r0 + i * step < p.rows ? r0 + i * step : p.rows - 1;
            rx[i].load(at_elem(p.x, row * p.ld_x, p.x_bf16), (uint32_t)col, p.x_bf16);
            rd[i].load(at_elem(p.dy, row * p.ld_dy, p.dy_bf16), (uint32_t)col, p.dy_bf16);
            rstd[i] = p.rstd[row];
            mean[i] = LAYER ? p.mean[row] : 0.0f;
        }
#pragma unroll
        for (int i = 0; i < AT_ONCE; i++) {
            if (r0 + i * step >= p.rows) continue;
            float x[8], d[8];
            rx[i].get(x, p.x_bf16);
            rd[i].get(d, p.dy_bf16);
#pragma unroll
            for (int e = 0; e < 8; e++) {
                dg[e] += d[e] * ((LAYER ? x[e] - mean[i] : x[e]) * rstd[i]);
                db[e] += d[e];
            }
        }
    }
#pragma unroll
    for (int e = 0; e < 8; e++) {
        dg[e] = rows_sum(lanes_sum<LANES>(dg[e]));
        db[e] = rows_sum(lanes_sum<LANES>(db[e]));
    }
    if (lane < LANES) {
        store8(sums[0][wave], 8 * lane, dg, 0);
        store8(sums[1][wave], 8 * lane, db, 0);
    }
    __syncthreads();
    const int which = (int)threadIdx.x / kSlab, c = threadIdx.x % kSlab;
    float* out = which == 0 ? p.dgamma : which == 1 ? p.dbeta : nullptr;
    if (!out) return;
    out += (int64_t)block * kSlab + c;
    float s = p.accumulate ? *out : 0.0f;
    for (int w = 0; w < waves; w++) s += sums[which][w][c];
    *out = s;
}

// SUMS: the rows' workgroups add up the columns, dgamma's and with BIAS dbeta's. Otherwise the first `first` workgroups do that,
// reading x and dy once more.
template <int U, bool LAYER, bool SUMS, bool BIAS>
__global__ __launch_bounds__(64 * max_waves(U)) void fg_norm_bwd_kernel(FgNormBwd p, int waves, int64_t rows_each, int64_t partials, int first) {
    constexpr bool AHEAD = U == 1;                  // with more groups the registers do not hold a second row
    __shared__ float part[2][kMaxWaves][2];
    if constexpr (!SUMS) {
        __shared__ float sums[2][kMaxWaves][kSlab];
        if ((int)blockIdx.x < first) {
            sum_columns<LAYER>(p, blockIdx.x, sums);
            return;
        }
    }
    constexpr bool HELD = SUMS && U > 2;            // the columns' sums are held in LDS, dgamma's and then dbeta's
    extern __shared__ __attribute__((aligned(16))) float join[];       // else with more than one group [groups][cols] of dgamma's, then dbeta's
    const Place at(waves, p.cols);
    const int64_t row0 = (int64_t)(blockIdx.x - first) * rows_each;
    const int64_t end = row0 + rows_each < p.rows ? row0 + rows_each : p.rows;
    const float inv_n = 1.0f / (float)p.cols;
    // At.past, but asked of all groups after the first: the branches keep the compiler from working on all of them at once, for
    // which it has too few registers.
    auto behind = [&](int u) { return (u > 0 || U == 1) && at.t + u * at.span >= at.chunks; };
    float dg[HELD ? 1 : U][8], db[BIAS && !HELD ? U : 1][8];
#pragma unroll
    for (int u = 0; u < U; u++) {
        const float zero[8] = {};
        if constexpr (HELD) {
            if (behind(u)) continue;
            store8(join, 8 * (at.t + u * at.span), zero, 0);
            if constexpr (BIAS) store8(join + p.cols, 8 * (at.t + u * at.span), zero, 0);
        } else {
#pragma unroll
            for (int e = 0; e < 8; e++) dg[u][e] = db[BIAS ? u : 0][e] = 0.0f;
        }
    }
    // adds to a thread's own columns of the sums in LDS
    auto held = [&](float* sums, const float (&v)[8]) {
        v4f* s = reinterpret_cast<v4f*>(sums);
        s[0] += v4f{v[0], v[1], v[2], v[3]};
        s[1] += v4f{v[4], v[5], v[6], v[7]};
    };

    Raw8 rx[U], rd[U], rr[AHEAD ? U : 1], nx[AHEAD ? U : 1], nd[AHEAD ? U : 1], nr[AHEAD ? U : 1];
    float next_rstd, next_mean = 0.0f;
    auto load = [&](int64_t row, Raw8* x, Raw8* d) {
        row = row < end ? row : end - 1;
#pragma unroll
        for (int u = 0; u < U; u++) {
            const uint32_t c = 8 * (at.t + u * at.span);
            if (behind(u)) continue;
            x[u].load(at_elem(p.x, row * p.ld_x, p.x_bf16), c, p.x_bf16);
            d[u].load(at_elem(p.dy, row * p.ld_dy, p.dy_bf16), c, p.dy_bf16);
            if constexpr (AHEAD)
                if (p.dres) nr[u].load(at_elem(p.dres, row * p.ld_dres, p.dres_bf16), c, p.dres_bf16);
        }
        next_rstd = p.rstd[row];
        if (LAYER) next_mean = p.mean[row];
    };
    float gamma[AHEAD ? U : 1][8];
    auto load_gamma = [&](int u, float (&g)[8]) {
        Raw8 w;
        w.load(p.gamma, 8 * (at.t + u * at.span), p.w_bf16);
        w.get(g, p.w_bf16);
    };
    if constexpr (AHEAD) {
        load(row0 + at.group, nx, nd);
        if (!behind(0)) load_gamma(0, gamma[0]);
    }
    int parity = 0;
    for (int64_t base = row0; base < end; base += at.groups, parity ^= 1) {
        const int64_t row = base + at.group;
        const bool live = row < end;
        if constexpr (AHEAD) {
            rx[0] = nx[0];
            rd[0] = nd[0];
            rr[0] = nr[0];
        } else {
            load(row, rx, rd);
        }
        const float rstd = next_rstd, mean = next_mean;
        if constexpr (AHEAD) load(row + at.groups, nx, nd);     // behind the last row it again: a branch costs 12% at 4096 x 7168
        float t1 = 0.0f, t2 = 0.0f;
#pragma unroll
        for (int u = 0; u < U; u++) {
            if (behind(u)) continue;
            float x[8], d[8];
            if constexpr (!AHEAD) load_gamma(u, gamma[0]);
            rx[u].get(x, p.x_bf16);
            rd[u].get(d, p.dy_bf16);
#pragma unroll
            for (int e = 0; e < 8; e++) {
                const float h = (LAYER ? x[e] - mean : x[e]) * rstd, t = d[e] * gamma[0][e];
                x[e] = d[e] * h;
                t1 += t;
                t2 = __builtin_fmaf(t, h, t2);
            }
            if (SUMS && live) {
                if constexpr (HELD) {
                    held(join + 8 * (at.t + u * at.span), x);
                    if constexpr (BIAS) held(join + p.cols + 8 * (at.t + u * at.span), d);
                } else {
#pragma unroll
                    for (int e = 0; e < 8; e++) {
                        dg[u][e] += x[e];
                        if constexpr (BIAS) db[u][e] += d[e];
                    }
                }
            }
            if constexpr (U > 1) __builtin_amdgcn_sched_barrier(0);    // the groups one after the other: registers
        }
        t2 = wave_sum(t2);
        if constexpr (LAYER) t1 = wave_sum(t1);
        if (waves > 1) {
            if (at.lane == 0) {
                part[parity][at.wave][0] = t1;
                part[parity][at.wave][1] = t2;
            }
            __syncthreads();
            const int w = at.lane & 15;             // each DPP row joins the waves' parts, one a lane
            t2 = row16_sum(w < waves ? part[parity][at.first + w][1] : 0.0f);
            if constexpr (LAYER) t1 = row16_sum(w < waves ? part[parity][at.first + w][0] : 0.0f);
        }
        if (!live) continue;
        t1 *= inv_n;
        t2 *= inv_n;
#pragma unroll
        for (int u = 0; u < U; u++) {
            const uint32_t c = 8 * (at.t + u * at.span);
            if (behind(u)) continue;
            float x[8], d[8], r[8];
            if constexpr (!AHEAD) {
                load_gamma(u, gamma[0]);
                if (p.dres) rr[0].load(at_elem(p.dres, row * p.ld_dres, p.dres_bf16), c, p.dres_bf16);
                rx[u].hide();
                rd[u].hide();
            }
            rx[u].get(x, p.x_bf16);
            rd[u].get(d, p.dy_bf16);
#pragma unroll
            for (int e = 0; e < 8; e++) {
                const float h = (LAYER ? x[e] - mean : x[e]) * rstd;
                const float t = __builtin_fmaf(d[e], gamma[0][e], LAYER ? -t1 : 0.0f);
                d[e] = __builtin_fmaf(-h, t2, t) * rstd;
            }
            if (p.dres) {
                rr[0].get(r, p.dres_bf16);
#pragma unroll
                for (int e = 0; e < 8; e++) d[e] += r[e];
            }
            store8((char*)p.dx + (row * p.cols << (p.dx_bf16 ? 1 : 2)), c, d, p.dx_bf16);
            if constexpr (U > 1) __builtin_amdgcn_sched_barrier(0);
        }
    }
    if constexpr (!SUMS) return;
    float *out_g = p.partial + (int64_t)blockIdx.x * p.cols, *out_b = p.partial + (partials + (int64_t)blockIdx.x) * p.cols;
    if constexpr (HELD) {
#pragma unroll
        for (int u = 0; u < U; u++) {
            const int c = 8 * (at.t + u * at.span);
            if (behind(u)) continue;
            for (int e = 0; e < 8; e += 4) {
                if (p.dgamma) *reinterpret_cast<v4f*>(out_g + c + e) = *reinterpret_cast<const v4f*>(join + c + e);
                if constexpr (BIAS) *reinterpret_cast<v4f*>(out_b + c + e) = *reinterpret_cast<const v4f*>(join + p.cols + c + e);
            }
        }
    } else if (at.groups == 1) {
#pragma unroll
        for (int u = 0; u < U; u++) {
            const int c = 8 * (at.t + u * at.span);
            if (behind(u)) continue;
            if (p.dgamma) store8(out_g, c, dg[u], 0);
            if constexpr (BIAS) store8(out_b, c, db[u], 0);
        }
    } else {
        const int cols = (int)p.cols;
        float* join_b = join + at.groups * cols;
#pragma unroll
        for (int u = 0; u < U; u++) {
            const int c = at.group * cols + 8 * (at.t + u * at.span);
            if (behind(u)) continue;
            store8(join, c, dg[u], 0);
            if constexpr (BIAS) store8(join_b, c, db[u], 0);
        }
        __syncthreads();
        for (int c = threadIdx.x; c < cols; c += (int)blockDim.x) {
            float s = 0.0f, t = 0.0f;
            for (int g = 0; g < at.groups; g++) {
                s += join[g * cols + c];
                if constexpr (BIAS) t += join_b[g * cols + c];
            }
            if (p.dgamma) out_g[c] = s;
            if constexpr (BIAS) out_b[c] = t;
        }
    }
}

// Sums of the workgroups' partial sums: 64 columns a workgroup, the partials dealt to 16 waves in turn and the waves' sums
// added in order, so that the result depends on the sizes only.
constexpr int kSumWaves = 16;
__global__ __launch_bounds__(kSumWaves * 64) void fg_norm_sum_kernel(const float* __restrict__ partial, int64_t partials, int64_t cols,
                                                                    float* dgamma, float* dbeta, int accumulate) {
    __shared__ float sums[kSumWaves][64];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int64_t c = (int64_t)blockIdx.x * 64 + lane;
    float* out = blockIdx.y == 0 ? dgamma : dbeta;
    if (!out) return;
    const float* from = partial + (int64_t)blockIdx.y * partials * cols;
    float s = 0.0f;
    for (int64_t b = wave; b < partials; b += 4 * kSumWaves) {     // four loads in flight
        float v[4];
#pragma unroll
        for (int i = 0; i < 4; i++) v[i] = b + i * kSumWaves < partials ? from[(b + i * kSumWaves) * cols + c] : 0.0f;
#pragma unroll
        for (int i = 0; i < 4; i++) s += v[i];
    }
    sums[wave][lane] = s;
    __syncthreads();
    if (wave == 0) {
        s = accumulate ? out[c] : 0.0f;
#pragma unroll
        for (int w = 0; w < kSumWaves; w++) s += sums[w][lane];
        out[c] = s;
    }
}

// Groups of eight columns a thread and waves a row: as few groups as 16 waves (12 with more than one) allow.
int groups_of_thread(int64_t cols) {
    int u = 1;
    while (512 * u * max_waves(u) < cols) u++;
    return u;
}
int waves_of_row(int64_t cols) { return (int)((cols + 512 * groups_of_thread(cols) - 1) / (512 * groups_of_thread(cols))); }

template <class Fn>
hipError_t by_groups(int64_t cols, Fn&& fn) {
    static_assert(kFgNormMaxCols == 512 * 3 * max_waves(3), "three groups reach the widest row");
    switch (groups_of_thread(cols)) {
        case 1: return fn(std::integral_constant<int, 1>{});
        case 2: return fn(std::integral_constant<int, 2>{});
        default: return fn(std::integral_constant<int, 3>{});
    }
}

template <int U, bool FEW, bool TILES>
hipError_t launch_fwd(const FgNorm& p, int waves, int groups, int64_t fill, hipStream_t stream) {
    const int64_t each = ((p.rows + fill - 1) / fill + groups - 1) / groups * groups;
    const unsigned grid = (unsigned)((p.rows + each - 1) / each), threads = 64u * waves * groups;
    const int lds = FEW || !TILES ? 0 : (int)p.cols * (p.beta ? 8 : 4);
    auto go = [&](auto kern, std::atomic<uint64_t>& limit_set) {
        if (lds > 0) {
            const hipError_t e = fg_set_lds_limit_once((const void*)kern, (int)kFgNormMaxCols * 8, limit_set);
            if (e != hipSuccess) return e;
        }
        hipLaunchKernelGGL(kern, dim3(grid), dim3(threads), lds, stream, p, waves, each);
        return hipGetLastError();
    };
    static std::atomic<uint64_t> limits[4];
    if (p.x_bf16) return p.layer ? go(fg_norm_kernel<U, true, true, FEW, TILES>, limits[0]) : go(fg_norm_kernel<U, true, false, FEW, TILES>, limits[1]);
    return p.layer ? go(fg_norm_kernel<U, false, true, FEW, TILES>, limits[2]) : go(fg_norm_kernel<U, false, false, FEW, TILES>, limits[3]);
}

constexpr int64_t kMaxPartials = 256;
// FEW and many measured, bf16 rows: 64 of 7168 4.3 and 4.5 us, 256 of 18432 6.8 and 7.2; 512 of 7168 6.6 and 6.0, 512 of 18432 11.7
// and 9.7, 4096 of 7168 24.0 and 22.1.
constexpr int64_t kFewRows = 256;

// Rows whose backward is one launch, in which workgroups of their own sum the columns, and reads x and dy twice; with more rows the
// rows' workgroups keep the sums, and a second launch adds them. One and two launches: 64 x 1024 bf16 4.6
// and 7.5 us, 512 x 1024 5.3 and 8.0, 1024 x 1024 8.0 and 8.8, 2048 x 1024 12.8 and 10.7; f32 256 x 4096 6.6 and 11.0, 512 x 128 5.2
// and 7.0, 512 x 18432 40.9 and 43.7, 1024 x 128 8.7 and 7.0, 1024 x 4096 16.9 and 16.4.
constexpr int64_t kFewGradRows = 512;

int bwd_groups(int64_t cols) { return max_waves(groups_of_thread(cols)) / waves_of_row(cols); }
// Workgroups of the backward's rows, at most.
int64_t row_blocks(int64_t rows, int64_t cols) {
    const int64_t groups = bwd_groups(cols);
    return std::min(kMaxPartials, (rows + groups - 1) / groups);
}

}  // namespace

hipError_t fg_launch_norm(const FgNorm& p, hipStream_t stream) {
    auto rows = [&](auto tiles) {
        constexpr bool TILES = decltype(tiles)::value;
        const int64_t cus = fg_device_cus(), units = (p.cols + 511) / 512;
        if (TILES && p.rows <= kFewRows) {
            const int waves = waves_of_row(p.cols), groups = std::max(1, 4 / waves);
            return by_groups(p.cols, [&](auto u) {
                return launch_fwd<decltype(u)::value, true, true>(p, waves, groups, cus * (32 / (waves * groups)), stream);
            });
        }
        const int u = (int)std::min<int64_t>(units, units <= 32 ? 2 : 3), waves = (int)((units + u - 1) / u), groups = std::max(1, 4 / waves);
        // Waves of a CU: a bf16 row's need half the bytes, so more of them are in flight. 16 and 24: bf16 6000 x 5632 34.7 and 28.2 us, 4096
        // x 12288 41.8 and 36.7, 4096 x 7168 both 22, but 16384 x 2048 21.5 and 23.0 and three groups (4096 x 18432) 49.1 and 51.4; f32 6000
        // x 5632 36.1 and 38.7; the statistics alone 4096 x 18432 f32 145 and 146.
        const int resident = TILES && p.x_bf16 && u == 2 && p.cols > 2048 ? 24 : 16;
        // no more workgroups than a CU's 160 KB hold the weights of: with beta, 4096 x 7168 27 us, with three of them, of which two fit, 31
        const int64_t held = TILES ? (160 * 1024) / (p.cols * (p.beta ? 8 : 4) + 512) : 16;
        const int64_t fill = cus * std::max<int64_t>(1, std::min<int64_t>(resident / (waves * groups), held));
        switch (u) {
            case 1: return launch_fwd<1, false, TILES>(p, waves, groups, fill, stream);
            case 2: return launch_fwd<2, false, TILES>(p, waves, groups, fill, stream);
            default: return launch_fwd<3, false, TILES>(p, waves, groups, fill, stream);
        }
    };
    const hipError_t e = p.q_rows ? rows(std::false_type{}) : rows(std::true_type{});
    if (e != hipSuccess || !p.q_rows) return e;
    const unsigned tiles = (unsigned)((p.cols / FG_GROUP) * (p.rows / FG_GROUP));
    if (p.layer) hipLaunchKernelGGL((fg_norm_tiles_kernel<true>), dim3(tiles), dim3(512), 0, stream, p);
    else hipLaunchKernelGGL((fg_norm_tiles_kernel<false>), dim3(tiles), dim3(512), 0, stream, p);
    return hipGetLastError();
}

int64_t fg_norm_bwd_partials(int64_t rows, int64_t cols) {
    if (rows <= kFewGradRows) return 0;
    return row_blocks(rows, cols);
}

hipError_t fg_launch_norm_bwd(const FgNormBwd& p, hipStream_t stream) {
    const int waves = waves_of_row(p.cols), groups = bwd_groups(p.cols);
    const int64_t most = row_blocks(p.rows, p.cols);
    const bool weights = p.dgamma || p.dbeta, few = weights && p.rows > 0 && p.rows <= kFewGradRows, sums = weights && !few;
    const int first = few ? (int)(p.cols / kSlab) : 0;
    int64_t partials = 0;
    if (p.rows > 0) {
        const int64_t each = ((p.rows + most - 1) / most + groups - 1) / groups * groups;
        partials = (p.rows + each - 1) / each;
        const unsigned threads = 64u * waves * groups;
        // the groups' joins, or past 12288 columns the columns' sums
        const bool held = groups_of_thread(p.cols) > 2;
        const int bytes = !sums ? 0 : (int)p.cols * 4 * (p.dbeta ? 2 : 1) * (held ? 1 : groups > 1 ? groups : 0);
        const hipError_t e = by_groups(p.cols, [&](auto u) {
            constexpr int U = decltype(u)::value;
            auto go = [&](auto kern, std::atomic<uint64_t>& limit_set) {
                if (bytes > 0) {
                    const hipError_t e = fg_set_lds_limit_once((const void*)kern, (int)kFgNormMaxCols * 8, limit_set);
                    if (e != hipSuccess) return e;
                }
                hipLaunchKernelGGL(kern, dim3((unsigned)(first + partials)), dim3(threads), bytes, stream, p, waves, each, partials, first);
                return hipGetLastError();
            };
            static std::atomic<uint64_t> limits[6];
            if (p.layer) {
                if (!sums) return go(fg_norm_bwd_kernel<U, true, false, false>, limits[0]);
                return p.dbeta ? go(fg_norm_bwd_kernel<U, true, true, true>, limits[1]) : go(fg_norm_bwd_kernel<U, true, true, false>, limits[2]);
            }
            if (!sums) return go(fg_norm_bwd_kernel<U, false, false, false>, limits[3]);
            return p.dbeta ? go(fg_norm_bwd_kernel<U, false, true, true>, limits[4]) : go(fg_norm_bwd_kernel<U, false, true, false>, limits[5]);
        });
        if (e != hipSuccess) return e;
    }
    if (first > 0 || (!p.dgamma && !p.dbeta)) return hipSuccess;
    hipLaunchKernelGGL(fg_norm_sum_kernel, dim3((unsigned)(p.cols / 64), 2), dim3(kSumWaves * 64), 0, stream, p.partial, partials, p.cols,
                       p.dgamma, p.dbeta, p.accumulate);
    return hipGetLastError();
}

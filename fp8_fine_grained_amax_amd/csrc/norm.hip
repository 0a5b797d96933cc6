// Layer and RMS norm whose output leaves as FP8 tiles, and their backward pass (gfx950). Both are bound by HBM.
//
// A row's threads hold it in registers, eight neighbouring columns a thread and group, so a 1x128 tile is 16 lanes (one
// DPP row) and x is read once for statistics, tiles and output. Rows that a workgroup takes follow one another, so that the
// scales it writes (rows contiguous) meet in lines of its own L2.
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

// Sum over the wave, in every lane: within the DPP rows (row_ror 8 and 4, quad_perm [2,3,0,1] and [1,0,3,2]), then across.
__device__ __forceinline__ float wave_sum(float v) {
#define FG_STEP(ctrl) v += __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), ctrl, 0xF, 0xF, false));
    FG_STEP(0x128)
    FG_STEP(0x124)
    FG_STEP(0x4E)
    FG_STEP(0xB1)
#undef FG_STEP
    return rows_sum(v);
}

// The place of a workgroup's threads: `waves` to a row, so blockDim / (64 waves) rows at a time.
struct Place {
    int wave, lane, group, groups, first, t;       // first: of the row's waves; t: thread of the row
    __device__ __forceinline__ explicit Place(int waves) {
        wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
        lane = threadIdx.x & 63;
        group = wave / waves;
        first = group * waves;
        groups = (int)(blockDim.x >> 6) / waves;
        t = (int)threadIdx.x - first * 64;
    }
};

// Waves of a workgroup whose threads hold U groups of eight columns each: with more groups a thread needs more registers than
// 16 waves leave it.
constexpr int kMaxWaves = 16;
constexpr int max_waves(int u) { return u <= 2 ? 16 : 12; }

// ------------------------------------------------------------------------------------------------
// Forward, tiles along the columns. U groups of eight columns a thread.
// ------------------------------------------------------------------------------------------------
template <int U, bool LAYER>
__global__ __launch_bounds__(64 * max_waves(U)) void fg_norm_kernel(FgNorm p, int waves, int64_t rows_each) {
    __shared__ float part[2][kMaxWaves][2];         // a row's waves: sum, and sum of squares about the wave's mean
    const Place at(waves);
    const int chunks = (int)(p.cols / 8), span = 64 * waves;
    const int64_t row0 = (int64_t)blockIdx.x * rows_each;
    const int64_t end = row0 + rows_each < p.rows ? row0 + rows_each : p.rows;
    const float n = (float)p.cols;

    Raw8 next[U];
    auto load = [&](int64_t row) {
        row = row < end ? row : end - 1;
#pragma unroll
        for (int u = 0; u < U; u++)
            if (at.t + u * span < chunks) next[u].load(at_elem(p.x, row * p.ld, p.x_bf16), 8 * (at.t + u * span), p.x_bf16);
    };
    load(row0 + at.group);
    int parity = 0;
    for (int64_t base = row0; base < end; base += at.groups, parity ^= 1) {
        const int64_t row = base + at.group;
        float v[U][8];
#pragma unroll
        for (int u = 0; u < U; u++) next[u].get(v[u], p.x_bf16);
        load(row + at.groups);

        float sum = 0.0f, mean = 0.0f, square = 0.0f;
        int own = 0;                                // the wave's columns
#pragma unroll
        for (int u = 0; u < U; u++) {
            const int left = chunks - (at.wave - at.first) * 64 - u * span;
            own += 8 * (left < 0 ? 0 : left > 64 ? 64 : left);
        }
        if constexpr (LAYER) {
#pragma unroll
            for (int u = 0; u < U; u++) {
                if (at.t + u * span >= chunks) continue;
#pragma unroll
                for (int e = 0; e < 8; e++) sum += v[u][e];
            }
            sum = wave_sum(sum);
            mean = own ? sum / (float)own : 0.0f;
        }
#pragma unroll
        for (int u = 0; u < U; u++) {
            if (at.t + u * span >= chunks) continue;
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
            if constexpr (LAYER) {
                sum = 0.0f;
                for (int w = 0; w < waves; w++) sum += part[parity][at.first + w][0];
                mean = sum / n;
            }
            square = 0.0f;
            for (int w = 0; w < waves; w++) {
                square += part[parity][at.first + w][1];
                if constexpr (LAYER) {              // about the row's mean instead of the wave's
                    int cols = 0;
#pragma unroll
                    for (int u = 0; u < U; u++) {
                        const int left = chunks - w * 64 - u * span;
                        cols += 8 * (left < 0 ? 0 : left > 64 ? 64 : left);
                    }
                    const float d = cols ? part[parity][at.first + w][0] / (float)cols - mean : 0.0f;
                    square += (float)cols * d * d;
                }
            }
        }
        if (row >= end) continue;
        const float var = square / n;
        // a row that is not finite, or whose squares overflow, is NaN throughout (RMS would make its finite values zeros)
        const float rstd = var < __builtin_inff() ? 1.0f / __builtin_sqrtf(var + p.eps) : __builtin_nanf("");
        if (at.t == 0) {
            if (LAYER && p.mean) p.mean[row] = mean;
            if (p.rstd) p.rstd[row] = rstd;
        }
#pragma unroll
        for (int u = 0; u < U; u++) {
            const int c = at.t + u * span;
            if (c >= chunks) continue;              // whole DPP rows: cols is a multiple of 128
            Raw8 w;
            float gamma[8], beta[8], y[8];
            w.load(p.gamma, 8 * c, p.w_bf16);
            w.get(gamma, p.w_bf16);
#pragma unroll
            for (int e = 0; e < 8; e++) y[e] = (LAYER ? v[u][e] - mean : v[u][e]) * rstd;
            if (p.beta) {
                w.load(p.beta, 8 * c, p.w_bf16);
                w.get(beta, p.w_bf16);
#pragma unroll
                for (int e = 0; e < 8; e++) y[e] = __builtin_fmaf(y[e], gamma[e], beta[e]);
            } else {
#pragma unroll
                for (int e = 0; e < 8; e++) y[e] *= gamma[e];
            }
            const float s = fg_scale_from_amax(fg_row16_max(absmax8(y)), p.pow2);
            const uint2 q = fg_any_small(s) ? quant8<true>(y, s) : quant8<false>(y, s);
            *reinterpret_cast<uint2*>(p.q_cols + row * p.cols + 8 * (uint32_t)c) = q;
            if ((c & 15) == 0) p.s_cols[(c >> 4) * p.rows + row] = s;
            if (p.y) store8(p.y + row * p.cols, 8 * c, y, 1);
        }
    }
}

// ------------------------------------------------------------------------------------------------
// Forward, tiles along the rows: a 512-thread workgroup takes 128 rows x 128 columns and reads x again (from the Infinity
// Cache where it fits), with the statistics of the kernel above. Thread t holds rows 4 (t / 16) + i of the eight
// columns t % 16; the columns' maxima and the codes go through LDS.
// ------------------------------------------------------------------------------------------------
template <bool LAYER>
__global__ __launch_bounds__(512) void fg_norm_tokens_kernel(FgNorm p) {
    __shared__ __attribute__((aligned(16))) uint8_t smem[16384];       // maxima [32][128], then codes [128 columns][128 rows]
    __shared__ float col_s[128], col_r[128];
    __shared__ int small_w[2];
    float* colmax = reinterpret_cast<float*>(smem);
    const int tid = threadIdx.x, lane = tid & 63, chunk = tid & 15, rgrp = tid >> 4;
    const uint32_t blocks = (uint32_t)(p.cols / FG_GROUP);
    const int64_t g = blockIdx.x % blocks, br = blockIdx.x / blocks;
    const int64_t r0 = br * FG_GROUP + 4 * rgrp, col = g * FG_GROUP + 8 * chunk;

    Raw8 raw[4], w;
#pragma unroll
    for (int i = 0; i < 4; i++) raw[i].load(at_elem(p.x, (r0 + i) * p.ld, p.x_bf16), (uint32_t)col, p.x_bf16);
    float mean[4], rstd[4], gamma[8], beta[8], y[4][8];
#pragma unroll
    for (int i = 0; i < 4; i++) {
        rstd[i] = p.rstd[r0 + i];
        mean[i] = LAYER ? p.mean[r0 + i] : 0.0f;
    }
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
            const float h = (LAYER ? y[i][e] - mean[i] : y[i][e]) * rstd[i];
            y[i][e] = p.beta ? __builtin_fmaf(h, gamma[e], beta[e]) : h * gamma[e];
        }
    }
    float m[8];
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
        float top = 0.0f;
#pragma unroll
        for (int r = 0; r < 32; r++) top = __builtin_fmaxf(top, colmax[r * 128 + tid]);
        const float s = fg_scale_from_amax(top, p.pow2);
        const fg_divisor d = fg_divisor_of(s);
        col_s[tid] = d.s;
        col_r[tid] = d.r;
        const bool small = fg_any_small(s);
        if (lane == 0) small_w[tid >> 6] = small;
        p.s_rows[br * p.cols + g * FG_GROUP + tid] = s;
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
// Backward. The threads of a row as in the forward kernel; a workgroup's rows follow one another, and each thread adds up
// its own columns' dy xhat and dy over them. The groups of a workgroup join in LDS, the workgroups in a second launch.
// ------------------------------------------------------------------------------------------------
template <int U, bool LAYER>
__global__ __launch_bounds__(64 * max_waves(U)) void fg_norm_bwd_kernel(FgNormBwd p, int waves, int64_t rows_each, int64_t partials) {
    __shared__ float part[2][kMaxWaves][2];
    extern __shared__ __attribute__((aligned(16))) float join[];       // [groups][cols], with more than one group
    const Place at(waves);
    const int chunks = (int)(p.cols / 8), span = 64 * waves;
    const int64_t row0 = (int64_t)blockIdx.x * rows_each;
    const int64_t end = row0 + rows_each < p.rows ? row0 + rows_each : p.rows;
    const float inv_n = 1.0f / (float)p.cols;
    float dg[U][8], db[U][8];
#pragma unroll
    for (int u = 0; u < U; u++)
#pragma unroll
        for (int e = 0; e < 8; e++) dg[u][e] = db[u][e] = 0.0f;

    int parity = 0;
    for (int64_t base = row0; base < end; base += at.groups, parity ^= 1) {
        const int64_t row = base + at.group < end ? base + at.group : end - 1;
        const bool live = base + at.group < end;
        const float rstd = p.rstd[row], mean = LAYER ? p.mean[row] : 0.0f;
        Raw8 rx[U], rd[U];
#pragma unroll
        for (int u = 0; u < U; u++) {
            const uint32_t c = 8 * (at.t + u * span);
            if (at.t + u * span >= chunks) continue;
            rx[u].load(at_elem(p.x, row * p.ld_x, p.x_bf16), c, p.x_bf16);
            rd[u].load(at_elem(p.dy, row * p.ld_dy, p.dy_bf16), c, p.dy_bf16);
        }
        float t1 = 0.0f, t2 = 0.0f;
#pragma unroll
        for (int u = 0; u < U; u++) {
            if (at.t + u * span >= chunks) continue;
            float x[8], d[8], gamma[8];
            Raw8 w;
            w.load(p.gamma, 8 * (at.t + u * span), p.w_bf16);
            w.get(gamma, p.w_bf16);
            rx[u].get(x, p.x_bf16);
            rd[u].get(d, p.dy_bf16);
#pragma unroll
            for (int e = 0; e < 8; e++) {
                const float h = (LAYER ? x[e] - mean : x[e]) * rstd, t = d[e] * gamma[e];
                if (live) {
                    dg[u][e] = __builtin_fmaf(d[e], h, dg[u][e]);
                    db[u][e] += d[e];
                }
                t1 += t;
                t2 = __builtin_fmaf(t, h, t2);
            }
            if constexpr (U > 2) __builtin_amdgcn_sched_barrier(0);    // the groups one after the other: registers
        }
        t2 = wave_sum(t2);
        if constexpr (LAYER) t1 = wave_sum(t1);
        if (waves > 1) {
            if (at.lane == 0) {
                part[parity][at.wave][0] = t1;
                part[parity][at.wave][1] = t2;
            }
            __syncthreads();
            t1 = t2 = 0.0f;
            for (int w = 0; w < waves; w++) {
                t1 += part[parity][at.first + w][0];
                t2 += part[parity][at.first + w][1];
            }
        }
        if (!live) continue;
        t1 *= inv_n;
        t2 *= inv_n;
#pragma unroll
        for (int u = 0; u < U; u++) {
            const uint32_t c = 8 * (at.t + u * span);
            if (at.t + u * span >= chunks) continue;
            float x[8], d[8], gamma[8], r[8];
            Raw8 w;
            w.load(p.gamma, c, p.w_bf16);
            w.get(gamma, p.w_bf16);
            rx[u].get(x, p.x_bf16);
            rd[u].get(d, p.dy_bf16);
#pragma unroll
            for (int e = 0; e < 8; e++) {
                const float h = (LAYER ? x[e] - mean : x[e]) * rstd;
                const float t = __builtin_fmaf(d[e], gamma[e], LAYER ? -t1 : 0.0f);
                d[e] = __builtin_fmaf(-h, t2, t) * rstd;
            }
            if (p.dres) {
                w.load(at_elem(p.dres, row * p.ld_dres, p.dres_bf16), c, p.dres_bf16);
                w.get(r, p.dres_bf16);
#pragma unroll
                for (int e = 0; e < 8; e++) d[e] += r[e];
            }
            store8((char*)p.dx + (row * p.cols << (p.dx_bf16 ? 1 : 2)), c, d, p.dx_bf16);
            if constexpr (U > 2) __builtin_amdgcn_sched_barrier(0);
        }
    }
    if (!p.partial) return;
    auto put = [&](float (&v)[U][8], float* out) {
        if (at.groups > 1) {
            __syncthreads();
#pragma unroll
            for (int u = 0; u < U; u++)
                if (at.t + u * span < chunks) store8(join, at.group * (uint32_t)p.cols + 8 * (at.t + u * span), v[u], 0);
            __syncthreads();
            for (int c = threadIdx.x; c < (int)p.cols; c += (int)blockDim.x) {
                float s = 0.0f;
                for (int g = 0; g < at.groups; g++) s += join[g * (int)p.cols + c];
                out[c] = s;
            }
        } else {
#pragma unroll
            for (int u = 0; u < U; u++)
                if (at.t + u * span < chunks) store8(out, 8 * (at.t + u * span), v[u], 0);
        }
    };
    if (p.dgamma) put(dg, p.partial + (int64_t)blockIdx.x * p.cols);
    if (p.dbeta) put(db, p.partial + (partials + (int64_t)blockIdx.x) * p.cols);
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
    for (int64_t b = wave; b < partials; b += kSumWaves) s += from[b * cols + c];
    sums[wave][lane] = s;
    __syncthreads();
    if (wave == 0) {
        s = accumulate ? out[c] : 0.0f;
#pragma unroll
        for (int w = 0; w < kSumWaves; w++) s += sums[w][lane];
        out[c] = s;
    }
}

// Groups of eight columns a thread and waves a row: as few groups as 16 waves (12 with three groups) allow.
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

constexpr int64_t kMaxPartials = 256;
int bwd_groups(int64_t cols) { return max_waves(groups_of_thread(cols)) / waves_of_row(cols); }

}  // namespace

hipError_t fg_launch_norm(const FgNorm& p, hipStream_t stream) {
    const int waves = waves_of_row(p.cols), groups = std::max(1, 4 / waves);
    const unsigned threads = 64u * waves * groups;
    const int64_t fill = (int64_t)fg_device_cus() * (2048 / threads);
    int64_t each = (p.rows + fill - 1) / fill;
    each = (each + groups - 1) / groups * groups;
    const unsigned grid = (unsigned)((p.rows + each - 1) / each);
    hipError_t e = by_groups(p.cols, [&](auto u) {
        constexpr int U = decltype(u)::value;
        if (p.layer) hipLaunchKernelGGL((fg_norm_kernel<U, true>), dim3(grid), dim3(threads), 0, stream, p, waves, each);
        else hipLaunchKernelGGL((fg_norm_kernel<U, false>), dim3(grid), dim3(threads), 0, stream, p, waves, each);
        return hipGetLastError();
    });
    if (e != hipSuccess || !p.q_rows) return e;
    const unsigned tiles = (unsigned)((p.cols / FG_GROUP) * (p.rows / FG_GROUP));
    if (p.layer) hipLaunchKernelGGL((fg_norm_tokens_kernel<true>), dim3(tiles), dim3(512), 0, stream, p);
    else hipLaunchKernelGGL((fg_norm_tokens_kernel<false>), dim3(tiles), dim3(512), 0, stream, p);
    return hipGetLastError();
}

int64_t fg_norm_bwd_partials(int64_t rows, int64_t cols) {
    const int64_t groups = bwd_groups(cols);
    return std::min(kMaxPartials, (rows + groups - 1) / groups);
}

hipError_t fg_launch_norm_bwd(const FgNormBwd& p, hipStream_t stream) {
    const int waves = waves_of_row(p.cols), groups = bwd_groups(p.cols);
    const int64_t most = fg_norm_bwd_partials(p.rows, p.cols);
    int64_t partials = 0;
    if (p.rows > 0) {
        const int64_t each = ((p.rows + most - 1) / most + groups - 1) / groups * groups;
        partials = (p.rows + each - 1) / each;
        const unsigned threads = 64u * waves * groups;
        const size_t bytes = groups > 1 && p.partial ? (size_t)groups * (size_t)p.cols * 4 : 0;
        const hipError_t e = by_groups(p.cols, [&](auto u) {
            constexpr int U = decltype(u)::value;
            if (p.layer) hipLaunchKernelGGL((fg_norm_bwd_kernel<U, true>), dim3((unsigned)partials), dim3(threads), bytes, stream, p, waves, each, partials);
            else hipLaunchKernelGGL((fg_norm_bwd_kernel<U, false>), dim3((unsigned)partials), dim3(threads), bytes, stream, p, waves, each, partials);
            return hipGetLastError();
        });
        if (e != hipSuccess) return e;
    }
    if (!p.dgamma && !p.dbeta) return hipSuccess;
    hipLaunchKernelGGL(fg_norm_sum_kernel, dim3((unsigned)(p.cols / 64), 2), dim3(kSumWaves * 64), 0, stream, p.partial, partials, p.cols,
                       p.dgamma, p.dbeta, p.accumulate);
    return hipGetLastError();
}

// A Linear of few rows with its epilogue (gfx950): bound by the rate at which the weight's codes stream from HBM
// (see weight_stream.h).
#include "ffn_epilogue.h"
#include "ffn_launch.h"
#include "weight_stream.h"

namespace {

// ---------------------------------------------------------------------------------------------------------
// A Linear of few rows: y = act(x . W^T + bias) + residual. A workgroup owns 16 RT output columns and 16 NT
// tokens; its waves split the contraction, so that a CU has several K blocks' loads in flight and no loop is long.
// N = 7168, K = 18432, 16 rows: 26.6 us for 133 MB (5.0 TB/s). One row, N = K = 1024: 3.5 us, the latency of a load, an
// MFMA and the join. Many rows move the operands through L2 instead: 300 rows, N = 2001, K = 2048: 11.8 us.
// ---------------------------------------------------------------------------------------------------------
template <int RT, int NT, int NW, int DEPTH>
__global__ __launch_bounds__(NW * 64) void fg_stream_linear_kernel(const uint8_t* __restrict__ xq, const float* __restrict__ sx,
                                                                   const uint8_t* __restrict__ wq, const float* __restrict__ sw,
                                                                   int64_t M, int64_t N, int64_t K, FgEpilogue ep, void* y,
                                                                   int out_bf16) {
    __shared__ float red[NW][RT * NT * 4][64];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int l16 = lane & 15, g = lane >> 4, z = lane_zero(), source = operand_source(lane);
    const int64_t n0 = (int64_t)blockIdx.x * (16 * RT), m0 = (int64_t)blockIdx.y * (16 * NT);
    const int nkb = (int)(K / BK);
    const int k0 = (int)((int64_t)nkb * wave / NW), k1 = (int)((int64_t)nkb * (wave + 1) / NW);

    const uint8_t* wp[RT];
    const uint8_t* xp[NT];
    int64_t xm[NT];
#pragma unroll
    for (int r = 0; r < RT; r++) {
        const int64_t n = n0 + 16 * r + load_row(lane);         // columns past N read the last one again
        wp[r] = wq + (n < N ? n : N - 1) * K + 16 * load_group(lane);
    }
#pragma unroll
    for (int t = 0; t < NT; t++) {
        const int64_t m = m0 + 16 * t + l16, r = m0 + 16 * t + load_row(lane);     // and rows past M
        xm[t] = m < M ? m : M - 1;
        xp[t] = xq + (r < M ? r : M - 1) * K;
    }
    const float* sp = sw + (n0 / 128) * nkb + z;
    const int left = (int)((M - m0 + 15) / 16);       // token tiles with a row
    const int tiles = left >= NT ? (1 << NT) - 1 : (1 << left) - 1;

    v4f acc[RT][NT];
#pragma unroll
    for (int r = 0; r < RT; r++)
#pragma unroll
        for (int t = 0; t < NT; t++) acc[r][t] = v4f{0.f, 0.f, 0.f, 0.f};

    using Regs = StepRegs<RT, 1, NT, SRC_ROWS>;
    int lk = k0;
    stream_steps<DEPTH, Regs>(k0, k1,
        [&](Regs& b) {
            const int64_t k = (int64_t)lk * BK;
#pragma unroll
            for (int r = 0; r < RT; r++) {
                b.w[r][0] = load_weight(wp[r] + k);
                b.w[r][1] = load_weight(wp[r] + k + 64);
            }
            b.ws[0] = sp[lk];
#pragma unroll
            for (int t = 0; t < NT; t++) b.x[t].load(xp[t], sx + (int64_t)lk * M + xm[t], k, lane);
            lk = lk + 1 < k1 ? lk + 1 : lk;
        },
        [&](Regs& b) { consume<RT, 1, NT, SRC_ROWS, false>(b, 0, tiles, source, acc); });

#pragma unroll
    for (int r = 0; r < RT; r++)
#pragma unroll
        for (int t = 0; t < NT; t++)
#pragma unroll
            for (int q = 0; q < 4; q++) red[wave][(r * NT + t) * 4 + q][lane] = acc[r][t][q];
    __syncthreads();
    for (int id = wave; id < RT * NT; id += NW) {
        const int r = id / NT, t = id % NT;
        const int64_t m = m0 + 16 * t + l16, n = n0 + 16 * r + 4 * g;
        if (m >= M || n >= N) continue;
        v4f v = {0.f, 0.f, 0.f, 0.f}, res = {0.f, 0.f, 0.f, 0.f};
        if (ep.bias) v = fg_load_four(ep.bias, n, ep.bias_bf16, ep.vector_ok, N - n);
        if (ep.residual) res = fg_load_four(ep.residual, m * ep.ld_res + n, ep.residual_bf16, ep.vector_ok, N - n);
#pragma unroll
        for (int q = 0; q < 4; q++) {
            float sum = 0.0f;
#pragma unroll
            for (int w = 0; w < NW; w++) sum += red[w][id * 4 + q][lane];
            v[q] = fg_act_any(ep.act, sum + v[q]) + res[q];
        }
        if (out_bf16) {
            uint16_t* o = (uint16_t*)y + m * N + n;
            if ((N & 3) == 0) {
                *reinterpret_cast<uint2*>(o) = make_uint2(fg_bf16_bits(v[0]) | (fg_bf16_bits(v[1]) << 16),
                                                          fg_bf16_bits(v[2]) | (fg_bf16_bits(v[3]) << 16));
            } else {
#pragma unroll
                for (int q = 0; q < 4; q++)
                    if (n + q < N) o[q] = (uint16_t)fg_bf16_bits(v[q]);
            }
        } else {
            float* o = (float*)y + m * N + n;
            if ((N & 3) == 0) {
                *reinterpret_cast<float4*>(o) = make_float4(v[0], v[1], v[2], v[3]);
            } else {
#pragma unroll
                for (int q = 0; q < 4; q++)
                    if (n + q < N) o[q] = v[q];
            }
        }
    }
}

template <int RT, int NT, int NW, int DEPTH>
hipError_t launch_linear(const uint8_t* xq, const float* sx, const uint8_t* wq, const float* sw, int64_t M, int64_t N,
                         int64_t K, const FgEpilogue& e, void* y, int out_bf16, hipStream_t stream) {
    const dim3 grid((unsigned)((N + 16 * RT - 1) / (16 * RT)), (unsigned)((M + 16 * NT - 1) / (16 * NT)));
    hipLaunchKernelGGL((fg_stream_linear_kernel<RT, NT, NW, DEPTH>), grid, dim3(NW * 64), 0, stream, xq, sx, wq, sw, M, N, K,
                       e, y, out_bf16);
    return hipGetLastError();
}

// Which workgroup a problem gets: columns x rows, waves that split the contraction. A wider tile moves fewer bytes through
// L2 (an operand byte serves more products), a smaller one leaves more workgroups and waves to hide a load's latency
// with; so the widest that still fills the CUs. Boundaries and estimates from 15 weights (N, K = 1024 to 18432) at 17 to
// 1024 rows; in us, N x K at M rows:
//   up to 16 rows   32 columns from N = 4096 on (7168 x 18432, 16: 28.4 against 35.7), 16 below
//   more rows, as long as a workgroup for every CU holds them: 16x16 (512 x 7168, 128: 6.1; 8.5 with 32x32; 2048 x 16384,
//                   32: 13.2; 17.9 with 16x32; but 1024 x 1024, 256, four a CU: 5.3 against 4.1)
//   up to 32 rows   32x32, 16x32 below N = 4096 (7168 x 7168, 32: 14.1 against 21; 3968 x 8192, 32: 11.9 against 14.0 with
//                   16x16)
//   more, by the number of 32x32 tiles:
//     below 384     32x32 (2048 x 16384, 128: 21.1; 28.8 with 32x64)
//     below 800     32x64 (1024 x 4096, 512: 9.7; 10.5 with 32x32, 11.7 with 64x32)
//     above         64x32 (2001 x 2048, 512: 11.6; 14.5 with 32x64), and
//                   64x64 where one round of two a CU holds them all and fills it (7168 x 18432, 200: 75; 98 with 64x32)
enum LinearShape { L16x16, L32x16, L16x32, L32x32, L32x64, L64x32, L64x64 };

int64_t linear_tiles(int64_t M, int64_t N, int cols, int rows) { return ((N + cols - 1) / cols) * ((M + rows - 1) / rows); }

LinearShape linear_shape(int64_t M, int64_t N) {
    const bool wide = N >= 4096;
    if (M <= 16) return wide ? L32x16 : L16x16;
    if (linear_tiles(M, N, 16, 16) <= 256) return L16x16;
    if (M <= 32) return wide ? L32x32 : L16x32;
    const int64_t small = linear_tiles(M, N, 32, 32), large = linear_tiles(M, N, 64, 64);
    if (small < 384) return L32x32;
    if (small < 800) return L32x64;
    return large >= 384 && large <= 512 ? L64x64 : L64x32;
}

}  // namespace

// Estimated time in us of the weight-streaming Linear: launch and latency, then the larger of its tiles' K steps and the
// weights' bytes from HBM (slower the more rows share the waits).
double fg_stream_linear_us(int64_t M, int64_t N, int64_t K) {
    const double steps = (double)(K / BK), bytes = (double)N * (double)K;
    auto larger = [](double a, double b) { return a > b ? a : b; };
    switch (linear_shape(M, N)) {
        case L32x16: return 4.0 + bytes / 5.2e6;
        case L16x16:
        case L16x32: return 4.0 + bytes / 3.0e6;
        case L32x32: return 3.5 + larger(0.6e-3 * steps * (double)linear_tiles(M, N, 32, 32), bytes / 3.7e6);
        case L32x64: return 3.5 + 1.0e-3 * steps * (double)linear_tiles(M, N, 32, 64) + bytes / 17e6;
        case L64x32: return 3.5 + larger(0.83e-3 * steps * (double)linear_tiles(M, N, 64, 32), bytes / 2.5e6);
        case L64x64: return 5.0 + larger(0.52 * steps, bytes / 3.0e6);
    }
    return 0.0;
}

hipError_t fg_launch_stream_linear(const uint8_t* xq, const float* sx, const uint8_t* wq, const float* sw, int64_t M,
                                   int64_t N, int64_t K, const FgEpilogue& e, void* y, int out_bf16, hipStream_t stream) {
    switch (linear_shape(M, N)) {
        case L16x16:
            // two steps ahead where a wave has at least four (1 x 2048 x 16384: 10.7 us against 14.7); with one or two the
            // loads past the end cost 0.2 (16 x 1024 x 1024)
            if (K >= 4096) return launch_linear<1, 1, 8, 2>(xq, sx, wq, sw, M, N, K, e, y, out_bf16, stream);
            return launch_linear<1, 1, 8, 1>(xq, sx, wq, sw, M, N, K, e, y, out_bf16, stream);
        case L32x16: return launch_linear<2, 1, 4, 2>(xq, sx, wq, sw, M, N, K, e, y, out_bf16, stream);
        case L16x32: return launch_linear<1, 2, 8, 1>(xq, sx, wq, sw, M, N, K, e, y, out_bf16, stream);
        case L32x32: return launch_linear<2, 2, 8, 1>(xq, sx, wq, sw, M, N, K, e, y, out_bf16, stream);
        case L32x64: return launch_linear<2, 4, 8, 1>(xq, sx, wq, sw, M, N, K, e, y, out_bf16, stream);
        case L64x32: return launch_linear<4, 2, 4, 1>(xq, sx, wq, sw, M, N, K, e, y, out_bf16, stream);
        case L64x64: break;
    }
    return launch_linear<4, 4, 4, 1>(xq, sx, wq, sw, M, N, K, e, y, out_bf16, stream);
}

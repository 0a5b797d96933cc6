// A Linear of few rows with its epilogue (gfx950): bound by the rate at which the weight's codes stream from HBM
// (see weight_stream.h).
#include "ffn_epilogue.h"
#include "ffn_launch.h"
#include "stream_shape.h"
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

}  // namespace

double fg_stream_linear_us(int64_t M, int64_t N, int64_t K) { return stream_linear_us(M, N, K); }

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

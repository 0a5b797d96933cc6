// The Linear's epilogue: act(sum + bias) + residual in fp32, rounded once when it is stored.
#pragma once
#include "ffn_launch.h"
#include "ffn_math.h"

// The first `count` (up to 4) consecutive elements of f32 or bf16 from element i on, zeros behind them; `whole`: all
// four are there and aligned to their size.
__device__ __forceinline__ v4f fg_load_four(const void* p, int64_t i, int bf16, bool whole, int64_t count) {
    if (whole) {
        if (bf16) {
            const uint2 w = *reinterpret_cast<const uint2*>((const uint16_t*)p + i);
            return v4f{fg_bf16_lo(w.x), fg_bf16_hi(w.x), fg_bf16_lo(w.y), fg_bf16_hi(w.y)};
        }
        return *reinterpret_cast<const v4f*>((const float*)p + i);
    }
    v4f v = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int r = 0; r < 4; r++)
        if (r < count) v[r] = fg_load_elem(p, i + r, bf16);
    return v;
}

// Eight residual elements as loaded: 16 bytes of bf16, or 32 of f32.
struct FgResidual8 {
    uint4 a, b;
    __device__ __forceinline__ void load(const FgEpilogue& ep, int64_t i, bool ok) {
        a = b = make_uint4(0, 0, 0, 0);
        if (!ok) return;
        if (ep.residual_bf16) {
            a = *reinterpret_cast<const uint4*>((const uint16_t*)ep.residual + i);
        } else {
            a = *reinterpret_cast<const uint4*>((const float*)ep.residual + i);
            b = *reinterpret_cast<const uint4*>((const float*)ep.residual + i + 4);
        }
    }
    __device__ __forceinline__ void add(const FgEpilogue& ep, float (&v)[8]) const {
        const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
        for (int e = 0; e < 8; e++)
            v[e] += ep.residual_bf16 ? ((e & 1) ? fg_bf16_hi(w[e >> 1]) : fg_bf16_lo(w[e >> 1])) : __uint_as_float(w[e]);
    }
};

// Epilogue and store of a wave's MSUB x NSUB tiles of 16 x 16 in the MFMA layout (the lane holds row l % 16 and four
// columns of each): 32 rows at a time go through a private LDS region of 32 x WAVE_N floats, and come out as eight
// consecutive columns a lane. So bias, residual and output are read and written in whole rows, and the
// accumulators are out of the registers before the activation's variants need any: applied to the
// accumulators themselves, they spill the 8-wave shapes. With sizes or pointers that forbid 16-byte accesses, a lane
// takes one element at a time, still along the rows, eight elements' loads together. Behind a 256 x 288 tile of the training
// step (M = 4096, N = 18432, K = 7168, power-of-2 scales) 449 us with bias and GELU and 434 with neither, 429 for the
// Fprop: the waves of a tile reach it together, so nothing hides its VALU work (half of it the exponential and the
// reciprocal). An odd width costs 512 x 2001 x 2048
// 26 us instead of 18 on 128 x 128 tiles. (m, n): the tile's first row and column.
template <int WAVE_N, int MSUB, int NSUB>
__device__ __forceinline__ void fg_store_epilogue(const FgEpilogue& ep, const v4f (&acc)[MSUB][NSUB], uint8_t* region, int lane,
                                                  int64_t m, int64_t m_end, int64_t n, int64_t N, void* out, int out_bf16) {
    constexpr int CH = WAVE_N / 4, OCT = WAVE_N / 8;               // 16-byte chunks and groups of eight in a row
    constexpr int STEPS = 32 * OCT / 64, GROUP = STEPS % 4 == 0 ? 4 : 3;
    static_assert(STEPS % GROUP == 0 && MSUB % 2 == 0, "whole groups of rows");
    // 64 columns: chunk c of row r at c ^ (r % 16), free of conflicts both ways. 144: rows of 576 bytes shift by 16 banks,
    // so four rows apart meet, which the chunk's two low bits undo when it is written.
    auto chunk = [&](int r, int c) { return region + (r * CH + (WAVE_N == 64 ? c ^ (r & 15) : c ^ ((r >> 2) & 3))) * 16; };
    const int lrow = lane & 15, g = lane >> 4;
#pragma unroll
    for (int h = 0; h < MSUB / 2; h++) {
        const int64_t m_h = m + 32 * h;
#pragma unroll
        for (int i = 0; i < 2; i++)
#pragma unroll
            for (int j = 0; j < NSUB; j++) *reinterpret_cast<v4f*>(chunk(16 * i + lrow, 4 * j + g)) = acc[2 * h + i][j];
        if (ep.vector_ok) {
#pragma unroll 1
            for (int k0 = 0; k0 < STEPS; k0 += GROUP) {
                FgResidual8 res[GROUP];                             // a group's loads are issued together
#pragma unroll
                for (int k = 0; k < GROUP; k++) {
                    const int f = 64 * (k0 + k) + lane, r = f / OCT, c = f % OCT;
                    res[k].load(ep, (m_h + r) * ep.ld_res + n + 8 * c, ep.residual && m_h + r < m_end && n + 8 * c < N);
                }
#pragma unroll
                for (int k = 0; k < GROUP; k++) {
                    const int f = 64 * (k0 + k) + lane, r = f / OCT, c = f % OCT;
                    const int64_t row = m_h + r, col = n + 8 * c;
                    if (row >= m_end || col >= N) continue;
                    const v4f lo = *reinterpret_cast<const v4f*>(chunk(r, 2 * c)), hi = *reinterpret_cast<const v4f*>(chunk(r, 2 * c + 1));
                    float v[8] = {lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
                    if (ep.bias) {
                        const v4f b0 = fg_load_four(ep.bias, col, ep.bias_bf16, true, 4), b1 = fg_load_four(ep.bias, col + 4, ep.bias_bf16, true, 4);
#pragma unroll
                        for (int e = 0; e < 4; e++) {
                            v[e] += b0[e];
                            v[4 + e] += b1[e];
                        }
                    }
                    if (ep.act == FG_ACT_RELU) {
#pragma unroll
                        for (int e = 0; e < 8; e++) v[e] = fg_act_value<FG_ACT_RELU>(v[e]);
                    } else if (ep.act == FG_ACT_GELU_TANH) {
#pragma unroll
                        for (int e = 0; e < 8; e++) v[e] = fg_act_value<FG_ACT_GELU_TANH>(v[e]);
                    } else if (ep.act == FG_ACT_SILU) {
#pragma unroll
                        for (int e = 0; e < 8; e++) v[e] = fg_act_value<FG_ACT_SILU>(v[e]);
                    }
                    if (ep.residual) res[k].add(ep, v);
                    if (out_bf16) {
                        uint32_t w[4];
#pragma unroll
                        for (int e = 0; e < 4; e++) w[e] = fg_bf16_bits(v[2 * e]) | (fg_bf16_bits(v[2 * e + 1]) << 16);
                        *reinterpret_cast<uint4*>((uint16_t*)out + row * N + col) = make_uint4(w[0], w[1], w[2], w[3]);
                    } else {
                        float* o = (float*)out + row * N + col;
                        *reinterpret_cast<float4*>(o) = make_float4(v[0], v[1], v[2], v[3]);
                        *reinterpret_cast<float4*>(o + 4) = make_float4(v[4], v[5], v[6], v[7]);
                    }
                }
            }
        } else {
#pragma unroll 1
            for (int k0 = 0; k0 < 32 * WAVE_N / 64; k0 += 8) {
                uint32_t res[8], bias[8];                           // as loaded, a group's loads together (in bounds)
                auto at = [&](int k, int64_t& row, int64_t& col) {
                    const int f = 64 * (k0 + k) + lane;
                    row = m_h + f / WAVE_N < m_end ? m_h + f / WAVE_N : m_end - 1;
                    col = n + f % WAVE_N < N ? n + f % WAVE_N : N - 1;
                };
                auto load = [&](uint32_t (&raw)[8], const void* from, int64_t ld, int bf16) {
                    int64_t row, col;
                    if (!from) return;
                    if (bf16) {
#pragma unroll
                        for (int k = 0; k < 8; k++) at(k, row, col), raw[k] = ((const uint16_t*)from)[row * ld + col];
                    } else {
#pragma unroll
                        for (int k = 0; k < 8; k++) at(k, row, col), raw[k] = ((const uint32_t*)from)[row * ld + col];
                    }
                };
                load(res, ep.residual, ep.ld_res, ep.residual_bf16);
                load(bias, ep.bias, 0, ep.bias_bf16);
#pragma unroll
                for (int k = 0; k < 8; k++) {
                    const int f = 64 * (k0 + k) + lane, r = f / WAVE_N, c = f % WAVE_N;
                    const int64_t row = m_h + r, col = n + c;
                    if (row >= m_end || col >= N) continue;
                    float v = *reinterpret_cast<const float*>(chunk(r, c >> 2) + 4 * (c & 3));
                    if (ep.bias) v += __uint_as_float(ep.bias_bf16 ? bias[k] << 16 : bias[k]);
                    v = fg_act_any(ep.act, v);
                    if (ep.residual) v += __uint_as_float(ep.residual_bf16 ? res[k] << 16 : res[k]);
                    if (out_bf16) ((uint16_t*)out)[row * N + col] = (uint16_t)fg_bf16_bits(v);
                    else ((float*)out)[row * N + col] = v;
                }
            }
        }
    }
}

// Host arithmetic of the Linear of few rows: the workgroup that a problem gets, and its estimated time. No HIP: the
// boundaries are numbers of workgroups measured on the 256 CUs of an MI355X.
#pragma once
#include <stdint.h>

namespace {

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

inline int64_t linear_tiles(int64_t M, int64_t N, int cols, int rows) { return ((N + cols - 1) / cols) * ((M + rows - 1) / rows); }

inline LinearShape linear_shape(int64_t M, int64_t N) {
    const bool wide = N >= 4096;
    if (M <= 16) return wide ? L32x16 : L16x16;
    if (linear_tiles(M, N, 16, 16) <= 256) return L16x16;
    if (M <= 32) return wide ? L32x32 : L16x32;
    const int64_t small = linear_tiles(M, N, 32, 32), large = linear_tiles(M, N, 64, 64);
    if (small < 384) return L32x32;
    if (small < 800) return L32x64;
    return large >= 384 && large <= 512 ? L64x64 : L64x32;
}

// Estimated time in us: launch and latency, then the larger of the tiles' K steps and the weights' bytes from HBM (slower
// the more rows share the waits), and no less than reading both operands takes: the activations are the larger one where
// the output is narrow (N = 8, K = 16384, in us: 4096 rows 14.3, estimated 14.7; 16384 rows 48.9 and 48.2). Many 64x32
// tiles on a short contraction pay for their joins and stores as well (K = 128, in us: 8192 x 1024 15.5 and on tiles 10.3, where the
// steps alone would be 6.9; K = 512: 1024 x 2944 10.6 and 9.0, where they would be 8.4).
inline double stream_linear_us(int64_t M, int64_t N, int64_t K) {
    const double steps = (double)(K / 128), bytes = (double)N * (double)K;
    auto larger = [](double a, double b) { return a > b ? a : b; };
    double us = 0.0;
    switch (linear_shape(M, N)) {
        case L32x16: us = 4.0 + bytes / 5.2e6; break;
        case L16x16:
        case L16x32: us = 4.0 + bytes / 3.0e6; break;
        case L32x32: us = 3.5 + larger(0.6e-3 * steps * (double)linear_tiles(M, N, 32, 32), bytes / 3.7e6); break;
        case L32x64: us = 3.5 + 1.0e-3 * steps * (double)linear_tiles(M, N, 32, 64) + bytes / 17e6; break;
        case L64x32: us = 3.5 + larger(larger(0.83e-3 * steps, 2.3e-3 + 0.62e-3 * steps) * (double)linear_tiles(M, N, 64, 32), bytes / 2.5e6); break;
        case L64x64: us = 5.0 + larger(0.52 * steps, bytes / 3.0e6); break;
    }
    return larger(us, 3.5 + (bytes + (double)M * (double)K) / 6.0e6);
}

}  // namespace

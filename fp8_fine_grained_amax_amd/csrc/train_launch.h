// Launchers of the operators at the two ends of a Linear's training step (arguments already validated by train_api.cpp).
#pragma once
#include <hip/hip_runtime_api.h>
#include <stdint.h>

#include "fp8fg_train.h"

// Widest row of the norm: three groups of eight columns to each of a workgroup's 768 threads.
constexpr int64_t kFgNormMaxCols = 3 * 8 * 768;

struct FgNorm {
    const void *x, *gamma, *beta;
    uint8_t *q_cols, *q_rows;
    float *s_cols, *s_rows, *mean, *rstd;
    uint16_t* y;
    int64_t ld, rows, cols;
    float eps;
    int x_bf16, w_bf16, layer, pow2;
};

struct FgNormBwd {
    const void *x, *gamma, *dy, *dres;
    const float *mean, *rstd;
    void* dx;
    float *dgamma, *dbeta, *partial;
    int64_t ld_x, ld_dy, ld_dres, rows, cols;
    int x_bf16, w_bf16, dy_bf16, dres_bf16, dx_bf16, layer, accumulate;
};

struct FgOrtho {
    const void* g;
    uint16_t* out;
    void* workspace;
    int64_t ld, batch, N, K;
    float a, b, c, eps, scale;
    int g_bf16, steps;
};

hipError_t fg_launch_norm(const FgNorm& p, hipStream_t stream);
hipError_t fg_launch_norm_bwd(const FgNormBwd& p, hipStream_t stream);
int64_t fg_norm_bwd_partials(int64_t rows, int64_t cols);      // rows of partial sums: of dgamma's, and as many of dbeta's; 0 with few rows
hipError_t fg_launch_orthogonalize(const FgOrtho& p, hipStream_t stream);
int64_t fg_ortho_workspace_bytes(int64_t batch, int64_t N, int64_t K);

// Status of a launch; the HIP code is kept for fg_last_hip_error() on this thread.
fg_status fg_status_from_hip(hipError_t e);

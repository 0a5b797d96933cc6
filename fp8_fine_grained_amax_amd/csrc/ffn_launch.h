// Launchers of the feed-forward operators (arguments already validated by ffn_api.cpp).
#pragma once
#include <hip/hip_runtime_api.h>
#include <stdint.h>

#include "fp8fg_ffn.h"

// Epilogue of a Linear: y = act(z + bias) + residual.
struct FgEpilogue {
    const void* bias;
    const void* residual;
    int64_t ld_res;
    int bias_bf16, residual_bf16, act;
    int vector_ok;      // bias, residual and output allow 16-byte accesses at every eighth column
};

struct FgMoe {
    const uint16_t* x;
    const int32_t* ids;
    const float* weights;
    const uint8_t* w1q;
    const uint8_t* w2q;
    const float* s1;
    const float* s2;
    void* workspace;
    void* y;
    int64_t ld_x, ld_y, T, H, I;
    int topk, E, act, pow2, out_bf16;
};

struct FgActBwd {
    const uint8_t* zq;
    const float* sz;
    const void* da;
    int64_t ld_da, rows, F;
    int da_bf16, act, gated, pow2;
    uint8_t *dzq_cols, *dzq_rows, *aq_rows;
    float *sdz_cols, *sdz_rows, *sa_rows, *dbias, *partial;
};

// Estimated times in us of the two ways to compute a Linear with its epilogue: the smaller one is taken.
double fg_stream_linear_us(int64_t M, int64_t N, int64_t K);
double fg_gemm_epilogue_us(int64_t M, int64_t N, int64_t K);

hipError_t fg_launch_gemm_fprop_epilogue(const uint8_t* xq, const float* sx, const uint8_t* wq, const float* sw, int64_t M,
                                         int64_t N, int64_t K, const FgEpilogue& e, void* y, int out_bf16, int pow2,
                                         hipStream_t stream);
hipError_t fg_launch_stream_linear(const uint8_t* xq, const float* sx, const uint8_t* wq, const float* sw, int64_t M,
                                   int64_t N, int64_t K, const FgEpilogue& e, void* y, int out_bf16, hipStream_t stream);
hipError_t fg_launch_act_fwd(const uint16_t* z, int64_t rows, int64_t F, int64_t ld, int act, int gated, int pow2,
                             uint8_t* zq, float* sz, uint8_t* aq, float* sa, hipStream_t stream);
hipError_t fg_launch_act_bwd(const FgActBwd& p, hipStream_t stream);
hipError_t fg_launch_moe_few_tokens(const FgMoe& p, hipStream_t stream);
int64_t fg_moe_workspace_bytes(int64_t T, int topk, int64_t H, int64_t I);
int64_t fg_act_bwd_partial_rows(int64_t rows);

// Status of a launch; the HIP code is kept for fg_last_hip_error() on this thread.
fg_status fg_status_from_hip(hipError_t e);

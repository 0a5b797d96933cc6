// The argument checks of fp8_fine_grained_amax_amd/csrc/ffn_api.cpp with every launcher replaced by a stub that
// counts its calls, driven over extreme extents: each call either returns a refusal and reaches no launcher, or
// FG_OK and reaches exactly one (none for empty problems), and no check overflows an integer.
#include <stdint.h>
#include <stdio.h>

#include "ffn_launch.h"

namespace {
int g_calls = 0;
hipError_t g_ret = hipSuccess;
int g_failures = 0;
hipError_t hit() {
    g_calls++;
    return g_ret;
}
}  // namespace

double fg_stream_linear_us(int64_t M, int64_t, int64_t) { return (double)M; }
double fg_gemm_epilogue_us(int64_t, int64_t, int64_t) { return 64.0; }
hipError_t fg_launch_gemm_fprop_epilogue(const uint8_t*, const float*, const uint8_t*, const float*, int64_t, int64_t, int64_t,
                                         const FgEpilogue&, void*, int, int, hipStream_t) { return hit(); }
hipError_t fg_launch_stream_linear(const uint8_t*, const float*, const uint8_t*, const float*, int64_t, int64_t, int64_t,
                                   const FgEpilogue&, void*, int, hipStream_t) { return hit(); }
hipError_t fg_launch_act_fwd(const uint16_t*, int64_t, int64_t, int64_t, int, int, int, uint8_t*, float*, uint8_t*, float*,
                             hipStream_t) { return hit(); }
hipError_t fg_launch_act_bwd(const FgActBwd&, hipStream_t) { return hit(); }
hipError_t fg_launch_moe_few_tokens(const FgMoe&, hipStream_t) { return hit(); }
int64_t fg_moe_workspace_bytes(int64_t T, int topk, int64_t, int64_t I) { return T * topk * I * 4; }
int64_t fg_act_bwd_partial_rows(int64_t rows) { return rows > 128 ? (rows + 127) / 128 : 0; }
fg_status fg_status_from_hip(hipError_t e) { return e == hipSuccess ? FG_OK : FG_ERR_HIP; }

static void check(const char* what, fg_status s, bool empty) {
    const int want = s == FG_OK ? (empty ? 0 : 1) : s == FG_ERR_HIP ? 1 : 0;
    if (g_calls != want) {
        printf("%s: status %d with %d launches\n", what, (int)s, g_calls);
        g_failures++;
    }
    g_calls = 0;
}

int main() {
    const int64_t sizes[] = {INT64_MIN, -1, 0, 1, 8, 100, 128, 256, 1 << 20, 1 << 24, 1 << 30, (1LL << 31) + 128, 1LL << 40, 1LL << 62, INT64_MAX};
    uint8_t* q = (uint8_t*)(uintptr_t)(1 << 20);
    float* s = (float*)(uintptr_t)(2 << 20);
    void* p = (void*)(uintptr_t)(3 << 20);
    void* other = (void*)(uintptr_t)(4 << 20);
    for (int64_t a : sizes)
        for (int64_t b : sizes)
            for (int64_t c : sizes) {
                check("linear", fg_fp8_gemm_fprop_epilogue(q, s, q, s, a, b, c, p, FG_OUT_BF16, FG_ACT_SILU, p, FG_OUT_F32, b, other,
                                                           FG_OUT_BF16, FG_SCALE_FP32, nullptr), a == 0 || b == 0);
                for (int gated = 0; gated < 2; gated++) {
                    check("act fwd", fg_act_checkpoint_fwd(p, a, b, c, FG_ACT_SILU, gated, FG_SCALE_POW2, q, s, q, s, nullptr),
                          a == 0 || b == 0);
                    check("act bwd", fg_act_checkpoint_bwd(q, s, p, FG_OUT_F32, c, a, b, FG_ACT_RELU, gated, FG_SCALE_FP32, q, s, q, s,
                                                           q, s, s, p, INT64_MAX, nullptr), b == 0);
                    (void)fg_act_checkpoint_bwd_workspace(a, b, gated);
                }
                check("moe", fg_moe_few_tokens(p, c, (const int32_t*)p, s, 8, 4, q, s, q, s, 16, a, b, FG_ACT_SILU, FG_SCALE_FP32, p,
                                               INT64_MAX, other, c, FG_OUT_F32, nullptr), a == 0);
                check("moe tokens", fg_moe_few_tokens(p, 256, (const int32_t*)p, s, a, (int32_t)b, q, s, q, s, (int32_t)c, 256, 128,
                                                      FG_ACT_SILU, FG_SCALE_FP32, p, INT64_MAX, other, 256, FG_OUT_F32, nullptr), a == 0);
                (void)fg_moe_few_tokens_workspace(a, (int32_t)b, c, a);
            }
    g_ret = hipErrorInvalidValue;
    check("launch error", fg_act_checkpoint_fwd(p, 8, 128, 128, FG_ACT_SILU, 0, FG_SCALE_FP32, q, s, q, s, nullptr), false);
    if (g_failures) return 1;
    printf("ffn host driver done\n");
    return 0;
}

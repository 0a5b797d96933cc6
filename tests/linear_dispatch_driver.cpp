// Which launcher fg_fp8_gemm_fprop_epilogue (fp8_fine_grained_amax_amd/csrc/ffn_api.cpp) takes, and what it refuses: the
// launchers are replaced by stubs that note their name. Arguments: pairs of estimates and sizes, one question a line on
// stdin "stream_us tiles_us M N K"; one answer a line: the status and the launcher ("stream", "tiles" or "-").
#include <stdint.h>
#include <stdio.h>

#include "ffn_launch.h"

namespace {
const char* g_launched = "-";
double g_stream_us = 0, g_tiles_us = 0;
}  // namespace

double fg_stream_linear_us(int64_t, int64_t, int64_t) { return g_stream_us; }
double fg_gemm_epilogue_us(int64_t, int64_t, int64_t) { return g_tiles_us; }
hipError_t fg_launch_gemm_fprop_epilogue(const uint8_t*, const float*, const uint8_t*, const float*, int64_t, int64_t, int64_t,
                                         const FgEpilogue&, void*, int, int, hipStream_t) { return g_launched = "tiles", hipSuccess; }
hipError_t fg_launch_stream_linear(const uint8_t*, const float*, const uint8_t*, const float*, int64_t, int64_t, int64_t,
                                   const FgEpilogue&, void*, int, hipStream_t) { return g_launched = "stream", hipSuccess; }
hipError_t fg_launch_act_fwd(const uint16_t*, int64_t, int64_t, int64_t, int, int, int, uint8_t*, float*, uint8_t*, float*,
                             hipStream_t) { return hipSuccess; }
hipError_t fg_launch_act_bwd(const FgActBwd&, hipStream_t) { return hipSuccess; }
hipError_t fg_launch_moe_few_tokens(const FgMoe&, hipStream_t) { return hipSuccess; }
int64_t fg_moe_workspace_bytes(int64_t, int, int64_t, int64_t) { return 0; }
int64_t fg_act_bwd_partial_rows(int64_t) { return 0; }
fg_status fg_status_from_hip(hipError_t e) { return e == hipSuccess ? FG_OK : FG_ERR_HIP; }

int main() {
    uint8_t* q = (uint8_t*)(uintptr_t)(1 << 20);
    float* s = (float*)(uintptr_t)(2 << 20);
    void* y = (void*)(uintptr_t)(4 << 20);
    long long M, N, K;
    while (scanf("%lf %lf %lld %lld %lld", &g_stream_us, &g_tiles_us, &M, &N, &K) == 5) {
        g_launched = "-";
        const fg_status r = fg_fp8_gemm_fprop_epilogue(q, s, q, s, M, N, K, nullptr, FG_OUT_F32, FG_ACT_NONE, nullptr, FG_OUT_F32, N,
                                                       y, FG_OUT_BF16, FG_SCALE_FP32, nullptr);
        printf("%d %s\n", (int)r, g_launched);
    }
    return 0;
}

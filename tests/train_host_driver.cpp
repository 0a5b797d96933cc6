// Drives the argument checks of train_api.cpp with extreme sizes, its launchers replaced by recorders (built under
// sanitizers by tests/test_train_abi.py).
#include <cmath>
#include <cstdio>
#include <cstdlib>
#include <limits>

#include "train_launch.h"

static int launches = 0;
static FgOrtho last_ortho;
hipError_t fg_launch_norm(const FgNorm&, hipStream_t) { return launches++, hipSuccess; }
hipError_t fg_launch_norm_bwd(const FgNormBwd&, hipStream_t) { return launches++, hipSuccess; }
int64_t fg_norm_bwd_partials(int64_t rows, int64_t) { return rows < 256 ? rows : 256; }
hipError_t fg_launch_orthogonalize(const FgOrtho& p, hipStream_t) { return last_ortho = p, launches++, hipSuccess; }
int64_t fg_ortho_workspace_bytes(int64_t batch, int64_t N, int64_t K) { return batch * (N + 63) / 64 * (K + 63); }
fg_status fg_status_from_hip(hipError_t e) { return e == hipSuccess ? FG_OK : FG_ERR_HIP; }

#define EXPECT(cond)                                              \
    if (!(cond)) {                                                \
        std::printf("line %d: %s\n", __LINE__, #cond);            \
        std::exit(1);                                             \
    }

int main() {
    const int64_t sizes[] = {0, 1, 127, 128, 18432, 18560, 65536, 65537, 1LL << 25, (1LL << 25) + 1, 1LL << 40, INT64_MAX - 1, INT64_MAX};
    char* a = (char*)(1 << 20);
    float* f = (float*)a;
    int accepted = 0;
    for (int64_t rows : sizes)
        for (int64_t cols : sizes)
            for (int64_t ld : {cols, INT64_MAX})
                for (int type : {0, 1})
                    for (int tokens : {0, 1}) {
                        const int before = launches;
                        const fg_status s = fg_norm_quantize(a, (fg_out_dtype)type, ld, rows, cols, FG_NORM_LAYER, a, a, FG_OUT_F32, 1e-5f,
                                                             FG_SCALE_FP32, (uint8_t*)a, f, tokens ? (uint8_t*)a : nullptr, tokens ? f : nullptr, a, f, f, nullptr);
                        EXPECT((launches > before) == (s == FG_OK && rows > 0 && cols > 0));
                        const int64_t need = fg_norm_bwd_workspace(rows, cols);
                        EXPECT(need >= 0 && need <= 2 * 256 * 18432 * 4);
                        const int middle = launches;
                        const fg_status b = fg_norm_bwd(a, (fg_out_dtype)type, ld, f, f, a, FG_OUT_F32, a, FG_OUT_BF16, cols, a + 4096, FG_OUT_BF16, ld,
                                                        rows, cols, FG_NORM_RMS, a + 64, FG_OUT_F32, f, f, 0, a, need, nullptr);
                        EXPECT(launches == middle || b == FG_OK);
                        accepted += s == FG_OK && b == FG_OK;
                    }
    for (int64_t batch : sizes)
        for (int64_t n : sizes)
            for (int64_t k : sizes) {
                const int64_t need = fg_orthogonalize_workspace(batch, n, k);
                EXPECT(need >= 0);
                const int before = launches;
                const fg_status s = fg_orthogonalize(a, FG_OUT_F32, k, batch, n, k, 5, 3.4445f, -4.775f, 2.0315f, 1e-7f, 1.0f, a, a, need, nullptr);
                EXPECT((launches > before) == (need > 0) && (s == FG_OK || s == FG_ERR_UNSUPPORTED_SHAPE));
                accepted += s == FG_OK;
            }
    // coefficients: finite ones are judged without overflow, others are refused
    const float inf = std::numeric_limits<float>::infinity(), big = std::numeric_limits<float>::max();
    const float values[] = {0.0f, -0.0f, 1.0f, 1.5f, -0.5f, 3.4445f, -4.775f, 2.0315f, 1e-30f, -1e30f, big, -big, inf, NAN};
    for (float x : values)
        for (float y : values)
            for (float z : values)
                for (int steps : {1, 5, 32}) {
                    const fg_status s = fg_orthogonalize(a, FG_OUT_BF16, 8, 1, 8, 8, steps, x, y, z, 1e-7f, 1.0f, a, a, 1 << 20, nullptr);
                    EXPECT(s == FG_OK || s == FG_ERR_INVALID_ARG);
                    EXPECT(s != FG_OK || (std::fabs(y) < 30 && std::fabs(z) < 30 && std::isfinite(x)));
                    accepted += s == FG_OK;
                }
    EXPECT(accepted > 20);
    std::printf("train host driver done, %d launches\n", launches);
    return 0;
}

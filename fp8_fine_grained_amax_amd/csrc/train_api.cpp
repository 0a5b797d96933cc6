// C-ABI entry points of the operators at the two ends of a Linear's training step: host-side argument checks, then the
// launches on the caller's stream. Declarations, layouts and error behaviour: include/fp8fg_train.h.
#include "fp8fg_train.h"

#include <algorithm>
#include <cmath>

#include "train_launch.h"

namespace {

constexpr int64_t kMaxRows = 1LL << 25;
constexpr int64_t kMaxStride = 1LL << 40;
constexpr int64_t kMaxSide = 65536;              // of a weight: 32-bit offsets inside a tile of its padded copies
constexpr int64_t kMaxBlocks = (1LL << 24) - 1;  // 64 x 64 blocks of all matrices: a launch has less than 2^32 threads
constexpr int64_t kMaxBatch = 65535;             // a grid's y
constexpr int kMaxSteps = 32;

bool aligned(const void* p, uintptr_t n) { return ((uintptr_t)p & (n - 1)) == 0; }
bool valid_type(int o) { return o == FG_OUT_F32 || o == FG_OUT_BF16; }
bool valid_kind(int k) { return k == FG_NORM_LAYER || k == FG_NORM_RMS; }
int64_t size_of(int type) { return type == FG_OUT_F32 ? 4 : 2; }
int64_t cdiv(int64_t a, int64_t b) { return a / b + (a % b != 0); }
// Row stride of a matrix read in 16-byte pieces.
bool odd_stride(int64_t ld, int type) { return ld * size_of(type) % 16 != 0; }

// Largest |a s + b s^3 + c s^5| for 0 <= s <= u: at the end or where the slope is 0.
double largest(double a, double b, double c, double u) {
    auto value = [&](double s) { return std::fabs(s * (a + s * s * (b + s * s * c))); };
    double most = value(u);
    auto consider = [&](double square) {
        if (square > 0 && square < u * u) most = std::max(most, value(std::sqrt(square)));
    };
    if (c != 0) {
        const double root = 9 * b * b - 20 * a * c;
        if (root >= 0) {
            consider((-3 * b + std::sqrt(root)) / (10 * c));
            consider((-3 * b - std::sqrt(root)) / (10 * c));
        }
    } else if (b != 0) {
        consider(-a / (3 * b));
    }
    return most;
}

// Whether the steps keep every product inside fp16's range: |X| below u, |A| below u^2, |B| below |a| + |b| u^2 + |c| u^4.
bool in_range(double a, double b, double c, int steps) {
    double u = 1.0;
    for (int s = 0; s < steps; s++) {
        if (!(std::fabs(a) + std::fabs(b) * u * u + std::fabs(c) * u * u * u * u < 30.0)) return false;
        u = std::max(u, largest(a, b, c, u));
        if (!(u < 5.0)) return false;
    }
    return true;
}

bool side_ok(int64_t batch, int64_t N, int64_t K) {
    return N <= kMaxSide && K <= kMaxSide && batch <= kMaxBatch && batch <= kMaxBlocks / (cdiv(N, 64) * cdiv(K, 64));
}

}  // namespace

extern "C" {

fg_status fg_norm_quantize(const void* x, fg_out_dtype x_type, int64_t ld_x, int64_t rows, int64_t cols, fg_norm_kind kind,
                           const void* gamma, const void* beta, fg_out_dtype weight_type, float eps, fg_scale_mode mode,
                           uint8_t* q_cols, float* s_cols, uint8_t* q_rows, float* s_rows, void* y, float* mean, float* rstd,
                           hipStream_t stream) {
    if (rows < 0 || cols < 0 || ld_x < cols || !valid_type(x_type) || !valid_type(weight_type) || !valid_kind(kind) ||
        (mode != FG_SCALE_FP32 && mode != FG_SCALE_POW2) || !std::isfinite(eps) || !(eps > 0))
        return FG_ERR_INVALID_ARG;
    if (cols % 128 != 0 || cols > kFgNormMaxCols || rows > kMaxRows || ld_x > kMaxStride) return FG_ERR_UNSUPPORTED_SHAPE;
    if (rows == 0 || cols == 0) return FG_OK;
    if (!x || !gamma || !q_cols || !s_cols || !q_rows != !s_rows) return FG_ERR_INVALID_ARG;
    if (q_rows && (!rstd || (kind == FG_NORM_LAYER && !mean))) return FG_ERR_INVALID_ARG;
    // tiles along the rows: 512 threads to 128 x 128 elements
    if (q_rows && (rows % 128 != 0 || rows * cols >= 1LL << 36)) return FG_ERR_UNSUPPORTED_SHAPE;
    if (!aligned(x, 16) || odd_stride(ld_x, x_type) || !aligned(gamma, 16) || !aligned(beta, 16) || !aligned(q_cols, 16) ||
        !aligned(q_rows, 16) || !aligned(y, 16) || !aligned(s_cols, 4) || !aligned(s_rows, 4) || !aligned(mean, 4) ||
        !aligned(rstd, 4))
        return FG_ERR_MISALIGNED;
    FgNorm p{};
    p.x = x; p.gamma = gamma; p.beta = beta;
    p.q_cols = q_cols; p.q_rows = q_rows; p.s_cols = s_cols; p.s_rows = s_rows; p.mean = mean; p.rstd = rstd;
    p.y = (uint16_t*)y;
    p.ld = ld_x; p.rows = rows; p.cols = cols; p.eps = eps;
    p.x_bf16 = x_type == FG_OUT_BF16; p.w_bf16 = weight_type == FG_OUT_BF16;
    p.layer = kind == FG_NORM_LAYER; p.pow2 = mode == FG_SCALE_POW2;
    return fg_status_from_hip(fg_launch_norm(p, stream));
}

int64_t fg_norm_bwd_workspace(int64_t rows, int64_t cols) {
    if (rows < 1 || rows > kMaxRows || cols < 1 || cols > kFgNormMaxCols || cols % 128 != 0) return 0;
    return 2 * fg_norm_bwd_partials(rows, cols) * cols * (int64_t)sizeof(float);
}

fg_status fg_norm_bwd(const void* x, fg_out_dtype x_type, int64_t ld_x, const float* mean, const float* rstd, const void* gamma,
                      fg_out_dtype weight_type, const void* dy, fg_out_dtype dy_type, int64_t ld_dy, const void* dres,
                      fg_out_dtype dres_type, int64_t ld_dres, int64_t rows, int64_t cols, fg_norm_kind kind, void* dx,
                      fg_out_dtype dx_type, float* dgamma, float* dbeta, int accumulate, void* workspace,
                      int64_t workspace_bytes, hipStream_t stream) {
    if (rows < 0 || cols < 0 || ld_x < cols || ld_dy < cols || !valid_type(x_type) || !valid_type(weight_type) ||
        !valid_type(dy_type) || !valid_type(dx_type) || !valid_kind(kind) || (accumulate != 0 && accumulate != 1) ||
        workspace_bytes < 0 || (dres && (!valid_type(dres_type) || ld_dres < cols)))
        return FG_ERR_INVALID_ARG;
    if (cols % 128 != 0 || cols > kFgNormMaxCols || rows > kMaxRows || ld_x > kMaxStride || ld_dy > kMaxStride ||
        (dres && ld_dres > kMaxStride))
        return FG_ERR_UNSUPPORTED_SHAPE;
    if (cols == 0 || (rows == 0 && ((!dgamma && !dbeta) || accumulate))) return FG_OK;
    if (rows > 0 && (!x || !rstd || (kind == FG_NORM_LAYER && !mean) || !gamma || !dy || !dx)) return FG_ERR_INVALID_ARG;
    // x and dy may be read again after dx is written
    if (rows > 0 && (dx == x || dx == dy)) return FG_ERR_INVALID_ARG;
    // dx as its own addend is read where it is written; with another type or stride it would be overwritten first
    if (dres && dres == dx && (dres_type != dx_type || ld_dres != cols)) return FG_ERR_INVALID_ARG;
    const int64_t need = dgamma || dbeta ? fg_norm_bwd_workspace(rows, cols) : 0;
    if (need > 0 && (!workspace || workspace_bytes < need)) return FG_ERR_INVALID_ARG;
    if (!aligned(x, 16) || odd_stride(ld_x, x_type) || !aligned(gamma, 16) || !aligned(dy, 16) || odd_stride(ld_dy, dy_type) ||
        (dres && (!aligned(dres, 16) || odd_stride(ld_dres, dres_type))) || !aligned(dx, 16) || !aligned(mean, 4) ||
        !aligned(rstd, 4) || !aligned(dgamma, 4) || !aligned(dbeta, 4) || (need > 0 && !aligned(workspace, 16)))
        return FG_ERR_MISALIGNED;
    FgNormBwd p{};
    p.x = x; p.gamma = gamma; p.dy = dy; p.dres = dres; p.mean = mean; p.rstd = rstd; p.dx = dx;
    p.dgamma = dgamma; p.dbeta = dbeta; p.partial = need > 0 ? (float*)workspace : nullptr;
    p.ld_x = ld_x; p.ld_dy = ld_dy; p.ld_dres = ld_dres; p.rows = rows; p.cols = cols;
    p.x_bf16 = x_type == FG_OUT_BF16; p.w_bf16 = weight_type == FG_OUT_BF16; p.dy_bf16 = dy_type == FG_OUT_BF16;
    p.dres_bf16 = dres && dres_type == FG_OUT_BF16; p.dx_bf16 = dx_type == FG_OUT_BF16;
    p.layer = kind == FG_NORM_LAYER; p.accumulate = accumulate;
    return fg_status_from_hip(fg_launch_norm_bwd(p, stream));
}

int64_t fg_orthogonalize_workspace(int64_t batch, int64_t N, int64_t K) {
    if (batch < 1 || N < 1 || K < 1 || !side_ok(batch, N, K)) return 0;
    return fg_ortho_workspace_bytes(batch, N, K);
}

fg_status fg_orthogonalize(const void* g, fg_out_dtype g_type, int64_t ld_g, int64_t batch, int64_t N, int64_t K, int steps,
                           float a, float b, float c, float eps, float scale, void* out, void* workspace,
                           int64_t workspace_bytes, hipStream_t stream) {
    if (batch < 0 || N < 0 || K < 0 || ld_g < K || !valid_type(g_type) || steps < 1 || steps > kMaxSteps || workspace_bytes < 0 ||
        !std::isfinite(a) || !std::isfinite(b) || !std::isfinite(c) || !std::isfinite(eps) || !(eps > 0) ||
        !std::isfinite(scale) || !in_range(a, b, c, steps))
        return FG_ERR_INVALID_ARG;
    if (batch == 0 || N == 0 || K == 0) return FG_OK;
    if (!side_ok(batch, N, K) || ld_g > kMaxStride) return FG_ERR_UNSUPPORTED_SHAPE;
    if (!g || !out || !workspace || workspace_bytes < fg_orthogonalize_workspace(batch, N, K)) return FG_ERR_INVALID_ARG;
    if (!aligned(g, (uintptr_t)size_of(g_type)) || !aligned(out, 2) || !aligned(workspace, 256)) return FG_ERR_MISALIGNED;
    FgOrtho p{};
    p.g = g; p.out = (uint16_t*)out; p.workspace = workspace;
    p.ld = ld_g; p.batch = batch; p.N = N; p.K = K;
    p.a = a; p.b = b; p.c = c; p.eps = eps; p.scale = scale;
    p.g_bf16 = g_type == FG_OUT_BF16; p.steps = steps;
    return fg_status_from_hip(fg_launch_orthogonalize(p, stream));
}

}  // extern "C"

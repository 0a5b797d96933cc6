// C-ABI entry points of the feed-forward operators: host-side argument checks, then the launches on the
// caller's stream. Declarations, layouts and error behaviour: include/fp8fg_ffn.h.
#include "fp8fg_ffn.h"

#include <stdlib.h>

#include "ffn_launch.h"

namespace {

constexpr int64_t kMaxThreads = (1LL << 32) - 1; // of a launch along one dimension
constexpr int64_t kMaxContraction = 1LL << 24;   // as in the other GEMMs: 32-bit operand offsets
constexpr int64_t kMaxCols = 1LL << 23;          // 32-bit offsets inside a 128-row block of up to 2 F codes or F fp32 values
constexpr int64_t kMaxRows = 1LL << 25;          // and inside a 128-column block of a tiling along the rows
constexpr int64_t kMaxStride = 1LL << 40;
constexpr int64_t kMaxExpertDim = 1LL << 20;
constexpr int64_t kMaxTokens = 64;
constexpr int64_t kMaxStreamRows = 65535 * 16;   // a grid's y, of 16 rows at least
// Past 4096 rows only weights of few columns are streamed. There the estimates were measured on both sides (4097 to
// 262144 rows, K = 128 to 16384), and nothing streams for more than 6% longer than the tiles take: in us, streaming and on
// tiles, 8192 rows of 64 x 7168 21 and 45, of 256 x 512 9.2 and 8.7; 65536 of 256 x 1024, which go to the tiles, 69 and 29.
// On more columns they put the tiles too far behind: 5000 rows of 512 x 2048 count 20.2 and 20.4 and take 22.2 and 16.7.
constexpr int64_t kFewCols = 256, kFewColsRows = 4096;
constexpr int64_t kMaxStreamCols = 1LL << 26;    // kMaxThreads: 512 threads to 16 columns
constexpr int kMaxTopk = 32, kMaxExperts = 2048;

bool aligned(const void* p, uintptr_t n) { return ((uintptr_t)p & (n - 1)) == 0; }
bool valid_mode(int m) { return m == FG_SCALE_FP32 || m == FG_SCALE_POW2; }
bool valid_type(int o) { return o == FG_OUT_F32 || o == FG_OUT_BF16; }
bool valid_act(int a) { return a >= FG_ACT_NONE && a <= FG_ACT_SILU; }
int64_t cdiv(int64_t a, int64_t b) { return a / b + (a % b != 0); }
bool prod_over(int64_t a, int64_t b, int64_t limit) { return a != 0 && b > limit / a; }
// Whether a Linear's launch on GEMM tiles would have too many threads: 256 to 128x128 outputs. The larger shapes are taken
// where they need no more; a forced one may need up to 768 to 256x192.
bool linear_threads_over(int64_t M, int64_t N) {
    return prod_over(cdiv(M, 128), cdiv(N, 128), kMaxThreads / 256) ||
           (getenv("FG_GEMM_TILE") && prod_over(cdiv(M, 256), cdiv(N, 192), kMaxThreads / 768));
}
uintptr_t size_of(int type) { return type == FG_OUT_F32 ? 4 : 2; }

}  // namespace

extern "C" {

fg_status fg_fp8_gemm_fprop_epilogue(const uint8_t* xq, const float* sx, const uint8_t* wq, const float* sw, int64_t M,
                                     int64_t N, int64_t K, const void* bias, fg_out_dtype bias_type, fg_act act,
                                     const void* residual, fg_out_dtype residual_type, int64_t ld_res, void* y,
                                     fg_out_dtype out, fg_scale_mode scales, hipStream_t stream) {
    if (M < 0 || N < 0 || K < 0 || !valid_mode(scales) || !valid_type(out) || !valid_act(act)) return FG_ERR_INVALID_ARG;
    if ((bias && !valid_type(bias_type)) || (residual && (!valid_type(residual_type) || ld_res < N)))
        return FG_ERR_INVALID_ARG;
    if (M == 0 || N == 0) return FG_OK;
    if (!y || (K > 0 && (!xq || !sx || !wq || !sw))) return FG_ERR_INVALID_ARG;
    // y as its own residual is read where it is written; with another type or stride it would be overwritten first
    if (residual == y && (residual_type != out || ld_res != N)) return FG_ERR_INVALID_ARG;
    if (K % 128 != 0 || K > kMaxContraction || (residual && ld_res > kMaxStride) || linear_threads_over(M, N))
        return FG_ERR_UNSUPPORTED_SHAPE;
    if (!aligned(xq, 16) || !aligned(wq, 16) || !aligned(y, 16) || !aligned(sx, 4) || !aligned(sw, 4) ||
        (bias && !aligned(bias, size_of(bias_type))) || (residual && !aligned(residual, size_of(residual_type))))
        return FG_ERR_MISALIGNED;
    const bool vector_ok = N % 8 == 0 && (!bias || aligned(bias, 16)) &&
                           (!residual || (ld_res % 8 == 0 && aligned(residual, 16)));
    const FgEpilogue e{bias, residual, ld_res, bias && bias_type == FG_OUT_BF16,
                       residual && residual_type == FG_OUT_BF16, (int)act, vector_ok};
    const int bf16 = out == FG_OUT_BF16;
    const bool may_stream = M <= kMaxStreamRows && N <= kMaxStreamCols && (M <= kFewColsRows || N <= kFewCols);
    if (may_stream && fg_stream_linear_us(M, N, K) <= fg_gemm_epilogue_us(M, N, K))
        return fg_status_from_hip(fg_launch_stream_linear(xq, sx, wq, sw, M, N, K, e, y, bf16, stream));
    return fg_status_from_hip(
        fg_launch_gemm_fprop_epilogue(xq, sx, wq, sw, M, N, K, e, y, bf16, scales == FG_SCALE_POW2, stream));
}

fg_status fg_act_checkpoint_fwd(const void* z, int64_t rows, int64_t F, int64_t ld_z, fg_act act, int gated,
                                fg_scale_mode mode, uint8_t* zq, float* sz, uint8_t* aq, float* sa, hipStream_t stream) {
    if (rows < 0 || F < 0 || !valid_mode(mode) || !valid_act(act) || (gated != 0 && gated != 1)) return FG_ERR_INVALID_ARG;
    if (F > kMaxCols || rows > kMaxRows || ld_z > kMaxStride) return FG_ERR_UNSUPPORTED_SHAPE;
    if (ld_z < (gated ? 2 : 1) * F) return FG_ERR_INVALID_ARG;
    if (rows == 0 || F == 0) return FG_OK;
    if (!z || !zq || !sz || !aq || !sa) return FG_ERR_INVALID_ARG;
    if (F % 128 != 0 || prod_over(F / 128, cdiv(rows, 32), kMaxThreads / 256)) return FG_ERR_UNSUPPORTED_SHAPE;
    if (!aligned(z, 16) || ld_z % 8 != 0 || !aligned(zq, 16) || !aligned(aq, 16) || !aligned(sz, 4) || !aligned(sa, 4))
        return FG_ERR_MISALIGNED;
    return fg_status_from_hip(fg_launch_act_fwd((const uint16_t*)z, rows, F, ld_z, (int)act, gated, mode == FG_SCALE_POW2,
                                                zq, sz, aq, sa, stream));
}

int64_t fg_act_checkpoint_bwd_workspace(int64_t rows, int64_t F, int gated) {
    if (rows < 0 || rows > kMaxRows || F < 0 || F > kMaxCols) return 0;
    return fg_act_bwd_partial_rows(rows) * F * (gated ? 2 : 1) * (int64_t)sizeof(float);
}

fg_status fg_act_checkpoint_bwd(const uint8_t* zq, const float* sz, const void* da, fg_out_dtype da_type, int64_t ld_da,
                                int64_t rows, int64_t F, fg_act act, int gated, fg_scale_mode mode, uint8_t* dzq_cols,
                                float* sdz_cols, uint8_t* dzq_rows, float* sdz_rows, uint8_t* aq_rows, float* sa_rows,
                                float* dbias, void* workspace, int64_t workspace_bytes, hipStream_t stream) {
    if (rows < 0 || F < 0 || ld_da < F || !valid_mode(mode) || !valid_act(act) || !valid_type(da_type) ||
        (gated != 0 && gated != 1) || workspace_bytes < 0)
        return FG_ERR_INVALID_ARG;
    if (F > kMaxCols || rows > kMaxRows || ld_da > kMaxCols) return FG_ERR_UNSUPPORTED_SHAPE;
    if (F == 0 || (rows == 0 && !dbias)) return FG_OK;
    if (!dzq_rows != !sdz_rows || !aq_rows != !sa_rows) return FG_ERR_INVALID_ARG;
    if (rows > 0 && (!zq || !sz || !da || !dzq_cols || !sdz_cols)) return FG_ERR_INVALID_ARG;
    if (F % 128 != 0 || ((dzq_rows || aq_rows) && rows % 128 != 0) || prod_over(F / 128, cdiv(rows, 128), kMaxThreads / 512))
        return FG_ERR_UNSUPPORTED_SHAPE;
    const int64_t need = dbias ? fg_act_checkpoint_bwd_workspace(rows, F, gated) : 0;
    if (need > 0 && (!workspace || workspace_bytes < need)) return FG_ERR_INVALID_ARG;
    if (!aligned(zq, 16) || !aligned(da, 16) || (ld_da * (int64_t)size_of(da_type)) % 16 != 0 || !aligned(dzq_cols, 16) ||
        !aligned(dzq_rows, 16) || !aligned(aq_rows, 16) || !aligned(sz, 4) || !aligned(sdz_cols, 4) || !aligned(sdz_rows, 4) ||
        !aligned(sa_rows, 4) || !aligned(dbias, 4) || (need > 0 && !aligned(workspace, 4)))
        return FG_ERR_MISALIGNED;
    FgActBwd p{};
    p.zq = zq; p.sz = sz; p.da = da; p.ld_da = ld_da; p.rows = rows; p.F = F;
    p.da_bf16 = da_type == FG_OUT_BF16; p.act = (int)act; p.gated = gated; p.pow2 = mode == FG_SCALE_POW2;
    p.dzq_cols = dzq_cols; p.dzq_rows = dzq_rows; p.aq_rows = aq_rows;
    p.sdz_cols = sdz_cols; p.sdz_rows = sdz_rows; p.sa_rows = sa_rows;
    p.dbias = dbias; p.partial = need > 0 ? (float*)workspace : nullptr;
    return fg_status_from_hip(fg_launch_act_bwd(p, stream));
}

int64_t fg_moe_few_tokens_workspace(int64_t T, int32_t topk, int64_t H, int64_t I) {
    if (T < 0 || T > kMaxTokens || topk < 1 || topk > kMaxTopk || H < 0 || H > kMaxExpertDim || I < 0 || I > kMaxExpertDim ||
        H % 128 != 0 || I % 128 != 0)
        return 0;      // sizes that fg_moe_few_tokens refuses
    return fg_moe_workspace_bytes(T, topk, H, I);
}

fg_status fg_moe_few_tokens(const void* x, int64_t ld_x, const int32_t* ids, const float* weights, int64_t T, int32_t topk,
                            const uint8_t* w1q, const float* s1, const uint8_t* w2q, const float* s2, int32_t E, int64_t H,
                            int64_t I, fg_act act, fg_scale_mode act_scales, void* workspace, int64_t workspace_bytes,
                            void* y, int64_t ld_y, fg_out_dtype out, hipStream_t stream) {
    if (T < 0 || topk < 1 || E < 1 || H < 0 || I < 0 || ld_x < H || ld_y < H || !valid_act(act) ||
        !valid_mode(act_scales) || !valid_type(out) || workspace_bytes < 0)
        return FG_ERR_INVALID_ARG;
    if (T > kMaxTokens || topk > kMaxTopk || E > kMaxExperts || H > kMaxExpertDim || I > kMaxExpertDim || H % 128 != 0 ||
        I % 128 != 0 || ld_x > kMaxStride || ld_y > kMaxStride)
        return FG_ERR_UNSUPPORTED_SHAPE;
    // the up-projection: 256 threads to 32 hidden columns of an expert
    if (prod_over(T * topk < E ? T * topk : E, I / 32, kMaxThreads / 256)) return FG_ERR_UNSUPPORTED_SHAPE;
    if (T == 0 || H == 0) return FG_OK;
    if (!x || !ids || !weights || !y || (I > 0 && (!w1q || !s1 || !w2q || !s2))) return FG_ERR_INVALID_ARG;
    const int64_t need = fg_moe_few_tokens_workspace(T, topk, H, I);
    if (need > 0 && (!workspace || workspace_bytes < need)) return FG_ERR_INVALID_ARG;
    if (!aligned(x, 16) || ld_x % 8 != 0 || !aligned(w1q, 16) || !aligned(w2q, 16) || !aligned(y, 16) || !aligned(ids, 4) ||
        !aligned(weights, 4) || !aligned(s1, 4) || !aligned(s2, 4) || (need > 0 && !aligned(workspace, 16)))
        return FG_ERR_MISALIGNED;
    FgMoe p{};
    p.x = (const uint16_t*)x; p.ids = ids; p.weights = weights; p.w1q = w1q; p.w2q = w2q; p.s1 = s1; p.s2 = s2;
    p.workspace = workspace; p.y = y; p.ld_x = ld_x; p.ld_y = ld_y; p.T = T; p.H = H; p.I = I;
    p.topk = topk; p.E = E; p.act = (int)act; p.pow2 = act_scales == FG_SCALE_POW2; p.out_bf16 = out == FG_OUT_BF16;
    return fg_status_from_hip(fg_launch_moe_few_tokens(p, stream));
}

}  // extern "C"

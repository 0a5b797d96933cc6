/*
 * fp8fg — the two ends of a Linear's training step: the norm whose output is the Linear's FP8 operand, with its backward
 * pass behind the Dgrad, and the orthogonalised update of the weight from the gradient that the Wgrad writes.
 *
 * The rules of fp8fg.h hold: every pointer is DEVICE memory of the caller (workspaces included), all work is enqueued on
 * `stream` and can be captured in a HIP graph, nothing is kept between calls, arguments are checked on the host before
 * any HIP call, and a failed check enqueues nothing. Formats and the quantization rule are those of fp8fg.h, applied to
 * the norm's fp32 values, which are not rounded to bf16 first. One call's workspace contents mean nothing to the next;
 * calls that may run at the same time need workspaces of their own.
 */
#ifndef FP8FG_TRAIN_H
#define FP8FG_TRAIN_H

#include "fp8fg.h"

#ifdef __cplusplus
extern "C" {
#endif

/* LAYER: y = (x - mean) rstd gamma + beta with rstd = 1 / sqrt(mean((x - mean)^2) + eps), over a row's columns.
 * RMS:   y = x rstd gamma + beta with rstd = 1 / sqrt(mean(x^2) + eps). */
typedef enum { FG_NORM_LAYER = 0, FG_NORM_RMS = 1 } fg_norm_kind;

/* Norm of every row, quantized: the next Linear's FP8 operand.
 *   x       [rows][cols] of type x_type, row stride ld_x.
 *   gamma   [cols] of type weight_type; beta NULL, or [cols] of the same type.
 *   q_cols  u8 [rows][cols], s_cols f32 [cols/128][rows]: y in 1x128 tiles along the columns, the Fprop's operand.
 *   q_rows  u8 [cols][rows], s_rows f32 [rows/128][cols]: y in tiles along the rows, the Wgrad's operand; both NULL: not
 *           written.
 *   y       NULL, or bf16 [rows][cols], rounded from fp32.
 *   mean, rstd  f32 [rows] each, for the backward pass. mean may be NULL; it is written by FG_NORM_LAYER only. rstd may be
 *           NULL. With q_rows rstd has to be there, and with FG_NORM_LAYER mean too.
 *   Statistics, y and maxima are fp32. A row that holds a NaN or an infinity, or whose sums (of LAYER's squares about the mean, of RMS's
 *   squares) overflow fp32, gets NaN codes, under finite scales; with q_rows its values are NaN codes there too, and the other rows are
 *   as without it. gamma and beta may be as large or small as fp32 allows, as long as y is finite.
 *   cols % 128 == 0, cols <= 18432; rows % 128 == 0 where q_rows is asked for, any rows otherwise; rows <= 2^25, and
 *   rows * cols < 2^36 where q_rows is asked for. eps finite and > 0. x, gamma, beta, q_cols, q_rows, y 16-byte aligned,
 *   ld_x a multiple of 16 bytes; the fp32 outputs 4-byte aligned. rows == 0 or cols == 0 is a no-op. Outputs must not
 *   overlap the inputs or each other. */
fg_status fg_norm_quantize(const void* x, fg_out_dtype x_type, int64_t ld_x, int64_t rows, int64_t cols, fg_norm_kind kind,
                           const void* gamma, const void* beta, fg_out_dtype weight_type, float eps, fg_scale_mode mode,
                           uint8_t* q_cols, float* s_cols, uint8_t* q_rows, float* s_rows, void* y, float* mean, float* rstd,
                           hipStream_t stream);

/* Backward of the norm. With xhat = (x - mean) rstd (RMS: x rstd) and t = dy gamma,
 *   dx = rstd (t - mean(t) - xhat mean(t xhat)) + dres (RMS: without mean(t)),
 *   dgamma = column sums of dy xhat, dbeta = column sums of dy.
 * All in fp32: t, t xhat and their sums over a row have to stay in its range, or the row's dx is not finite.
 *   x, gamma  as for fg_norm_quantize; mean, rstd f32 [rows], as it wrote them (mean not read, and may be NULL, with
 *             FG_NORM_RMS).
 *   dy        [rows][cols] of type dy_type, row stride ld_dy: the Dgrad of the Linear behind the norm.
 *   dres      NULL, or [rows][cols] of type dres_type, row stride ld_dres: the gradient that reaches x past the norm. It may
 *             be dx itself (same type, ld_dres == cols).
 *   dx        [rows][cols] of type dx_type, rounded once from fp32.
 *   dgamma, dbeta  f32 [cols] each, or NULL: not computed. accumulate != 0: added to what they hold. The rows are added up
 *             in an order that depends on the sizes only.
 *   workspace fg_norm_bwd_workspace(rows, cols) bytes (0 up to 512 rows), 16-byte aligned, read and written only where
 *             dgamma or dbeta is there; may be NULL where neither is, and where it has no bytes.
 *   cols % 128 == 0, cols <= 18432, rows <= 2^25. x, gamma, dy, dres, dx 16-byte aligned, row strides multiples of 16 bytes;
 *   the fp32 vectors 4-byte aligned. rows == 0: no-op, but for dgamma and dbeta, which become 0 (or stay, with accumulate).
 *   cols == 0 is a no-op. Outputs and workspace must not overlap the inputs (but dx dres) or each other. */
int64_t fg_norm_bwd_workspace(int64_t rows, int64_t cols);
fg_status fg_norm_bwd(const void* x, fg_out_dtype x_type, int64_t ld_x, const float* mean, const float* rstd, const void* gamma,
                      fg_out_dtype weight_type, const void* dy, fg_out_dtype dy_type, int64_t ld_dy, const void* dres,
                      fg_out_dtype dres_type, int64_t ld_dres, int64_t rows, int64_t cols, fg_norm_kind kind, void* dx,
                      fg_out_dtype dx_type, float* dgamma, float* dbeta, int accumulate, void* workspace,
                      int64_t workspace_bytes, hipStream_t stream);

/* Orthogonalised update of a weight by Newton-Schulz products (the Muon optimiser's): for each of `batch` matrices
 *   X = G / (|G| + eps), |G| the Frobenius norm,
 *   `steps` times: A = X X^T (X^T X where N > K), B = a I + b A + c A A, X = B X (X B),
 *   out = scale X.
 *   g    [batch][N][K] of type g_type, row stride ld_g, matrices N ld_g elements apart: the gradient or momentum.
 *   out  bf16 [batch][N][K].
 *   The products' operands are held in fp16, X scaled by 2^12 and A and B by 2^11, and their sums in fp32. What that changes of
 *   out, besides its own rounding to bf16 (1.7e-3), goes by G's singular values, as the steps raise the roundings in small and in
 *   empty directions as they raise those directions themselves. In the 2-norm, relative, with the default coefficients and five steps:
 *     the product of random tokens, more of them than the smaller side has rows    1.0e-3 to 1.6e-3
 *     singular values all alike, or falling as 1 / sqrt(i)                        2e-3
 *     falling as 1 / i, 1 / i^2                                                   4.5e-3, 2.5e-2
 *     falling as exp(-i / 100), exp(-i / 20)                                      6.5e-3, 1.5e-2
 *     1, 4, 16, 64, 256 alike and the others zero                                 0.15, 0.08, 0.05, 0.03, 0.009
 *   Along the directions that G has, out is as exact as in the first row.
 *   Entries of X below 2^-26 are held with fewer bits and those below 2^-37 as zeros, which counts where |G| is far below eps: a 256 x
 *   1024 product of random tokens is off by 2e-3 at |G| = 1e-5 eps, 3e-3 at 1e-6 eps, 3e-2 at 1e-7 eps, and lost at 1e-9 eps.
 *   The coefficients have to keep the iteration inside fp16's range: with u0 = 1 and u the largest |a s + b s^3 + c s^5| for
 *   0 <= s <= u (or u itself, if that is larger), every u stays below 5 and |a| + |b| u^2 + |c| u^4
 *   below 30 (FG_ERR_INVALID_ARG otherwise). (3.4445, -4.7750, 2.0315) does, for any steps.
 *   A matrix of zeros gives zeros; one that holds a NaN or an infinity, or whose norm overflows fp32, gives NaN.
 *   workspace  fg_orthogonalize_workspace(batch, N, K) bytes, 256-byte aligned; 0 for sizes that are refused here.
 *   N and K at most 65536, batch at most 65535, batch * ceil(N / 64) * ceil(K / 64) < 2^24, 1 <= steps <= 32, a, b, c, eps and scale finite, eps >
 *   0. g aligned to its elements, out 2-byte aligned. batch, N or K == 0 is a no-op. The workspace must not overlap g or out;
 *   out may be g itself only where nothing else of g's storage is needed: other overlaps are undefined. */
int64_t fg_orthogonalize_workspace(int64_t batch, int64_t N, int64_t K);
fg_status fg_orthogonalize(const void* g, fg_out_dtype g_type, int64_t ld_g, int64_t batch, int64_t N, int64_t K, int steps,
                           float a, float b, float c, float eps, float scale, void* out, void* workspace,
                           int64_t workspace_bytes, hipStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* FP8FG_TRAIN_H */

/*
 * fp8fg — the feed-forward operators around the FP8 GEMMs of fp8fg.h: a Linear with bias, activation and
 * residual in its epilogue, an activation function whose input is kept as an FP8 checkpoint, its backward
 * pass from that checkpoint, and a whole mixture-of-experts feed-forward for a few tokens.
 *
 * The rules of fp8fg.h hold: every pointer is DEVICE memory of the caller (workspaces included), all work is
 * enqueued on `stream` and can be captured in a HIP graph, nothing is kept between calls, arguments are
 * checked on the host before any HIP call, and a failed check enqueues nothing. Formats, the quantization
 * rule and the GEMM rule are those of fp8fg.h; where a quantizer below takes values that the kernel itself
 * computed, the rule is applied to their fp32 values, which are not rounded to bf16 first. Inputs must be
 * finite unless stated otherwise; of values that overflow fp32 on the way (a gate times its factor), an infinite one gets
 * the code NaN, and its tile's scale comes from the largest finite float.
 */
#ifndef FP8FG_FFN_H
#define FP8FG_FFN_H

#include "fp8fg.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Activation functions, evaluated in fp32:
 *   NONE z;   RELU max(z, 0), slope 0 at 0;   SILU z / (1 + exp(-z));
 *   GELU_TANH 0.5 z (1 + tanh(sqrt(2 / pi) (z + 0.044715 z^3))). */
typedef enum { FG_ACT_NONE = 0, FG_ACT_RELU = 1, FG_ACT_GELU_TANH = 2, FG_ACT_SILU = 3 } fg_act;

/* Fprop with its epilogue: Y[M][N] = act(X[M][K] . W[N][K]^T + bias) + residual.
 *   xq, sx, wq, sw   as for fg_fp8_gemm_fprop. With FG_SCALE_POW2 every scale has to be a power of two
 *                    (precondition; another scale gives NaN or the product with its own value).
 *   bias      NULL, or [N] of type bias_type.
 *   residual  NULL, or [M][N] of type residual_type, row stride ld_res (elements, >= N). It may be y itself
 *             (same type, ld_res == N); any other overlap with y is undefined.
 *   y         [M][N] f32 or bf16 (row stride N). The sum, bias, activation and residual are fp32, and the
 *             result is rounded once, when it is stored.
 *   K % 128 == 0; any M, N >= 0 (M == 0 or N == 0: no-op; K == 0: act(bias) + residual). xq, wq, y 16-byte
 *   aligned; sx, sw 4-byte aligned; bias and residual aligned to their elements. K <= 2^24;
 *   ceil(M / 128) * ceil(N / 128) < 2^24, and with FG_GEMM_TILE also ceil(M / 256) * ceil(N / 192) <= 5592405 (a launch
 *   has less than 2^32 threads). The problem's sizes choose between a kernel that streams the weights past
 *   the rows, for few rows or few columns, and the GEMM tiles (128x128 or the Fprop's); the streaming kernel adds a row's blocks up in another order,
 *   and it and the 128x128 tiles apply power-of-2 scales as any others, so sums may differ in their last bits.
 *   FG_GEMM_TILE forces a tile, as there; 128x128 is one of them here. */
fg_status fg_fp8_gemm_fprop_epilogue(const uint8_t* xq, const float* sx, const uint8_t* wq, const float* sw, int64_t M,
                                     int64_t N, int64_t K, const void* bias, fg_out_dtype bias_type, fg_act act,
                                     const void* residual, fg_out_dtype residual_type, int64_t ld_res, void* y,
                                     fg_out_dtype out, fg_scale_mode scales, hipStream_t stream);

/* Activation function with an FP8 checkpoint of its input: one read of z, which need not be kept.
 *   z   bf16 [rows][W], row stride ld_z; W = F, or 2 F when gated (columns [0, F) the gate, [F, 2 F) the other
 *       factor: a = act(gate) * up).
 *   zq  u8 [rows][W], sz f32 [W/128][rows]: fg_quantize_act_1x128(z, FG_ALONG_COLS, mode), bit for bit.
 *   aq  u8 [rows][F], sa f32 [F/128][rows]: a in the same tiling, the next Linear's input.
 *   F % 128 == 0, F <= 2^23, rows <= 2^25, F * ceil(rows / 32) < 2^31. z, zq, aq 16-byte aligned; ld_z % 8 == 0; sz, sa 4-byte aligned.
 *   rows == 0 or F == 0 is a no-op. Outputs must not overlap z or each other. */
fg_status fg_act_checkpoint_fwd(const void* z, int64_t rows, int64_t F, int64_t ld_z, fg_act act, int gated,
                                fg_scale_mode mode, uint8_t* zq, float* sz, uint8_t* aq, float* sa, hipStream_t stream);

/* Backward of the activation function from its FP8 checkpoint. With z^ the checkpoint's values:
 *   dz = da * act'(z^), or when gated dgate = da * up * act'(gate), dup = da * act(gate); a = act(z^) or
 *   act(gate) * up, computed again instead of having been kept.
 *   zq, sz  the checkpoint, as fg_act_checkpoint_fwd wrote it (any fp32 scales).
 *   da      [rows][F] of type da_type, row stride ld_da: the Dgrad of the next Linear.
 *   dzq_cols u8 [rows][W], sdz_cols f32 [W/128][rows]: dz tiled along the columns, this Linear's Dgrad operand.
 *   dzq_rows u8 [W][rows], sdz_rows f32 [rows/128][W]: dz tiled along the rows, its Wgrad operand; both NULL: not
 *            written.
 *   aq_rows  u8 [F][rows], sa_rows f32 [rows/128][F]: a tiled along the rows, the next Linear's Wgrad operand;
 *            both NULL: not written.
 *   dbias    NULL, or f32 [W]: the column sums of dz (fp32, in an order that depends on the sizes only).
 *   workspace  fg_act_checkpoint_bwd_workspace(rows, F, gated) bytes, read and written only with dbias; may be NULL
 *            where that is 0 or dbias is NULL. 4-byte aligned. One call's contents mean nothing to the next; calls
 *            that may run at the same time need workspaces of their own.
 *   F % 128 == 0; rows % 128 == 0 where a tiling along the rows is asked for, any rows otherwise; F and ld_da at most
 *   2^23, rows at most 2^25, F * ceil(rows / 128) < 2^30. zq, da, dzq_cols, dzq_rows, aq_rows 16-byte aligned, ld_da a multiple of 16 bytes; the fp32 outputs and sz 4-byte aligned.
 *   rows == 0 or F == 0: no-op, but for dbias, which becomes 0. Outputs and workspace must not overlap the inputs or each
 *   other. */
int64_t fg_act_checkpoint_bwd_workspace(int64_t rows, int64_t F, int gated);
fg_status fg_act_checkpoint_bwd(const uint8_t* zq, const float* sz, const void* da, fg_out_dtype da_type, int64_t ld_da,
                                int64_t rows, int64_t F, fg_act act, int gated, fg_scale_mode mode, uint8_t* dzq_cols,
                                float* sdz_cols, uint8_t* dzq_rows, float* sdz_rows, uint8_t* aq_rows, float* sa_rows,
                                float* dbias, void* workspace, int64_t workspace_bytes, hipStream_t stream);

/* A whole mixture-of-experts feed-forward for at most 64 tokens: for every token t
 *   y[t] = sum over j < topk with 0 <= ids[t][j] < E of weights[t][j] * down_e(act(gate_e(x[t])) * up_e(x[t])),
 * e = ids[t][j], with every product an FP8 GEMM of fp8fg.h's rule: x[t] is quantized 1x128 along its columns, and
 * so is the fp32 product act(gate) * up before the down-projection.
 *   x    bf16 [T][H], row stride ld_x. A token none of whose ids is in [0, E) is not used: its y is 0 whatever x
 *        holds.
 *   ids  int32 [T][topk], weights f32 [T][topk]. Any id outside [0, E) is skipped (experts of another GPU), and so
 *        is its weight. The same id twice in a row counts with the sum of its weights.
 *   w1q  u8 [E][2 I][H], s1 f32 [E][2 I/128][H/128]: gate rows [0, I), up rows [I, 2 I).
 *   w2q  u8 [E][H][I], s2 f32 [E][H/128][I/128].
 *   act_scales  the scale mode of the two activations; the weights' scales may be any fp32 in both.
 *   workspace   fg_moe_few_tokens_workspace(T, topk, H, I) bytes, 16-byte aligned; calls that may run at the same
 *               time need workspaces of their own. The size of a T, topk, H or I that is refused here is 0.
 *   y    [T][H] f32 or bf16, row stride ld_y.
 *   0 <= T <= 64, 1 <= topk <= 32, 1 <= E <= 2048, H % 128 == 0, I % 128 == 0, H and I at most 2^20, I * min(E, T * topk) <
 *   2^29. x, w1q, w2q, y
 *   16-byte aligned, ld_x % 8 == 0; ids, weights, s1, s2 4-byte aligned; ld_y >= H. T == 0 or H == 0 is a no-op;
 *   I == 0 writes zeros. x, the weights and the workspace must not overlap y. */
int64_t fg_moe_few_tokens_workspace(int64_t T, int32_t topk, int64_t H, int64_t I);
fg_status fg_moe_few_tokens(const void* x, int64_t ld_x, const int32_t* ids, const float* weights, int64_t T, int32_t topk,
                            const uint8_t* w1q, const float* s1, const uint8_t* w2q, const float* s2, int32_t E, int64_t H,
                            int64_t I, fg_act act, fg_scale_mode act_scales, void* workspace, int64_t workspace_bytes,
                            void* y, int64_t ld_y, fg_out_dtype out, hipStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* FP8FG_FFN_H */

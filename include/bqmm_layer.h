/*
 * bqmm_layer.h -- the operators around the projection matmul of bqmm.h, in
 * the same library (libbqmm.so) and under the same conventions: device
 * pointers owned by the caller, no allocation, no host synchronization, work
 * enqueued on `stream`, outputs fully overwritten, the same return codes, and
 * every argument check before any HIP call.
 *
 *   - root-mean-square norm with the residual's addition, written as plain
 *     values or as the 8-bit operands of bqm_q8_0_gemv / bqm_q8_0_gemm
 *     (q8_1) and of bqm_e4m3_blk_gemm (block-128 e4m3);
 *   - MXFP4, microscaled 4-bit floating point: quantization, dequantization,
 *     the product of two quantized operands and the decode product with f32
 *     activations;
 *   - log probabilities of given tokens, with the log-sum-exp, the entropy
 *     and the top alternatives of each row of logits.
 *
 * Value types of inputs and outputs where a call takes a choice of them.
 * Arithmetic is f32 whatever the type; each output is rounded once, to
 * nearest even.
 */
#ifndef BQMM_LAYER_H
#define BQMM_LAYER_H

#include "bqmm.h"

#ifdef __cplusplus
extern "C" {
#endif

#define BQM_F32 0
#define BQM_F16 1
#define BQM_BF16 2

/* Largest m of bqm_mxfp4_gemv. */
#define BQM_MXFP4_GEMV_MAX_M 16
/* Largest top_k of bqm_logprobs. */
#define BQM_LOGPROBS_MAX_TOP 32

/*
 * Root-mean-square norm of x, or of x + res:
 *   s[t][i] = x[t][i] (+ res[t][i]);  h = s;
 *   y[t][i] = s[t][i] * (1 / sqrt(sum_i s[t][i]^2 / k + eps)) * gain[i].
 * s is the unrounded f32 sum; h is s rounded to x's type.
 *
 *   x, ldx   : x_type [m][k], rows ldx >= k elements apart.
 *   res, ldr : x_type [m][k], the residual; NULL for none.
 *   gain     : f32 [k], 4-byte aligned; NULL for ones.
 *   eps      : finite, >= 0 (else BQM_EINVAL).  An all-zero row with eps = 0
 *              is 0 * inf = NaN, as the formula has it.
 *   h, ldh   : x_type [m][k] out; given if and only if res is (else
 *              BQM_EINVAL).  h may be x or res itself (same pointer and
 *              stride); no other outputs may overlap an input.
 *   y        : y_type [m][k] out, dense; y_type is BQM_F32 or x_type (else
 *              BQM_EUNSUPPORTED).
 *   m, k >= 1 (else BQM_EINVAL), any k.  Every pointer is aligned to its
 *   element (else BQM_EUNSUPPORTED); rows that are aligned to 16 bytes take
 *   wide loads.  Strides are unused when m is 1.
 * The order of the sums depends on k and x_type alone: a row's result does
 * not depend on m, on the strides or on the alignment.
 */
int bqm_add_rmsnorm(const void *x, int64_t ldx, const void *res, int64_t ldr, const float *gain, float eps, void *h,
                    int64_t ldh, void *y, int x_type, int y_type, int m, int k, void *stream);

/*
 * The same norm with y in 8 bits: bqm_q8_1_quantize's rule applied to the f32
 * y, bit for bit what the two calls give.
 *   xq, xds : as bqm_q8_1_quantize writes them.
 *   k % 32 == 0 (else BQM_EUNSUPPORTED).
 */
int bqm_add_rmsnorm_q8_1(const void *x, int64_t ldx, const void *res, int64_t ldr, const float *gain, float eps,
                         void *h, int64_t ldh, int8_t *xq, float *xds, int x_type, int m, int k, void *stream);

/*
 * The same norm with bqm_e4m3_blk_quantize's rule applied to the f32 y, bit
 * for bit what the two calls give.
 *   xq, xs : as bqm_e4m3_blk_quantize writes them.
 *   k >= 16 (else BQM_EINVAL), k % 16 == 0 (else BQM_EUNSUPPORTED).
 */
int bqm_add_rmsnorm_e4m3_blk(const void *x, int64_t ldx, const void *res, int64_t ldr, const float *gain, float eps,
                             void *h, int64_t ldh, uint8_t *xq, float *xs, int x_type, int m, int k, void *stream);

/*
 * MXFP4 (OCP Microscaling Formats v1.0): 32 consecutive values along k share
 * one E8M0 scale byte s, and value i of the block stands for
 * 2^(s - 127) * e2m1(c), c a 4-bit code: sign (bit 3), then 0, 0.5, 1, 1.5,
 * 2, 3, 4, 6.  s = 255 makes the block NaN.
 *   codes  : uint8 [rows][k/2]; value 2j of a row in the low half of byte j,
 *            value 2j + 1 in its high half.
 *   scales : uint8 [rows][k/32].
 *
 * bqm_mxfp4_quantize: s = max(floor(log2(amax)) - 2 + 127, 0) over the
 * block's largest magnitude, codes of x * 2^(127 - s) rounded to nearest even
 * and saturated at +-6, sign of zero kept.  A block of zeros has s = 0; a
 * block that holds an infinity or a NaN has s = 255 and codes 0.  Activations
 * and weights are quantized alike.
 *   x, ldx : x_type [m][k], 16-byte aligned rows (x and ldx elements, else
 *            BQM_EUNSUPPORTED), ldx >= k.
 *   codes 4-byte aligned.  m >= 1, k >= 32 (else BQM_EINVAL); k % 32 == 0
 *   (else BQM_EUNSUPPORTED).
 */
int bqm_mxfp4_quantize(const void *x, int64_t ldx, uint8_t *codes, uint8_t *scales, int x_type, int m, int k,
                       void *stream);

/*
 * bqm_mxfp4_dequantize: y[t][i] = 2^(s - 127) * e2m1(c), rounded once to
 * y_type: exact in f32 and, for normal results, in bf16, but for values past
 * the type's range (in both from 4 at s = 253 and from 2 at s = 254), which
 * become infinite.
 *   codes 4-byte aligned; y 16-byte aligned, dense; sizes as above.
 */
int bqm_mxfp4_dequantize(const uint8_t *codes, const uint8_t *scales, void *y, int y_type, int m, int k,
                         void *stream);

/*
 * bqm_mxfp4_gemm: y[t][r] = sum_b 2^(xs[t][b] + ws[r][b] - 254) * sum_{i in b}
 * e2m1(xq[t][i]) * e2m1(w[r][i]), f32 accumulation; the scales enter the
 * matrix cores with the codes.
 *   w, ws  : codes [n][k/2] and scales [n][k/32] of the weights.
 *   xq, xs : codes [m][k/2] and scales [m][k/32] of the activations.
 *   y      : f32 [m][n] out, 4-byte aligned.
 *   m, n >= 1, k >= 32 (else BQM_EINVAL); k % 32 == 0; w and xq 16-byte
 *   aligned (else BQM_EUNSUPPORTED).
 * Any scales but 255 count, at each side up to 254: only their sum matters,
 * and a result past the range of f32 is infinite (NaN where such infinities
 * cancel).  A block with scale 255 makes its row or token NaN.  The order of
 * the sums depends on the sizes, m too, so where sums round, a token's last
 * bits may differ between calls of different m.
 */
int bqm_mxfp4_gemm(const uint8_t *w, const uint8_t *ws, const uint8_t *xq, const uint8_t *xs, float *y, int m, int k,
                   int n, void *stream);

/*
 * bqm_mxfp4_gemv: the decode / verify product on MXFP4 weights and f32
 * activations, 1 <= m <= BQM_MXFP4_GEMV_MAX_M:
 * y[t][r] = sum_b 2^(ws[r][b] - 127) * sum_{i in b} x[t][i] * e2m1(w[r][i]),
 * f32 accumulation.  A token's result does not depend on m or on the other
 * tokens.  An infinity or NaN among a token's activations makes that token's
 * results infinite or NaN.  Scales are at most 252, which is what
 * bqm_mxfp4_quantize writes for finite values, or 255 (NaN): with 253 and 254
 * the largest codes leave the range of f32.  Bits of x below 2^-133 are lost.
 *   x : f32 [m][k], 16-byte aligned, dense; the rest as bqm_mxfp4_gemm.
 */
int bqm_mxfp4_gemv(const uint8_t *w, const uint8_t *ws, const float *x, float *y, int m, int k, int n, void *stream);

/*
 * Log probabilities of rows of logits l[t][0..n):
 *   lse[t]     = log sum_j exp(l[t][j]),
 *   logp[t][i] = l[t][tokens[t][i]] - lse[t],
 *   entropy[t] = -sum_j p_j log p_j, p_j = exp(l[t][j] - lse[t]) (p_j = 0
 *                adds nothing),
 *   top_ids[t] = the top_k largest logits' columns, largest first, the lowest
 *                column first among equals (-0 and +0 are equal; a NaN is
 *                below -inf), top_logp[t] their log probabilities.
 * Masked logits are -inf or any low value.  A row of -inf alone (a mask that
 * leaves nothing) has lse and every log probability -inf and entropy 0.  A
 * row with a NaN or +inf has NaN in lse, entropy and every log probability.
 *
 *   logits, ld : type [m][n], rows ld >= n elements apart, aligned to an
 *                element.
 *   tokens     : int32 [m][n_tokens]; NULL with n_tokens = 0.  A token
 *                outside 0..n-1 (padding) gets NaN and reads nothing.
 *   logp       : f32 [m][n_tokens] out;  lse, entropy : f32 [m] out.
 *   top_ids    : int32 [m][top_k] out, top_logp : f32 [m][top_k] out; NULL
 *                with top_k = 0.
 *   workspace  : bqm_logprobs_workspace(m, n, top_k) bytes, 16-byte aligned;
 *                needs no initial contents; NULL if that is 0.
 *   m, n >= 1, 0 <= n_tokens, 0 <= top_k <= min(n, BQM_LOGPROBS_MAX_TOP)
 *   (else BQM_EINVAL).
 * One read of the logits: rows are split over workgroups when there are few.
 */
int bqm_logprobs(const void *logits, int64_t ld, int type, const int *tokens, int n_tokens, float *logp, float *lse,
                 float *entropy, int *top_ids, float *top_logp, int top_k, void *workspace, int m, int n,
                 void *stream);

/* Bytes of workspace for bqm_logprobs; 0 for none, -1 for sizes it refuses. */
int64_t bqm_logprobs_workspace(int m, int n, int top_k);

#ifdef __cplusplus
}
#endif

#endif /* BQMM_LAYER_H */

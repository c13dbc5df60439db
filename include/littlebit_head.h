/*
 * littlebit_head.h -- C ABI of the dense operators around the LittleBit layers
 * on MI355X (gfx950): the residual root-mean-square norm, the 8-bit integer
 * product and the token log probabilities.
 *
 * A LittleBit model replaces the linear layers of its Transformer blocks and
 * keeps the rest (trueseeker.com case, "The trace / claim to source": only
 * the Transformer blocks are quantized, embedding and head stay FP16).  The
 * norms in front of the projections (littlebit_block_fwd's x_qkv and x_gu)
 * and the head after the last block are therefore the caller's: these are
 * the operators for them.  At 0.1 bits per weight the head is the largest
 * read of a decode step, which is why it is offered in 8 bits.
 *
 * A library of its own (liblittlebit_head.so).  The conventions of
 * littlebit.h hold: device pointers, caller-owned memory, nothing is
 * allocated, freed or synchronised, work is enqueued on `stream` of the
 * current device, arguments are validated before anything is enqueued, a
 * negative lb_status reports a refusal and littlebit_head_last_error its
 * reason (thread-local).  Calls may overlap; a workspace holds nothing
 * between calls and needs no initialization, but calls that run at the same
 * time must not share one.
 *
 * Matrices are row-major with a row stride (ld*, in elements) of at least the
 * row length.  Any alignment of a whole element is accepted; rows that start
 * at a multiple of 16 bytes are fastest.  `rows` (`batch`) may be 0 (nothing is
 * computed; a gradient summed over rows is then 0) and is at most 2^21 a call.
 */
#ifndef LITTLEBIT_HEAD_H
#define LITTLEBIT_HEAD_H

#include "littlebit.h"

#ifdef __cplusplus
extern "C" {
#endif

/* bfloat16, beside lb_dtype's LB_F32 and LB_F16 (dtype arguments are ints). */
#define LB_BF16 2

/* Largest row length of the norm and of the row quantiser. */
#define LB_NORM_MAX_N 32768
/* Most alternatives littlebit_logprobs_fwd returns for a token. */
#define LB_TOP_MAX 64

/*
 * Residual root-mean-square norm.  Per row
 *     h   = round(x + residual)             (h = x without a residual)
 *     y_j = h_j * weight_j / sqrt(mean_i h_i^2 + eps)
 * and, for the 8-bit output,
 *     scale = max_j |y_j| / 127,  q_j = rint(y_j / scale)   (ties to even)
 * so that q_j * scale stands for y_j.  The norm is taken of the stored,
 * rounded h; sums are held in fp32; y is rounded to the type once, and q is
 * taken from the unrounded y.
 *   dtype     LB_F16 or LB_BF16: the type of x, residual, weight, hidden, y.
 *   residual  may be NULL; then hidden must be NULL too (h is x).
 *   hidden    receives h; may be x or residual itself (same stride).
 *   y         dense output, or NULL.
 *   q, scale  8-bit output (int8 and one fp32 scale a row), or both NULL.  At
 *             least one of y and q is given.  y and q overlap no input.
 * A row of zeros has scale 0 (eps > 0; with eps = 0 its y is NaN).  A row with a
 * NaN or an infinity in h or in a weighted value h_j * weight_j has scale NaN and q 0.
 * Rows of any other size are normed, those whose squares fp32 does not hold (bf16) too.
 * (h_j * weight_j is formed in fp32 first: of fp16 values it always fits, of bf16
 * ones it does for weights below 1e19.)  1 <= n <= LB_NORM_MAX_N.
 */
lb_status littlebit_rmsnorm_fwd(const void *x, int64_t ldx, const void *residual, int64_t ldr,
                                const void *weight, int dtype, int64_t rows, int64_t n, float eps,
                                void *hidden, int64_t ldh, void *y, int64_t ldy, int8_t *q,
                                int64_t ldq, float *scale, void *stream);

/*
 * Backward pass of the dense norm (and, with the rounding to 8 bits passed
 * straight through, of the 8-bit one).  With r = 1 / sqrt(mean h^2 + eps):
 *     dx_j  = dhidden_j + r * weight_j dy_j - h_j (r^3 / n) sum_i weight_i dy_i h_i
 *     dweight_j = sum over rows of dy_j h_j r
 * dx is the gradient of x and of the residual alike.
 *   hidden    h as littlebit_rmsnorm_fwd left it (x without a residual).
 *   dhidden   gradient that arrives at h by itself, or NULL.
 *   dx        type `dtype`; may be dy, dhidden or hidden itself (same stride).
 *   dweight   fp32 [n].
 *   ws        littlebit_rmsnorm_bwd_workspace_bytes(rows, n) bytes, 16-byte
 *             aligned.
 * The sums over rows run in a fixed order: the same call gives the same bits.
 * With eps = 0 every row needs a normal value of its type: r is held in fp32.
 * sum_i weight_i dy_i h_i has to stay in fp32's range (that of h / 2^80, where the
 * squares of h do not).
 */
size_t littlebit_rmsnorm_bwd_workspace_bytes(int64_t rows, int64_t n);

lb_status littlebit_rmsnorm_bwd(const void *dy, int64_t lddy, const void *dhidden, int64_t lddh,
                                const void *hidden, int64_t ldh, const void *weight, int dtype,
                                int64_t rows, int64_t n, float eps, void *dx, int64_t lddx,
                                float *dweight, void *ws, size_t ws_bytes, void *stream);

/*
 * 8-bit codes of each row of a matrix (a head's weight by output channel, or
 * tokens): scale = max_j |x_j| / 127, q_j = rint(x_j / scale).  dtype LB_F32,
 * LB_F16 or LB_BF16.  Rows of zeros, NaN and infinities as for the norm.
 * 1 <= n <= LB_NORM_MAX_N.
 */
lb_status littlebit_q8_quantize(const void *x, int64_t ldx, int dtype, int64_t rows, int64_t n,
                                int8_t *q, int64_t ldq, float *scale, void *stream);

/*
 * Product of 8-bit integers with a scale for each token and each output
 * channel, beside littlebit_linear_fwd for the matrices that stay dense:
 *     y[t][o] = xscale[t] * wscale[o] * sum_k xq[t][k] * wq[o][k]
 * The sum is exact (int32); it is scaled in fp32 and rounded to the output's
 * type once.
 *   xq        batch rows of n codes; wq m rows of n codes.
 *   xscale    fp32 [batch]; wscale fp32 [m].
 *   y         batch rows of m values, y_dtype LB_F32, LB_F16 or LB_BF16.
 * batch >= 0, 1 <= m <= 2^24, 1 <= n <= 131071 (where 128^2 n stays below 2^31),
 * batch x m <= 2^38.
 */
lb_status littlebit_q8_linear_fwd(const int8_t *xq, int64_t ldx, const float *xscale,
                                  const int8_t *wq, int64_t ldw, const float *wscale, int64_t batch,
                                  int64_t m, int64_t n, void *y, int64_t ldy, int y_dtype,
                                  void *stream);

/*
 * Log probabilities of given tokens, entropy and the most probable
 * alternatives, from logits x (one row a token):
 *     lse = log sum_v exp x_v        p_v = exp(x_v - lse)
 *     logprob = x_target - lse       entropy = lse - sum_v p_v x_v
 *     top_index[0..top-1], top_logprob: the `top` largest logits in falling
 *     order, the lowest index first among equals, as x - lse.
 *   dtype     LB_F32, LB_F16 or LB_BF16.  Sums are held in fp32.
 *   targets   int64 [rows], or NULL (then logprob is NULL too).  A negative
 *             target gives no token: logprob 0.  One of vocab or more:
 *             logprob NaN.
 *   logprob, entropy  fp32 [rows]; entropy may be NULL.
 *   lse       fp32 [2][rows]: the row's maximum m, then log sum exp(x - m);
 *             lse is their sum.  (Apart, so that nothing is lost where the
 *             logits lie far from 0, as in a row masked with the type's
 *             lowest value.)  A row of -infinity has the lowest fp32 value and
 *             -infinity.
 *   top       0 <= top <= min(vocab, LB_TOP_MAX); top_logprob fp32 and
 *             top_index int64, rows x top each, contiguous; NULL for top = 0.
 *   ws        littlebit_logprobs_workspace_bytes(rows, vocab, dtype, top)
 *             bytes (may be 0, then ws may be NULL), 16-byte aligned.
 * A logit of -infinity is a masked token: probability 0, no part of the
 * entropy.  A row of nothing else has lse and every log probability
 * -infinity and entropy 0.  NaN or +infinity anywhere in a row makes lse,
 * logprob and entropy NaN; among the alternatives NaN ranks first.
 * 1 <= vocab <= 2^30.
 */
size_t littlebit_logprobs_workspace_bytes(int64_t rows, int64_t vocab, int dtype, int top);

lb_status littlebit_logprobs_fwd(const void *logits, int64_t ld, int dtype, int64_t rows,
                                 int64_t vocab, const int64_t *targets, float *logprob,
                                 float *entropy, float *lse, int top, float *top_logprob,
                                 int64_t *top_index, void *ws, size_t ws_bytes, void *stream);

/*
 * Gradient of the logits:
 *     dlogits_v = [v = target] dlogprob + sum_j [v = top_index_j] dtop_j
 *                 - p_v (dlogprob + sum_j dtop_j) - p_v (log p_v + entropy) dentropy
 * rounded to the type once (a target among the alternatives included).
 *   targets, dlogprob   both NULL where logprob has no gradient.  Rows
 *             without a token (negative target) ignore dlogprob; a target
 *             of vocab or more makes its row NaN.
 *   entropy, dentropy   both NULL where entropy has no gradient.
 *   top_index, dtop     rows x top, contiguous; NULL for top = 0.
 *   lse, entropy, top_index  as littlebit_logprobs_fwd gave them.
 *   dlogits   the logits' type; may be the logits themselves (same stride).
 * The p_v terms of a masked logit are 0; a row of nothing else has gradient 0, whatever
 * its target.
 * rows x ceil(vocab / 8192) < 2^24.
 */
lb_status littlebit_logprobs_bwd(const void *logits, int64_t ld, int dtype, int64_t rows,
                                 int64_t vocab, const int64_t *targets, const float *lse,
                                 const float *entropy, const float *dlogprob, const float *dentropy,
                                 int top, const int64_t *top_index, const float *dtop,
                                 void *dlogits, int64_t ldd, void *stream);

/* Thread-local message for the most recent failing call of this library. */
const char *littlebit_head_last_error(void);

#ifdef __cplusplus
}
#endif

#endif /* LITTLEBIT_HEAD_H */

/*
 * mlp_experts.h -- C ABI of what stands around the products by expert of mlp_block.h (same library,
 * libmlp_chain.so), forward and backward:
 *
 *   route      from the router's logits: every token's top experts with their gates, how many rows each
 *              expert gets, the row of every (token, choice) in expert order, and the balance loss;
 *   dispatch   the tokens' rows, copied into expert order for mlp_linear_forward;
 *   combine    the experts' rows, weighted by the gates and added to the residual, in token order.
 *
 * Conventions are those of mlp_block.h: device pointers on the current device, calls only enqueue on
 * `stream`, nothing is allocated or kept between calls, errors are returned.  Strides (ld*) are in
 * elements between rows, a row is contiguous.  Inputs may alias one another but not an output; the
 * exceptions are named at the call.  Results do not change from run to run.  A workspace is used from a
 * call's start to its end on the stream: calls that may run at the same time, replayed graphs among them,
 * need one each.
 */
#ifndef MLP_EXPERTS_H_
#define MLP_EXPERTS_H_

#include "mlp_block.h"

#ifdef __cplusplus
extern "C" {
#endif

#define MLP_MAX_TOP 32

/* --------------------------------------------------------------------------------------- route --
 * tokens x experts logits (BF16 or F32), 0 <= tokens, 1 <= experts <= MLP_MAX_EXPERTS,
 * 1 <= top <= min(experts, MLP_MAX_TOP), tokens * top < 2^31.
 *
 * p = softmax over a token's logits, in fp32.  Its choices are the `top` largest logits, the first of
 * equal ones first; a logit of -inf is never chosen (p = 0).  A choice's gate is its p, or with
 * normalize != 0 its p divided by the sum of the chosen ones' p.  A token whose mask is 0 makes no choice,
 * nor does one whose logits are all -inf; one with fewer finite logits than `top` makes fewer.  NaN counts
 * as the largest value, and a token with a logit of NaN or +inf has NaN among its gates and in the loss.
 *
 *   mask      uint8 per token, 0: padding; NULL: none is
 *   gates     fp32 [tokens][top], 0 without a choice
 *   chosen    int32 [tokens][top], experts, best first; -1 without a choice
 *   slots     int32 [tokens][top]: the row of this choice when the choices are sorted by expert, and by
 *             token and place within an expert; -1 without a choice
 *   offsets   int32 [experts + 1]: expert e has rows offsets[e] .. offsets[e + 1] (as mlp_linear_forward
 *             takes them); offsets[experts] is the number of choices made
 *   counts    int32 [experts], or NULL
 *   loss      fp32 [1], or NULL: with M choices made and P_e the sum of p_e over the tokens that made one,
 *             experts * top / M^2 * sum_e counts_e P_e, 1 when all experts get the same (0 when M = 0)
 *   workspace >= mlp_route_workspace_size bytes, 256-byte aligned */
mlp_status mlp_route_forward(int64_t tokens, int64_t experts, int32_t top, const void *logits, int64_t ldl,
                             mlp_dtype dtype, const uint8_t *mask, int32_t normalize, float *gates,
                             int32_t *chosen, int32_t *slots, int32_t *offsets, int32_t *counts, float *loss,
                             void *workspace, void *stream);

mlp_status mlp_route_workspace_size(int64_t tokens, int64_t experts, size_t *bytes);

/* dlogits from the gradients of the gates (fp32 [tokens][top]; NULL: 0) and of the loss (fp32 [1] on the
 * device; NULL: 0).  The choices and counts are constants of the gradient.  chosen and offsets are those of the forward pass;
 * rows of tokens without a choice are zero.  An expert outside [0, experts) counts as no choice; a token's choices
 * differ from one another.  dlogits may be logits (same ld). */
mlp_status mlp_route_backward(int64_t tokens, int64_t experts, int32_t top, const void *logits, int64_t ldl,
                              mlp_dtype dtype, int32_t normalize, const int32_t *chosen, const int32_t *offsets,
                              const float *dgates, const float *dloss, void *dlogits, int64_t ldd, void *stream);

/* ------------------------------------------------------------------------ dispatch and combine --
 * `tokens` token rows and `rows` expert rows of `cols` elements, all of one dtype (BF16 or F32); slots
 * int32 [tokens][top] as mlp_route_forward writes them, a slot outside [0, rows) means no row; gates fp32
 * [tokens][top].  tokens, rows >= 0, cols >= 1, 1 <= top <= MLP_MAX_TOP.  tokens * top, rows and cols are below
 * 2^31, and so is tokens times the pieces of 128 bytes that a row of cols takes.  Sums are fp32, rounded once.
 * Expert rows that no slot names are neither read nor written.  Slots differ from one another.  Base
 * pointers aligned to their element; rows that are 16-byte aligned throughout run faster. */

/* y[slots[t][j]] = x[t] */
mlp_status mlp_dispatch_forward(int64_t tokens, int64_t cols, int32_t top, const void *x, int64_t ldx,
                                mlp_dtype dtype, const int32_t *slots, int64_t rows, void *y, int64_t ldy,
                                void *stream);

/* dx[t] = sum_j dy[slots[t][j]] + dx_add[t].  dx_add (NULL: none): a gradient that arrives by another path,
 * such as the router's; it may be dx (same ld). */
mlp_status mlp_dispatch_backward(int64_t tokens, int64_t cols, int32_t top, const void *dy, int64_t lddy,
                                 mlp_dtype dtype, const int32_t *slots, int64_t rows, const void *dx_add,
                                 int64_t ldadd, void *dx, int64_t lddx, void *stream);

/* y[t] = sum_j gates[t][j] z[slots[t][j]] + residual[t].  residual (NULL: none) may be y (same ld). */
mlp_status mlp_combine_forward(int64_t tokens, int64_t cols, int32_t top, const void *z, int64_t ldz,
                               mlp_dtype dtype, const float *gates, const int32_t *slots, int64_t rows,
                               const void *residual, int64_t ldr, void *y, int64_t ldy, void *stream);

/* dz[slots[t][j]] = gates[t][j] dy[t],  dgates[t][j] = sum_c dy[t][c] z[slots[t][j]][c] (0 without a row);
 * the residual's gradient is dy.  dz and dgates may each be NULL (not computed), z without dgates, gates
 * without dz.  dz may be z (same ld). */
mlp_status mlp_combine_backward(int64_t tokens, int64_t cols, int32_t top, const void *dy, int64_t lddy,
                                const void *z, int64_t ldz, mlp_dtype dtype, const float *gates,
                                const int32_t *slots, int64_t rows, void *dz, int64_t lddz, float *dgates,
                                void *stream);

#ifdef __cplusplus
}
#endif

#endif /* MLP_EXPERTS_H_ */

/*
 * mlp_block.h -- C ABI of the operators around the GEMM chain of mlp_chain.h that make up a pre-norm
 * MLP block, forward and backward (same library, libmlp_chain.so):
 *
 *   layer norm        y = (x - mean) rstd * gamma + beta, and its gradients;
 *   linear            Y = act(X W + b) + R with the bias, activation and residual in the product's
 *                     epilogue, and the gradients of X, W and b;
 *   linear by expert  the same product for rows grouped by expert: rows offsets[e] .. offsets[e+1] use
 *                     W[e] and b[e], any number of rows per expert, none included.
 *
 * Conventions (those of mlp_chain.h unless said here).
 *   - Device pointers on the handle's (or the current) device; `stream` is a cudaStream_t as void*.
 *     Every call only enqueues work on that stream; nothing synchronises, allocates or is kept between
 *     calls, so calls with different buffers may run on different streams at the same time.
 *   - Errors are returned, never thrown or trapped: INVALID_ARG for sizes, pointers, strides and
 *     alignments, UNSUPPORTED for a dtype or option the library does not implement, CUDA.
 *   - Strides (ld*) are in elements between rows; a row is contiguous.  They may exceed the row length
 *     (a slice of a wider matrix).  Inputs may alias one another but not an output; the exceptions are
 *     named at the call.
 *   - Gradients are written, not accumulated.
 */
#ifndef MLP_BLOCK_H_
#define MLP_BLOCK_H_

#include "mlp_chain.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ---------------------------------------------------------------------------------- layer norm --
 * rows x cols, both any size >= 0 (cols >= 1); x, y, dy, dx, dx_add of one dtype (BF16 or F32), gamma,
 * beta, dgamma, dbeta of one dtype (BF16 or F32); mean and rstd fp32, one per row.  All sums are fp32;
 * the variance is the mean of the squared deviations from the mean (no cancellation).  Base pointers
 * aligned to their element; rows that are 16-byte aligned throughout run faster.
 *   gamma NULL: 1; beta NULL: 0.  mean and rstd (forward) may be NULL.  y may be x. */
mlp_status mlp_layernorm_forward(int64_t rows, int64_t cols, const void *x, int64_t ldx, mlp_dtype dtype,
                                 const void *gamma, const void *beta, mlp_dtype w_dtype, float eps, void *y,
                                 int64_t ldy, float *mean, float *rstd, void *stream);

/* With xh = (x - mean) rstd and g = dy gamma:
 *   dx = rstd (g - mean(g) - xh mean(g xh)) + dx_add,  dgamma = sum_rows dy xh,  dbeta = sum_rows dy.
 * dx_add (NULL: none) is a gradient that reaches x by another path, such as the block's skip connection.
 * dx, dgamma and dbeta may each be NULL (not computed).  dx may be dy, x or dx_add (same ld).  The sums over
 * rows are taken in a fixed order: results do not change from run to run.  workspace: >=
 * mlp_layernorm_workspace_size bytes, 256-byte aligned (unused, may be NULL, without dgamma and dbeta). */
mlp_status mlp_layernorm_backward(int64_t rows, int64_t cols, const void *dy, int64_t lddy, const void *x,
                                  int64_t ldx, mlp_dtype dtype, const void *gamma, mlp_dtype w_dtype,
                                  const float *mean, const float *rstd, const void *dx_add, int64_t ldadd,
                                  void *dx, int64_t lddx, void *dgamma, void *dbeta, void *workspace,
                                  void *stream);

mlp_status mlp_layernorm_workspace_size(int64_t rows, int64_t cols, size_t *bytes);

/* -------------------------------------------------------------------------------------- linear -- */
typedef enum { MLP_ACT_NONE = 0, MLP_ACT_RELU = 1, MLP_ACT_GELU_TANH = 2, MLP_ACT_SILU = 3 } mlp_activation;

#define MLP_MAX_EXPERTS 1024

typedef struct {
    int64_t K, N;             /* input and output columns, multiples of 8                              */
    int32_t experts;          /* 0: one weight for all rows; E in 1..MLP_MAX_EXPERTS: W is E matrices,
                                 b is E x N, and every call takes the row offsets                       */
    int32_t weight_layout;    /* 0: K x N row-major; 1: N x K row-major (nn.Linear.weight)               */
    mlp_activation activation;
    mlp_dtype bias_dtype;     /* BF16 or F32: bias and its gradient                                     */
    mlp_dtype dw_dtype;       /* BF16 or F32: the weights' gradient                                     */
    int32_t device;
    uint32_t timeout_us;      /* limit of every device wait, the longest of which is for the reduction of a
                                 tile; work before the call on its stream does not count; 0 = 2 000 000 and
                                 one more for every 64 terms of the longest reduction                  */
} mlp_linear_desc;

typedef struct mlp_linear *mlp_linear_t;

mlp_status mlp_linear_create(const mlp_linear_desc *desc, mlp_linear_t *out);
mlp_status mlp_linear_destroy(mlp_linear_t h);

/* Bytes of workspace mlp_linear_backward needs for `rows` rows (mlp_linear_forward needs none). */
mlp_status mlp_linear_workspace_size(mlp_linear_t h, int64_t rows, size_t *bytes);

/* Y = act(Z) + R, Z = X W + b.  X: rows x K, Y, R, Z: rows x N, all bf16 with 16-byte aligned bases and
 * strides that are multiples of 8; W bf16, contiguous, 16-byte aligned; rows >= 0.  Products are
 * accumulated in fp32, bias, activation and residual are applied to the fp32 sum, and Y and Z are each
 * rounded once from it.
 *   bias NULL: 0.  residual NULL: none.  Z NULL: not stored (a backward pass with an activation needs
 * it).  residual may be Y (same stride).
 *   offsets (device, int32, experts + 1, ascending, 0 <= offsets[0], offsets[E] <= rows; NULL when
 * experts = 0).  Rows outside every expert's range are neither read nor written.  Offsets that are out
 * of order or range are clamped and make mlp_linear_check return INVALID_ARG. */
mlp_status mlp_linear_forward(mlp_linear_t h, int64_t rows, const void *X, int64_t ldx, const void *W,
                              const void *bias, const void *residual, int64_t ldr, const int32_t *offsets,
                              void *Z, int64_t ldz, void *Y, int64_t ldy, void *stream);

/* dZ = dY act'(Z), dX = dZ W^T, dW = X^T dZ (in W's layout), db = sum_rows dZ; the residual's gradient is dY.
 * dZ is rounded to bf16 for the two products (the tensor cores' operand type); db sums it unrounded.
 * Any of dX, dW, dbias may be NULL (not computed); Z may be NULL without an activation; X may be NULL
 * without dW, W without dX.  The gradients of an expert without rows are zero.  dX rows outside every
 * expert's range are not written.  Bad offsets are clamped and reported as above.  workspace: >=
 * mlp_linear_workspace_size bytes, 256-byte aligned. */
mlp_status mlp_linear_backward(mlp_linear_t h, int64_t rows, const void *dY, int64_t lddy, const void *X,
                               int64_t ldx, const void *W, const void *Z, int64_t ldz, const int32_t *offsets,
                               void *dX, int64_t lddx, void *dW, void *dbias, void *workspace, void *stream);

/* Synchronise `stream`, read the handle's device status word and clear it: OK, TIMEOUT, or INVALID_ARG
 * (bad offsets), the first that occurred.  After a TIMEOUT further calls of the handle store no output until this
 * is called (but for the zeros of a gradient without rows). */
mlp_status mlp_linear_check(mlp_linear_t h, void *stream);

/* The variant a product of this handle runs with for `rows` rows: pass 0 = Y, 1 = dX, 2 = dW. */
typedef struct {
    int32_t form;        /* 0: MMA rows are activation rows; 1: MMA rows are weight columns; 2: dW        */
    int32_t cta_pair;    /* 2: 256-row tiles on CTA pairs                                                 */
    int32_t tile_cols;   /* columns of a tile (activation rows in form 1)                                 */
    int32_t k_split;     /* CTAs sharing a tile's reduction                                               */
    int32_t pipe_stages;
} mlp_linear_plan;
mlp_status mlp_linear_get_plan(mlp_linear_t h, int64_t rows, int32_t pass, mlp_linear_plan *plan);

#ifdef __cplusplus
}
#endif

#endif /* MLP_BLOCK_H_ */

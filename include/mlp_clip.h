/*
 * mlp_clip.h -- C ABI of the global norm of many tensors and of clipping by it (same library,
 * libmlp_chain.so): what a training step does with all its gradients before the update.
 *
 * Conventions are those of mlp_block.h: device pointers on the current device, calls only enqueue on
 * `stream`, nothing is allocated or kept between calls, errors are returned.  The list of tensors is read
 * during the call and may be freed after it.  Results do not change from run to run.  A workspace is used from a
 * call's start to its end on the stream: calls that may run at the same time, replayed graphs among them,
 * need one each.
 */
#ifndef MLP_CLIP_H_
#define MLP_CLIP_H_

#include "mlp_chain.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef struct {
    const void *data;   /* `count` contiguous elements, aligned to their element (NULL if none)           */
    void *out;          /* of as many elements of the same type; may be data (clipped in place)          */
    int64_t count;      /* >= 0                                                                          */
    mlp_dtype dtype;    /* BF16 or F32                                                                   */
} mlp_tensor;

/* norm (fp32 [1] on the device) = the square root of the sum of the squares of all elements of all tensors.  Sums are fp32 with
 * the exponent's range kept: values whose squares leave it are summed scaled, so the norm of any finite values is finite, up to
 * fp32's largest value, and not 0 unless they are.  NaN and infinities in, NaN or infinity out.  `out` is not read.
 * 0 <= tensors <= 2^20, with fewer than 2^40 elements in all.
 * workspace: >= mlp_clip_workspace_size bytes, 256-byte aligned, apart from all tensors. */
mlp_status mlp_gradient_norm(int64_t tensors, const mlp_tensor *list, float *norm, void *workspace, void *stream);

/* The same, and out = c * data with c = max_norm / (norm + eps), 1 where that is larger (also for a norm of 0), rounded once.
 * Tensors that are clipped in place (out = data) are not written when c = 1.  max_norm >= 0 (infinity: c = 1), eps >= 0.
 * A norm of NaN makes c NaN, an infinite element makes c 0; finite elements whose norm is past fp32's largest value are scaled by
 * the norm itself.  c has fp32's 24 bits however small it is.
 * An out overlaps no other tensor's data or out; it is its own data, or does not overlap it.  norm lies in none of them, nor in the
 * workspace. */
mlp_status mlp_clip_gradients(int64_t tensors, const mlp_tensor *list, float max_norm, float eps, float *norm,
                              void *workspace, void *stream);

mlp_status mlp_clip_workspace_size(int64_t tensors, size_t *bytes);

#ifdef __cplusplus
}
#endif

#endif /* MLP_CLIP_H_ */

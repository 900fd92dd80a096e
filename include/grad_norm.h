/*
 * grad_norm.h - C ABI of the global gradient norm over many tensors, with the scale that clips
 * to a largest norm.
 *
 * What one call computes for gradients g_0 .. g_{n-1}:
 *   norms[i] = ||g_i||  (2-norm),   norm = sqrt(sum_i ||g_i||^2)
 *   scale    = max_norm / norm  if norm > max_norm,  else 1;  NaN if norm is NaN or infinite
 * Squares and sums are formed in double, so that every finite fp32 value is in range; norm,
 * scale and norms[i] are rounded to fp32 once (a norm beyond fp32's range is reported as
 * infinity, with the scale of its true value). The order of the sums depends on the plan
 * alone: equal inputs give equal bits.
 *
 * The scale can be applied in place (muon_grad_scale: for optimizers that take no scale) or
 * read by the step itself (adamw.h's grad_scale, which saves reading and writing the
 * gradients once more).
 *
 * Conventions are those of muon.h (device buffers, 16-byte alignment of the gradients,
 * validation before anything is enqueued, no synchronisation, no allocation). A plan is not
 * changed by a call. Calls that may overlap on the device need a workspace each.
 */
#ifndef MUON_GRAD_NORM_H
#define MUON_GRAD_NORM_H

#include "muon.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef struct muon_grad_plan muon_grad_plan; /* opaque; holds host metadata only */

/* Builds a plan for n gradients (n >= 0) of numel[i] contiguous elements (in [0, 2^35]) and
 * dtype[i]. Host-only: makes no HIP call. On success *out owns the plan (release it with
 * muon_grad_plan_destroy); on failure *out is set to NULL. */
int muon_grad_plan_create(muon_grad_plan **out, const int64_t *numel, const muon_dtype *dtype,
                          int64_t n);

/* Bytes of device workspace that muon_grad_norm needs on this plan (16-byte aligned, no
 * initial contents required, not preserved between calls). 0 for a NULL plan. */
size_t muon_grad_plan_workspace_size(const muon_grad_plan *plan);

/* out[0] = norm, out[1] = scale; norms: NULL, or n fp32 that receive each gradient's norm.
 * grads[0..n-1] (n the plan's count) are read only; one may stand in the list more than once
 * and then counts each time; NULL counts as zero. max_norm >= 0, infinity for no clipping.
 * With n = 0 the norm is 0. */
int muon_grad_norm(const muon_grad_plan *plan, const void *const *grads, int64_t n,
                   float max_norm, float *out, float *norms, void *workspace,
                   size_t workspace_bytes, hipStream_t stream);

/* grads[i] <- round(*scale * grads[i]) in place, for each i (NULL: none); scale: one fp32 on
 * the device. Where *scale is 1 nothing is read or written. No gradient may overlap another. */
int muon_grad_scale(const muon_grad_plan *plan, void *const *grads, int64_t n,
                    const float *scale, hipStream_t stream);

void muon_grad_plan_destroy(muon_grad_plan *plan); /* NULL is ignored */

#ifdef __cplusplus
}
#endif
#endif /* MUON_GRAD_NORM_H */

/*
 * adamw.h - C ABI of the library's AdamW step over many tensors at once, with the two moments
 * held in fp32 or in 8 bits.
 *
 * What one step computes for every element of every tensor (t = cfg->step, counting from 1;
 * s = *cfg->grad_scale, or 1 without it):
 *   g  = s * grad
 *   m <- beta1 m + (1 - beta1) g
 *   v <- beta2 v + (1 - beta2) g^2
 *   u  = (m / (1 - beta1^t)) / (sqrt(v) / sqrt(1 - beta2^t) + eps)
 *   p <- p - lr (u + weight_decay * wd_mul * p)
 * p is the fp32 master copy where the tensor has one (the parameter then receives its rounded
 * value and is not read), else the parameter itself. Arithmetic is fp32; a bf16 parameter is
 * rounded to nearest even once, after the update. 1 - beta^t is formed in double on the host.
 *
 * 8-bit states (MUON_ADAMW_8BIT). Each tensor's elements are taken in blocks of 256 in their
 * memory order (the last one may be shorter). A block holds m and r = sqrt(v), one byte of
 * e4m3 (OCP, no infinities, largest value 448) each, and for each of the two a power-of-two
 * scale 2^(b - 127), b one byte (e8m0):
 *   b is the smallest byte with max |x| <= T * 2^(b - 127) over the block, x = m or r, where
 *   T = 256 * (1 + 0x629146 / 2^23) = 453.137 (values between 448 and T are held as 448);
 *   m is rounded to nearest even;
 *   r is rounded to nearest even, or stochastically (cfg->stochastic): up with the probability
 *   of what is cut off, by 16 bits drawn from (cfg->seed, cfg->step, the element's index);
 *   an r over zero is held as 2^-9 of its scale at least, so v = 0 only where it is 0.
 * The step uses the new m and v before they are rounded for storage. In this form m, v and r
 * are formed operation by operation, each rounded to fp32, in the order written above: stored
 * bytes do not depend on how the compiler contracts products and sums.
 * Why r and not v: its range is half of v's in the exponent. Why a floor: |u| stays bounded,
 * since an element's m cannot outlive its v. Why stochastic: beta2 = 0.999 moves v by at most
 * 0.1% a step unless the gradient jumps, and half a step of the format is 3% or more, so that
 * rounding to nearest would leave v where it is.
 * The random bits: with e the element's index in its tensor, j = e / 2, all in 32 bits,
 *   h(x): x ^= x >> 16; x *= 0xEB26D985; x ^= x >> 15; x *= 0x4A08C6ED; x ^= x >> 16
 *   bits = h(low32(j) ^ key ^ high32(j) * 0xEB26D985): the low 16 for even e, the high for odd
 *   r's code is the truncation, to the format, of r + (bits + 1/2) / 65536 of a step of it;
 *   key: z = seed + step * 0x1493FA689CA113AD in 64 bits, twice z = (z ^ z >> 32) *
 *   0xE9F8AC216EBC06F5, then the low 32 bits of z ^ z >> 32.
 * Elements of equal index in different tensors draw the same bits.
 *
 * NaN and infinities are propagated and never leave their tensor. In the 8-bit form a NaN
 * stays NaN in m and v; an infinite m is held as NaN and takes its block's scale to the
 * largest, so that the block's other m become 0; a finite |m| over 240 * 2^120 is held as that,
 * the largest finite code there; an r over 240 * 2^56 (a v over 0.88 * 2^128, infinity
 * included) is held as 240 * 2^56, the largest code whose square is finite.
 * cfg->skip_nonfinite is the guard against what is not finite. An eps below 2^-126 counts as 0.
 *
 * Conventions are those of muon.h: device buffers on the current HIP device, contiguous, owned
 * by the caller, 16-byte aligned base addresses (the scales' need no alignment); work enqueued
 * on `stream` without synchronising; arguments validated on the host before anything is
 * enqueued. A step allocates nothing, and a plan is not changed by a step: steps on one plan
 * may be called from several host threads, but the buffers they update are the plan's, so that
 * the steps themselves must be ordered on the device. A captured step replays with the cfg it
 * was captured with, step index and seed included; the plan's buffers and its table must stay
 * allocated as long as the graph is replayed.
 */
#ifndef MUON_ADAMW_H
#define MUON_ADAMW_H

#include "muon.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef struct muon_adamw_plan muon_adamw_plan; /* opaque; holds host metadata only */

typedef enum { MUON_ADAMW_F32 = 0, MUON_ADAMW_8BIT = 1 } muon_adamw_state;

/* Elements of one block of the 8-bit states. */
#define MUON_ADAMW_BLOCK 256

/* One tensor, viewed as numel contiguous elements (any shape).
 *   param             param_dtype, updated in place
 *   master            NULL, or for a bf16 parameter numel fp32: the master copy, updated in
 *                     place (param is then written only)
 *   exp_avg           m: numel fp32, or numel bytes of e4m3
 *   exp_avg_sq        v: numel fp32, or r: numel bytes of e4m3
 *   exp_avg_scale     8-bit states: ceil(numel / 256) bytes of e8m0; ignored otherwise
 *   exp_avg_sq_scale  likewise
 *   numel             in [0, 2^35]; a tensor with numel 0 is skipped, its pointers may be NULL
 *   wd_mul            finite multiplier of cfg->weight_decay for this tensor
 * Zero-fill every state and scale buffer before step 1. No buffer may overlap another. */
typedef struct {
  void *param;
  float *master;
  void *exp_avg;
  void *exp_avg_sq;
  uint8_t *exp_avg_scale;
  uint8_t *exp_avg_sq_scale;
  int64_t numel;
  muon_dtype param_dtype;
  muon_dtype grad_dtype;
  float wd_mul;
} muon_adamw_tensor;

/* Hyper-parameters of one step, shared by the plan's tensors. lr, eps and weight_decay are
 * finite with eps >= 0; beta1 and beta2 are in [0, 1); step >= 1.
 *   grad_scale      NULL, or one fp32 on the device that every gradient is multiplied by (the
 *                   scale that muon_grad_norm writes); read when the step runs
 *   skip_nonfinite  1: if *grad_scale is NaN or infinite when the step runs, the step leaves
 *                   every buffer as it was (needs grad_scale)
 *   stochastic      8-bit states: 1 rounds r stochastically, 0 to nearest; ignored otherwise
 *   seed            of the stochastic rounding */
typedef struct {
  float lr;
  float beta1;
  float beta2;
  float eps;
  float weight_decay;
  int64_t step;
  const float *grad_scale;
  int skip_nonfinite;
  int stochastic;
  uint64_t seed;
} muon_adamw_config;

/* Fills cfg with lr 1e-3, beta1 0.9, beta2 0.999, eps 1e-8, weight_decay 0.01, step 1,
 * grad_scale NULL, skip_nonfinite 0, stochastic 1, seed 0. A NULL cfg is ignored. */
void muon_adamw_config_default(muon_adamw_config *cfg);

/* Builds a plan for tensors[0..n-1] (n >= 0), whose buffers it keeps the addresses of: they
 * must stay allocated as long as the plan is used. Host-only: makes no HIP call. On success
 * *out owns the plan (release it with muon_adamw_plan_destroy); on failure *out is NULL. */
int muon_adamw_plan_create(muon_adamw_plan **out, const muon_adamw_tensor *tensors, int64_t n,
                           muon_adamw_state state);

/* Bytes of the plan's device table (what a step reads of the tensors but the gradients'
 * addresses). 0 for a NULL plan and one without elements. */
size_t muon_adamw_plan_table_size(const muon_adamw_plan *plan);

/* Fills the table, 16-byte aligned device memory of the caller's that must stay allocated and
 * untouched as long as the plan is used, by work on `stream`; steps on other streams have to be
 * ordered behind it. Needed once before the plan's first step (unless its table size is 0). Not
 * for a stream under capture: the table would first be filled by the graph's replay. */
int muon_adamw_plan_upload(muon_adamw_plan *plan, void *table, size_t table_bytes,
                           hipStream_t stream);

/* One AdamW step over the plan's tensors with gradients grads[0..n-1] (n the plan's count;
 * grads[i] of tensor i's grad_dtype, read only, may be shared between tensors, must not
 * overlap a buffer of the plan; NULL leaves tensor i out of this step). */
int muon_adamw_step(const muon_adamw_plan *plan, const void *const *grads, int64_t n,
                    const muon_adamw_config *cfg, hipStream_t stream);

/* What muon_adamw_step would return of its arguments, without the step: for a caller whose step
 * is several calls, so that none is made where a later one would be refused. */
int muon_adamw_check(const muon_adamw_plan *plan, const void *const *grads, int64_t n,
                     const muon_adamw_config *cfg);

void muon_adamw_plan_destroy(muon_adamw_plan *plan); /* NULL is ignored */

#ifdef __cplusplus
}
#endif
#endif /* MUON_ADAMW_H */

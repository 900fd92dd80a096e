/*
 * orthogonalize.h - C ABI of the Newton-Schulz orthogonalisation of a stack of small matrices
 * (attention heads, low-rank factors: the shorter side up to 128), strided as they lie in a
 * larger tensor, in one set of launches.
 *
 * What it computes for every matrix X of the stack (short side s, long side l, X taken with the
 * short side as its rows): X_0 = X / (||X||_F + eps), then per round X <- (a I + b A + c A A) X,
 * A = X X^T: the rounds of muon.h, with its coefficients, schedules and limits on rounds. Here
 * the rounds run on the Gram matrix alone: every X_r is P_r X_0 with P_r a polynomial of
 * A_0 = X_0 X_0^T, so the stack is read once for A_0 and once for P X_0, whatever the rounds.
 * A small singular value is known from A_0 to the square root of its precision only, and so the
 * Gram matrix and the rounds are formed in double (bf16 stacks: of sums of 32 exact products in
 * fp32, where fp32's range holds them) and P is rounded to fp32 once; the result is as exact as
 * rounds in fp32 on X itself, or rounded to bf16 once where that is its dtype. The sums in fp32 leave
 * A_0 (trace 1, long side l) off by up to about 2^-19 / sqrt(l) in norm; after five rounds of the
 * default coefficients that is a small part of what rounding the result to bf16 takes.
 *
 * Rounds that could lift a direction of X by more than 2^15 in all (eight of the default coefficients
 * lift by 2^14.3) are done in several passes over the stack, each with a Gram matrix of its own, as the
 * rounds on a matrix without full rank otherwise run off. Between passes an fp32 stack is held in out;
 * a bf16 stack is refused for such rounds (MUON_ERR_UNSUPPORTED): convert it to fp32. bf16 stacks
 * whose rounds lift by more than 2^9 (five of the default ones: 485) are summed in double.
 *
 * Every finite value of either dtype is in range. A matrix of zeros gives zeros (for eps > 0). A NaN or
 * infinity makes its own matrix NaN and no other. Equal inputs give equal bits, wherever in a
 * stack a matrix stands, as long as the stack's sizes are equal.
 *
 * Conventions are those of muon.h, but that stacks need be aligned to their elements only.
 */
#ifndef MUON_ORTHOGONALIZE_H
#define MUON_ORTHOGONALIZE_H

#include "muon.h"

#ifdef __cplusplus
extern "C" {
#endif

/* The stack: outer * inner matrices of rows x cols; element (o, i, r, c) at
 * o * stride[0] + i * stride[1] + r * stride[2] + c * stride[3] elements. One of stride[2] and
 * stride[3] must be 1 (or its side 1). The same strides hold for the result, whose elements
 * must have places of their own. */
typedef struct {
  const void *in;
  void *out;
  int64_t outer, inner, rows, cols;
  int64_t in_stride[4];
  int64_t out_stride[4];
  muon_dtype dtype; /* of both */
} muon_stack;

/* Bytes of workspace (256-byte aligned, no initial contents required) that a stack of these
 * sizes needs; 0: none. SIZE_MAX for sizes outside the limits (min(rows, cols) <= 128, max <= 2^24,
 * outer * inner <= 2^24). */
size_t muon_orthogonalize_workspace_size(int64_t outer, int64_t inner, int64_t rows, int64_t cols);

/* The passes over a stack that the rounds of cfg take (ns_steps, a, b, c, schedule; above), 1 or more,
 * or the (negative) status of a configuration that is refused. */
int muon_orthogonalize_passes(const muon_config *cfg);

/* out <- the orthogonalised matrices; of cfg: ns_steps (>= 0), a, b, c, schedule and eps. in and
 * out may not overlap (but in == out with equal strides is taken: in place). */
int muon_orthogonalize(const muon_stack *stack, const muon_config *cfg, void *workspace,
                       size_t workspace_bytes, hipStream_t stream);

#ifdef __cplusplus
}
#endif
#endif /* MUON_ORTHOGONALIZE_H */

/*
 * What stands around the routed experts in a layer, for any number of tokens,
 * as calls beside those of moe_rows.h:
 *
 *   moe_dense_gemm          a dense product with bias, activation and residual:
 *                           the router's logits, projections into and out of a
 *                           latent, the products of a dense expert in BF16
 *   moe_route_rows_scored   routing by sigmoid or softmax scores, limited to the
 *                           best groups of experts, and the tokens grouped by
 *                           expert as moe_route_rows does
 *   moe_join_rmsnorm_quant  a block's output normalised, gated and added to the
 *                           scaled residual, the sum normalised for the next
 *                           block in BF16 and 8 bits
 *
 * The conventions are moe_rows.h's: same library, number formats and error
 * codes; every call enqueues one to three kernels on `stream` (a hipStream_t
 * of the current device; NULL is the default stream), allocates nothing, never
 * synchronises, issues no memset and keeps nothing between calls, so that it
 * can be captured into a HIP graph and calls on different streams are
 * independent (each call in flight needs its own workspace). All pointers are
 * device pointers; outputs overlap no input (but for residual_out, below) and
 * no other output. Nothing is enqueued on an error: INVALID_ARG (negative
 * size, NULL or misaligned pointer, bad value), UNSUPPORTED (sizes or options
 * outside the limits), SCRATCH_TOO_SMALL, HIP (launch failure).
 */
#ifndef MOE_BLOCK_H
#define MOE_BLOCK_H

#include <stddef.h>
#include <stdint.h>

#include "moe_rows.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Activations of moe_dense_gemm. */
#define MOE_ACT_NONE 0
#define MOE_ACT_RELU 1      /* max(v, 0) */
#define MOE_ACT_SILU 2      /* v / (1 + exp(-v)) */
#define MOE_ACT_GELU 3      /* v / 2 (1 + erf(v / sqrt 2)) */
#define MOE_ACT_GELU_TANH 4 /* v / 2 (1 + tanh(sqrt(2 / pi) (v + 0.044715 v^3))) */
#define MOE_ACT_SIGMOID 5   /* 1 / (1 + exp(-v)) */

#define MOE_DENSE_MAX_DIM 1048576 /* N and K of moe_dense_gemm */

/* For each row t < T and column n < N:
 *   v = sum_c x[t, c] * w[n, c]    exact products of BF16 values, FP32 sums
 *   v = act(v + bias[n]), then v + residual[t, n], in FP32
 *   out[t, n] = v in FP32 or rounded once to BF16
 *   x        [T, K] BF16, rows ldx values apart
 *   w        [N, K] BF16, rows ldw values apart
 *   bias     [N] FP32 or BF16 (bias_dtype), or NULL
 *   residual [T, N] FP32 or BF16 (residual_dtype), rows ldr values apart, or NULL
 *   out      [T, N] FP32 or BF16 (out_dtype), contiguous
 * The sums of a row are taken in an order that T, N and K choose, so its last
 * FP32 bits may differ between calls of other sizes; they do not depend on the
 * other rows' values, and the same call gives the same bits every time. An
 * infinity or NaN in x or w reaches its own row or column of the output only.
 * Activations are within 4 * 2^-23 of their value (GELU and the tanh form: of
 * |v| where the value is small beside it) in FP32; values under 2^-118 may be 0.
 * ReLU keeps a NaN, an infinity is what the formula makes of it.
 *   workspace: NULL, or 16-byte aligned device memory of at least
 *   moe_dense_gemm_workspace bytes, with which calls that would leave compute
 *   units idle are split over K (SCRATCH_TOO_SMALL where it is shorter). Its
 *   contents need no preparation and mean nothing after the call; calls in
 *   flight at once need one each.
 * K a multiple of 8; N and K from 1 (8) to MOE_DENSE_MAX_DIM; 0 <= T <=
 * MOE_ROWS_MAX_TOKENS; ldx and ldw multiples of 8, at least K, ldr at least N, all
 * below 2^23;
 * rows of x, w 16-byte aligned, bias, residual to their element, out 16 bytes.
 * Strides of a tensor with a single row are not read. T = 0 is a valid empty
 * call. */
typedef struct moe_dense_args {
  int32_t T, N, K;
  int32_t act;            /* MOE_ACT_* */
  int32_t out_dtype;      /* MOE_DTYPE_F32 or MOE_DTYPE_BF16 */
  int32_t bias_dtype;     /* of bias, where there is one */
  int32_t residual_dtype; /* of residual, where there is one */
  int64_t ldx, ldw, ldr;
  const void* x;
  const void* w;
  const void* bias;
  const void* residual;
  void* out;
  void* workspace;
  size_t workspace_bytes;
} moe_dense_args;
int moe_dense_gemm(const moe_dense_args* a, void* stream);

/* Bytes of workspace with which a call of these sizes splits K over workgroups
 * (0 where it would not). */
size_t moe_dense_gemm_workspace(int32_t T, int32_t N, int32_t K);

/* Scores of moe_route_rows_scored. */
#define MOE_SCORES_SIGMOID 0 /* 1 / (1 + exp(-z)) */
#define MOE_SCORES_SOFTMAX 1 /* exp(z) / sum_e exp(z_e) over all E experts */

#define MOE_ROUTE_MAX_GROUPS 64

/* Routes T tokens and groups the routes by expert, as moe_route_rows but for
 * the picks:
 *   s_e   = the score of expert e in FP64, rounded to FP32 (a softmax row whose
 *           logits are all minus infinity has scores of 0)
 *   key_e = s_e + bias[e] in FP32 (s_e without a bias)
 *   Experts are in `groups` runs of E / groups. A group's value is its largest
 *   key (group_best = 1) or the FP32 sum of its two largest (2); the top_groups
 *   groups of the largest values take part, of equal ones the lower.
 *   ids   = the k largest keys of theirs, largest first, of equal ones the lower expert
 *   weights = (s / total) * routed_scale with renormalise, where total is the
 *           FP32 sum of the picked scores in their order (weights of 0 where it
 *           is 0); otherwise s * routed_scale
 * bias may be NULL. A NaN among a token's logits, of either sign, or in the bias makes
 * all of its weights NaN, plus infinity its softmax weights; its ids are still k
 * different experts. Of minus infinity (an expert switched off) the score is 0, of plus
 * infinity the sigmoid 1.
 * 1 <= groups <= MOE_ROUTE_MAX_GROUPS, a divisor of E; 1 <= top_groups <=
 * groups; group_best 1 or 2, at most E / groups; k <= top_groups * E / groups;
 * all else as in moe_route_rows, moe_route_rows_workspace among it. */
typedef struct moe_route_scored_args {
  moe_route_args route;
  int32_t scores; /* MOE_SCORES_* */
  int32_t groups, top_groups, group_best;
  int32_t renormalise; /* 0 or 1 */
} moe_route_scored_args;
int moe_route_rows_scored(const moe_route_scored_args* a, void* stream);

/* Gates of moe_join_rmsnorm_quant. */
#define MOE_GATE_NONE 0
#define MOE_GATE_ROW 1    /* [T], one value for a token */
#define MOE_GATE_COLUMN 2 /* [D], one value for a column */
#define MOE_GATE_FULL 3   /* [T, D] */

/* Between two blocks of a layer that normalises each block's output as well
 * as its input. For each token t:
 *   b = delta[t] + sum_j weights[t, j] * y[pos[t, j]]
 *       summed in FP64 in this order and rounded to FP32 (a position outside
 *       [0, R) adds nothing);
 *   n = (b * rstd(b)) * (post_gamma + gamma_offset) in FP32, or b without post_gamma,
 *       rstd(b) = FP32(1 / sqrt(sum_i b_i^2 / D + post_eps)), the statistics in FP64;
 *   h = gate * n + residual_scale * residual[t] of exact products, rounded to FP32
 *       once (by way of FP64 unless residual_scale is a multiple of 2^-15 up to 1);
 *   v = (h * rstd(h)) * (gamma + gamma_offset) in FP32, with eps, or h without gamma;
 *   residual_out[t] = BF16(h), out[t] = BF16(v), q[t] and scale[t] = the 8-bit
 *   form of v (not of BF16(v)).
 * T and k choose the order of the statistics' sums, which may move the last bit of
 * a value next to a rounding border; the same call gives the same bits.
 *   norm   sizes, quantisation and arrays as in moe_add_rmsnorm_quant;
 *          residual may be NULL (0), delta and the routed rows not both;
 *          residual_out may be `residual` or `delta` itself
 *   post_gamma [D] BF16 or NULL
 *   gate   by gate_kind: [T] FP32 or BF16 (gate_dtype), [D] or [T, D] BF16, 16-byte
 *          aligned ([T]: to its element); NULL with MOE_GATE_NONE
 * eps, post_eps >= 0; these, residual_scale and gamma_offset finite. */
typedef struct moe_join_args {
  moe_norm_args norm;
  float post_eps, residual_scale, gamma_offset;
  int32_t gate_kind;  /* MOE_GATE_* */
  int32_t gate_dtype; /* MOE_DTYPE_F32 or MOE_DTYPE_BF16 */
  const void* post_gamma;
  const void* gate;
} moe_join_args;
int moe_join_rmsnorm_quant(const moe_join_args* a, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* MOE_BLOCK_H */

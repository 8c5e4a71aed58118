/*
 * The routed-expert step for any number of tokens (prompts, batches of
 * requests), as calls that a serving program makes one after the other:
 *
 *   moe_add_rmsnorm_quant  residual + addend + weighted expert rows, RMSNorm,
 *                          BF16 and 8-bit outputs with scales
 *   moe_route_rows         router logits -> picks, weights, and the tokens
 *                          grouped by expert
 *   moe_grouped_swiglu     each expert's W13 with its own rows, clamped
 *                          SwiGLU, 8-bit hidden with scales
 *   moe_grouped_gemm       each expert's W2 with its own rows
 *   moe_add_rmsnorm_quant  again: the routing weights are applied here, once
 *
 * The arithmetic is that of moe_decode.h (which handles up to 256 tokens
 * behind one handle) and of moe_boundary.h; the weights are in the same
 * layouts. Same library, number formats and error codes. Every call enqueues
 * one to three kernels on `stream` (a hipStream_t of the current device; NULL
 * is the default stream), allocates nothing, never synchronises, issues no
 * memset and keeps nothing between calls: it can be captured into a HIP graph
 * and calls on different streams are independent (each call in flight needs
 * its own workspace).
 *
 * All pointers are device pointers, arrays row-major and contiguous; outputs
 * overlap no input (but for residual_out, below) and no other output. Nothing
 * is enqueued on an error: INVALID_ARG (negative size, NULL or misaligned
 * pointer, bad value), UNSUPPORTED (sizes or options outside the limits),
 * HIP (launch failure).
 */
#ifndef MOE_ROWS_H
#define MOE_ROWS_H

#include <stddef.h>
#include <stdint.h>

#include "moe_decode.h"

#ifdef __cplusplus
extern "C" {
#endif

/* 8-bit formats of activations: OCP e4m3 codes with
 *   MOE_QUANT_FP8     an FP32 scale per 128 values: s = max(amax, 1e-10) / 448,
 *                     q = e4m3(v * (1 / s))
 *   MOE_QUANT_FP8_P2  the same with s rounded up to a power of two (from at
 *                     least 1e-10)
 *   MOE_QUANT_MXFP8   an E8M0 byte b (2^(b - 127)) per 32 values:
 *                     b - 127 = floor(log2 amax) - 8 within [-127, 127] (-127
 *                     for a block of zeros), q = e4m3(v * 2^-(b - 127))
 * rounded to nearest even, saturating. A NaN keeps its place as a NaN code;
 * it takes no part in its block's amax. */
#define MOE_QUANT_NONE 0
#define MOE_QUANT_FP8 1
#define MOE_QUANT_FP8_P2 2
#define MOE_QUANT_MXFP8 3

#define MOE_ROWS_MAX_D 16384         /* longest row of moe_add_rmsnorm_quant */
#define MOE_ROWS_MAX_TOKENS 1048576  /* tokens of one moe_add_rmsnorm_quant or moe_route_rows call */
#define MOE_ROWS_MAX_DIM 131072      /* N and K of the grouped products */

/* Passages: "kimi_k3 ... ep.comm" page, EpCombine and rms_rstd (sum of a
 * token's rows in FP32 or more, then RMSNorm), EpDispatch (MXFP8), "mega_moe"
 * page, epilogue (FP8 per 128), nvfp4-megamoe-kernel README (routing weights
 * applied once, to the unweighted expert rows). For each token t:
 *   h = residual[t] + delta[t] + sum_j weights[t, j] * y[pos[t, j]]
 *       summed in FP64 in this order and rounded to FP32: the correctly
 *       rounded sum but next to a rounding border and where terms of 2^29 times
 *       the result and more cancel; a position outside [0, R) adds nothing (expert not local);
 *   residual_out[t] = BF16(h);
 *   rstd = FP32(1 / sqrt(sum_i h_i^2 / D + eps)), the statistics in FP64
 *       (T and k choose the order of this sum, which may move rstd's last bit
 *       next to a rounding border; the same call gives the same bits);
 *   v = (h * rstd) * gamma, two FP32 products (v = h when gamma is NULL);
 *   out[t] = BF16(v); q[t], scale[t] = the 8-bit form of v (not of BF16(v)).
 *   residual     [T, D] BF16, or NULL (0)
 *   delta        [T, D] BF16, or NULL (0)
 *   y            [R, D] BF16, pos [T, k] int32, weights [T, k] FP32; all
 *                three NULL and k = 0 when there are no routed rows
 *   gamma        [D] BF16, or NULL for no normalisation
 *   residual_out [T, D] BF16 or NULL; may be `residual` or `delta` itself
 *   out          [T, D] BF16 or NULL
 *   q            [T, D] e4m3 and scale [T, D/128] FP32 or [T, D/32] bytes
 *                (by `quant`); both NULL with MOE_QUANT_NONE
 * BF16 and e4m3 arrays 16-byte
 * aligned, the others to their element. D a multiple of 128 (FP8), 32 (MXFP8)
 * or 8 (no quantisation) up to MOE_ROWS_MAX_D; T <= MOE_ROWS_MAX_TOKENS;
 * 0 <= k <= 32; eps >= 0, finite. At least one output and at least one of residual, delta, y.
 * T = 0 is a valid empty call. */
typedef struct moe_norm_args {
  int32_t T, D, k, R;
  float eps;
  int32_t quant; /* MOE_QUANT_* */
  const void* residual;
  const void* delta;
  const void* y;
  const int32_t* pos;
  const float* weights;
  const void* gamma;
  void* residual_out;
  void* out;
  void* q;
  void* scale;
} moe_norm_args;
int moe_add_rmsnorm_quant(const moe_norm_args* a, void* stream);

/* Passage: "mega_moe" page, top_k_pick and _ordered (the routing of
 * moe_decode_run, the same arithmetic: ids are bit-identical to it).
 * Routes T tokens and groups the routes by expert:
 *   ids     [T, k] int32: picked experts, highest biased score first
 *   weights [T, k] FP32
 *   offsets [local_experts + 1] int32: the rows of local expert e are
 *           offsets[e] .. offsets[e + 1] - 1
 *   rows    [T * k] int32: the token of each grouped row; within an expert
 *           tokens ascend. Entries from offsets[local_experts] on are left
 *           as they were (none when every expert is local)
 *   pos     [T, k] int32: the grouped row of each pick, -1 for a pick whose
 *           expert lies outside [local_begin, local_begin + local_experts)
 *   logits  [T, E] FP32 or BF16 (logits_dtype), bias [E] FP32
 *   workspace: 4-byte aligned device memory of at least
 *           moe_route_rows_workspace(T, local_experts) bytes; its contents need no
 *           preparation and mean nothing after the call. May be NULL when
 *           that size is 0.
 * 1 <= k <= min(E, 32), E <= 1024, 0 <= T <= MOE_ROWS_MAX_TOKENS,
 * routed_scale finite, local_experts >= 1 within [0, E). T = 0 writes zero
 * offsets and touches nothing else: every other pointer may be NULL then. */
typedef struct moe_route_args {
  int32_t T, E, k;
  int32_t logits_dtype; /* MOE_DTYPE_F32 or MOE_DTYPE_BF16 */
  int32_t local_begin, local_experts;
  float routed_scale;
  const void* logits;
  const float* bias;
  int32_t* ids;
  float* weights;
  int32_t* offsets;
  int32_t* rows;
  int32_t* pos;
  void* workspace;
  size_t workspace_bytes;
} moe_route_args;
int moe_route_rows(const moe_route_args* a, void* stream);

/* Bytes of workspace moe_route_rows needs (0 for few tokens). */
size_t moe_route_rows_workspace(int32_t T, int32_t local_experts);

/* Products grouped by expert ("mega_moe" page, module docstring: every
 * 128-wide K block's partial is multiplied by its weight and activation scale
 * once). Grouped row i, offsets[e] <= i < offsets[e + 1], belongs to expert e
 * and reads activation row r = rows ? rows[i] : i:
 *   g[i, n] = sum_b w_scale[e, n/128, b] * sum_{c in block b} w[e, n, c] * x[r, c] * x_scale
 * with FP32 sums.
 *   x        [X, K] e4m3 with x_scale [X, K/128] FP32 (MOE_QUANT_FP8 or
 *            MOE_QUANT_FP8_P2) or [X, K/32] E8M0 bytes (MOE_QUANT_MXFP8);
 *            no E8M0 byte 255. Scales whose product with w_scale is finite
 *            (MXFP8: any, with w_scale below 2^64)
 *   rows     [R] int32 or NULL (then X >= R); an index outside [0, X) gives
 *            a row of zeros
 *   offsets  [E + 1] int32, ascending from 0 to at most R; rows from
 *            offsets[E] on are not written. Every value is clamped to [0, R]
 *            before its use, so offsets that are not so give wrong rows but
 *            no access out of bounds
 *   w        [E, N, K] e4m3, w_scale [E, N/128, K/128] FP32
 *   R        rows of the output
 * moe_grouped_gemm: out [R, N] BF16 = g, rounded once. With sums =
 *   MOE_SUMS_FP8 by the FP8 matrix instruction, faster where rows are many: it
 *   adds the products of eight neighbouring columns cut off 14 bits below the
 *   power of two of the largest, and these sums in FP32: off by some 2^-16 of a
 *   row's typical value before the rounding to BF16 (2^-9), but by up to 2^-11 of
 *   a group's largest product, which is all of the result where the large ones
 *   cancel; and E8M0 scales may take a block's sum past FP32 before w_scale
 *   brings it back.
 * moe_grouped_swiglu: w = W13, N = 2I rows (0..I-1 up, I..2I-1 gate):
 *   up = clamp(g[n], +-limit), gate = min(g[I + n], limit),
 *   act = gate / (1 + exp(-gate)) * up,
 *   out [R, I] e4m3 with out_scale [R, I/128] FP32: MOE_QUANT_FP8 of act
 *   ("mega_moe" page, hidden_block). act is within (5 + |gate| / 42) * 2^-23 of
 *   its value for the FP32 sums (the hardware's exp2 and reciprocal; a gate below
 *   -87 counts as -87). By the format's definition it is multiplied by the
 *   reciprocal of its scale, where moe_decode_run divides: a code next to a
 *   rounding border may differ from that call's.
 * workspace: NULL, or 16-byte aligned device memory of at least
 *   moe_grouped_gemm_workspace / moe_grouped_swiglu_workspace bytes, with which
 *   small calls are split over K, up to 3.6 times faster (SCRATCH_TOO_SMALL
 *   where it is shorter). Its contents need no preparation and mean nothing
 *   after the call; calls in flight at once need one each. Parts of K are
 *   added in FP32, in order; their number depends on R, E, N and K alone.
 * The same call gives the same bits every time. The last FP32 bits of a row's
 * sums may depend on R and E, on how many rows its expert has and, where K is a
 * multiple of 4096, on the expert's index, so that an expert's rows may differ in
 * them between calls for all experts and for a share of them; never on what is in
 * other rows or on the row's place among its expert's.
 * K and N multiples of 128 (N of 256 for the SwiGLU), at most
 * MOE_ROWS_MAX_DIM; E <= 1024; X, R >= 0, at most 2^23 - 9 tiles of work
 * (floor(R/128) + E rows of ceil(N/256) tiles). FP8 and output arrays 16-byte aligned, E8M0
 * bytes 4-byte aligned, the others to their element. R = 0 is a valid empty
 * call. */
#define MOE_SUMS_FP32 0
#define MOE_SUMS_FP8 1
typedef struct moe_grouped_args {
  int32_t R, X, E, N, K;
  int32_t quant;     /* of x: MOE_QUANT_FP8, MOE_QUANT_FP8_P2 or MOE_QUANT_MXFP8 */
  float limit;       /* moe_grouped_swiglu: > 0; above 2^127 it counts as that */
  const void* x;
  const void* x_scale;
  const int32_t* rows;
  const int32_t* offsets;
  const void* w;
  const float* w_scale;
  void* out;
  float* out_scale;  /* moe_grouped_swiglu */
  void* workspace;
  size_t workspace_bytes;
  int32_t sums;      /* moe_grouped_gemm: MOE_SUMS_*; else MOE_SUMS_FP32 */
} moe_grouped_args;
int moe_grouped_gemm(const moe_grouped_args* a, void* stream);
int moe_grouped_swiglu(const moe_grouped_args* a, void* stream);

/* Bytes of workspace with which a call of these sizes splits K over workgroups
 * (few rows or few columns; 0 where it would not). */
size_t moe_grouped_gemm_workspace(int32_t R, int32_t E, int32_t N, int32_t K);
size_t moe_grouped_swiglu_workspace(int32_t R, int32_t E, int32_t N, int32_t K);

#ifdef __cplusplus
}
#endif

#endif /* MOE_ROWS_H */

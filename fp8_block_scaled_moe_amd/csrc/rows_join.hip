// moe_join_rmsnorm_quant (include/moe_block.h): a block's output normalised, gated
// and added to the scaled residual, the sum normalised for the next block, BF16 and
// 8-bit outputs with scales, in one pass.
//
// As rows_norm.hip: one workgroup per token holds the whole row in registers, eight
// columns a lane and chunk, so every input is read once and every output written once.
// The second norm's statistics need the first's, so a row crosses the workgroup
// twice. Both sums of squares are taken in FP64. Both norms round as
// moe_add_rmsnorm_quant's does (two FP32 products of each value). The residual's row is
// rounded once: a scale that is a multiple of 2^-15 up to 1 gives FP32 products with a
// BF16 residual (16 by 8 bits, none below FP32's smallest value), to which the gated
// value is added by one fused instruction; other scales take both products and their sum
// through FP64. Bound by HBM: 8,191 x 3584 with a full gate and MXFP8 67 us in a graph, 4.8
// TB/s, by the first way and 70 by the second; 4,096 tokens of eight rows of 7168 154 us,
// 4.6; a large copy runs at 5.2.
#include <hip/hip_runtime.h>

#include <cmath>

#include "../../include/moe_block.h"
#include "rows_device.h"

namespace moe {
namespace {

constexpr int kBatch = 8;  // expert rows requested before they are added
constexpr int kFewTokens = 512;  // see the launch

// 1 / sqrt(mean + eps) of a sum of squares over the workgroup. Barrier inside.
__device__ __forceinline__ double row_rstd(double sq, double* part, int D, float eps) {
  sq = wave_sum_f64(sq);
  if ((threadIdx.x & (kWave - 1)) == 0) part[threadIdx.x / kWave] = sq;
  __syncthreads();
  double total = 0.0;
  for (int w = 0; w < (int)blockDim.x / kWave; ++w) total += part[w];
  return 1.0 / sqrt(total / (double)D + (double)eps);
}

template <int kChunks, bool kRouted>
__global__ __launch_bounds__(kChunks == 4 ? 512 : 1024) void join_kernel(moe_join_args ja) {
  __shared__ double part[2][16];
  const moe_norm_args& a = ja.norm;
  const int t = blockIdx.x, tid = threadIdx.x;
  const size_t row = (size_t)t * a.D;
  const u32x4_t zero = {0u, 0u, 0u, 0u};
  float h[kChunks][kVec];
  u32x4_t r[kChunks], d[kChunks], g[kChunks], p[kChunks], u[kChunks];
#pragma unroll
  for (int c = 0; c < kChunks; ++c) {  // lanes past the row read its start and drop it
    const int col = (c * (int)blockDim.x + tid) * kVec;
    const int at = col < a.D ? col : 0;
    d[c] = a.delta ? load16(a.delta, row + at) : zero;
    p[c] = ja.post_gamma ? load16(ja.post_gamma, at) : zero;
    r[c] = a.residual ? load16(a.residual, row + at) : zero;
    u[c] = ja.gate_kind >= MOE_GATE_COLUMN ? load16(ja.gate, ja.gate_kind == MOE_GATE_FULL ? row + at : (size_t)at) : zero;
    g[c] = a.gamma ? load16(a.gamma, at) : zero;
  }
  float gate = 1.f;  // of the token
  if (ja.gate_kind == MOE_GATE_ROW)
    gate = ja.gate_dtype == MOE_DTYPE_BF16 ? bf16_value(static_cast<const uint16_t*>(ja.gate)[t]) : static_cast<const float*>(ja.gate)[t];

  double sq = 0.0;
#pragma unroll
  for (int c = 0; c < kChunks; ++c) {
    const int col = (c * (int)blockDim.x + tid) * kVec;
    const bool live = col < a.D;
    unpack8(d[c], h[c]);
    if (kRouted) {
      const int at = live ? col : 0;
      double acc[kVec];
#pragma unroll
      for (int i = 0; i < kVec; ++i) acc[i] = (double)h[c][i];
      for (int j0 = 0; j0 < a.k; j0 += kBatch) {
        u32x4_t y[kBatch];
        double w[kBatch];
#pragma unroll
        for (int j = 0; j < kBatch; ++j) {
          w[j] = 0.0;
          y[j] = zero;
          if (j0 + j < a.k) {  // uniform: the token's own positions and weights
            const int q = a.pos[(size_t)t * a.k + j0 + j];
            if (q >= 0 && q < a.R) {
              w[j] = (double)a.weights[(size_t)t * a.k + j0 + j];
              y[j] = load16(a.y, (size_t)q * a.D + at);
            }
          }
        }
#pragma unroll
        for (int j = 0; j < kBatch; ++j) {
          float yv[kVec];
          unpack8(y[j], yv);
#pragma unroll
          for (int i = 0; i < kVec; ++i) acc[i] = fma(w[j], (double)yv[i], acc[i]);
        }
      }
#pragma unroll
      for (int i = 0; i < kVec; ++i) h[c][i] = (float)acc[i];
    }
#pragma unroll
    for (int i = 0; i < kVec; ++i) {
      h[c][i] = live ? h[c][i] : 0.f;
      sq = fma((double)h[c][i], (double)h[c][i], sq);
    }
  }
  const float rstd_post = ja.post_gamma ? (float)row_rstd(sq, part[0], a.D, ja.post_eps) : 1.f;
  const bool exact = fabsf(ja.residual_scale) <= 1.f && rintf(ja.residual_scale * 0x1p15f) == ja.residual_scale * 0x1p15f;
  sq = 0.0;
#pragma unroll
  for (int c = 0; c < kChunks; ++c) {
    const int col = (c * (int)blockDim.x + tid) * kVec;
    const bool live = col < a.D;
    float rv[kVec], uv[kVec], pv[kVec];
    unpack8(r[c], rv);
    unpack8(u[c], uv);
    unpack8(p[c], pv);
#pragma unroll
    for (int i = 0; i < kVec; ++i) {
      if (ja.gate_kind < MOE_GATE_COLUMN) uv[i] = gate;
      if (ja.post_gamma) h[c][i] = (h[c][i] * rstd_post) * (pv[i] + ja.gamma_offset);
    }
    if (exact)
#pragma unroll
      for (int i = 0; i < kVec; ++i) h[c][i] = fmaf(h[c][i], uv[i], rv[i] * ja.residual_scale);
    else
#pragma unroll
      for (int i = 0; i < kVec; ++i) h[c][i] = (float)fma((double)h[c][i], (double)uv[i], (double)rv[i] * (double)ja.residual_scale);
#pragma unroll
    for (int i = 0; i < kVec; ++i) {
      h[c][i] = live ? h[c][i] : 0.f;
      sq = fma((double)h[c][i], (double)h[c][i], sq);
    }
    if (a.residual_out && live) *reinterpret_cast<u32x4_t*>(static_cast<uint16_t*>(a.residual_out) + row + col) = pack8(h[c]);
  }
  if (a.gamma) {
    const float rstd = (float)row_rstd(sq, part[1], a.D, a.eps);
#pragma unroll
    for (int c = 0; c < kChunks; ++c) {
      float gv[kVec];
      unpack8(g[c], gv);
#pragma unroll
      for (int i = 0; i < kVec; ++i) h[c][i] = (h[c][i] * rstd) * (gv[i] + ja.gamma_offset);
    }
  }
#pragma unroll
  for (int c = 0; c < kChunks; ++c) {
    const int col = (c * (int)blockDim.x + tid) * kVec;
    const bool live = col < a.D;
    if (a.out && live) *reinterpret_cast<u32x4_t*>(static_cast<uint16_t*>(a.out) + row + col) = pack8(h[c]);
    if (a.quant != MOE_QUANT_NONE) store_quant(a, h[c], t, col, live);
  }
}

template <int kChunks, bool kRouted>
void launch_join(const moe_join_args& a, int threads, hipStream_t stream) {
  hipLaunchKernelGGL((join_kernel<kChunks, kRouted>), dim3(a.norm.T), dim3(threads), 0, stream, a);
}

}  // namespace
}  // namespace moe

extern "C" int moe_join_rmsnorm_quant(const moe_join_args* args, void* stream) {
  using namespace moe;
  if (!args) return MOE_DECODE_ERR_INVALID_ARG;
  const moe_join_args& a = *args;
  const int rc = check_norm(a.norm);
  if (rc != MOE_DECODE_OK || a.norm.T == 0) return rc;
  if (!a.norm.delta && !a.norm.k) return MOE_DECODE_ERR_INVALID_ARG;
  if (!(a.post_eps >= 0.f) || !std::isfinite(a.post_eps) || !std::isfinite(a.residual_scale) || !std::isfinite(a.gamma_offset))
    return MOE_DECODE_ERR_INVALID_ARG;
  if (a.gate_kind < MOE_GATE_NONE || a.gate_kind > MOE_GATE_FULL ||
      (a.gate_dtype != MOE_DTYPE_BF16 && !(a.gate_dtype == MOE_DTYPE_F32 && a.gate_kind <= MOE_GATE_ROW)))
    return MOE_DECODE_ERR_UNSUPPORTED;
  const uintptr_t unit = a.gate_kind != MOE_GATE_ROW ? 16 : a.gate_dtype == MOE_DTYPE_F32 ? 4 : 2;
  if ((a.gate != nullptr) != (a.gate_kind != MOE_GATE_NONE) || misaligned(a.gate, unit) || misaligned(a.post_gamma, 16))
    return MOE_DECODE_ERR_INVALID_ARG;
  const int lanes = a.norm.D / kVec;
  hipStream_t s = static_cast<hipStream_t>(stream);
  const auto waves = [](int n) { return (n + kWave - 1) / kWave * kWave; };
  // Chunks a lane. Few plain tokens: one, with all of a row's loads on their way at once.
  // Routed rows of more than 2048 columns: two, so that a CU holds two workgroups, of which
  // one loads while the other is between its barriers (eight rows of 7168 for 4,096 tokens:
  // 173 us with one chunk, 153 with two, 4% more with four; for 512 tokens 25.7 and 21.4 with one
  // and two; beyond 8192 columns there is one workgroup, and two chunks are faster than four
  // all the same: 4,096 x 12288 260 and 306, x 16384 349 and 352). A few tokens alone would
  // take less with one chunk, whose rows come at once: 1 x 7168 8.9 and 9.3, 1 x 4096 6.2
  // and 7.5, 128 x 7168 11.1 and 11.4. Many plain rows: two up to 4096 columns, four beyond (8,191 x 3584: 73, 68 and 71 us; 4,096 x 8192:
  // 73, 66 and 64).
  const bool few = a.norm.T <= kFewTokens;
  if (a.norm.k > 0 && lanes <= 256)
    launch_join<1, true>(a, waves(lanes), s);
  else if (a.norm.k > 0)
    launch_join<2, true>(a, waves((lanes + 1) / 2), s);
  else if (lanes <= (few ? 1024 : 256))
    launch_join<1, false>(a, waves(lanes), s);
  else if (few || lanes <= 512)
    launch_join<2, false>(a, waves((lanes + 1) / 2), s);
  else
    launch_join<4, false>(a, waves((lanes + 3) / 4), s);
  return hipGetLastError() == hipSuccess ? MOE_DECODE_OK : MOE_DECODE_ERR_HIP;
}

// moe_add_rmsnorm_quant (include/moe_rows.h): residual + addend + weighted
// expert rows, RMSNorm, BF16 and 8-bit outputs with scales, in one pass.
//
// One workgroup per token holds the whole row in registers, eight columns a
// lane and chunk, so every input is read once and every output written once:
// the bound is HBM (8,191 rows of 3584 with an addend, MXFP8: 54 us, 4.9 TB/s;
// 4,096 rows of 7168 with eight routed rows each: 142 us, 4.8 TB/s; a large copy
// runs at 4.9). The sum and the sum of squares are taken in FP64 (two
// more instructions per value, hidden behind memory): residual, addend, then the
// picks in their order, rounded to FP32. That is the correctly rounded sum but
// next to a rounding border and where terms of 2^29 times the result and more
// cancel; the same call gives the same bits every time. The sum of squares is
// joined over a workgroup's lanes, so the last bit of rstd may differ, next to a
// rounding border, between the workgroup sizes of the launch below.
#include <hip/hip_runtime.h>

#include "../../include/moe_rows.h"
#include "rows_device.h"

namespace moe {
namespace {

constexpr int kBatch = 8;  // expert rows requested before they are added
constexpr int kFewTokens = 512;  // see the launch

template <int kChunks, bool kRouted>
__global__ __launch_bounds__(1024) void norm_kernel(moe_norm_args a) {
  __shared__ double part[16];
  const int t = blockIdx.x, tid = threadIdx.x, lane = tid & (kWave - 1);
  const size_t row = (size_t)t * a.D;
  float h[kChunks][kVec];
  u32x4_t r[kChunks], d[kChunks], g[kChunks];
  const u32x4_t zero = {0u, 0u, 0u, 0u};
#pragma unroll
  for (int c = 0; c < kChunks; ++c) {  // lanes past the row read its start and drop it
    const int col = (c * (int)blockDim.x + tid) * kVec;
    const int at = col < a.D ? col : 0;
    r[c] = a.residual ? load16(a.residual, row + at) : zero;
    d[c] = a.delta ? load16(a.delta, row + at) : zero;
    g[c] = a.gamma ? load16(a.gamma, at) : zero;
  }
  double sq = 0.0;
#pragma unroll
  for (int c = 0; c < kChunks; ++c) {
    const int col = (c * (int)blockDim.x + tid) * kVec;
    const bool live = col < a.D;
    float rv[kVec], dv[kVec];
    unpack8(r[c], rv);
    unpack8(d[c], dv);
    if (kRouted) {
      const int at = live ? col : 0;
      double acc[kVec];
#pragma unroll
      for (int i = 0; i < kVec; ++i) acc[i] = (double)rv[i] + (double)dv[i];
      for (int j0 = 0; j0 < a.k; j0 += kBatch) {
        u32x4_t y[kBatch];
        double w[kBatch];
#pragma unroll
        for (int j = 0; j < kBatch; ++j) {
          w[j] = 0.0;
          y[j] = zero;
          if (j0 + j < a.k) {  // uniform: the token's own positions and weights
            const int p = a.pos[(size_t)t * a.k + j0 + j];
            if (p >= 0 && p < a.R) {
              w[j] = (double)a.weights[(size_t)t * a.k + j0 + j];
              y[j] = load16(a.y, (size_t)p * a.D + at);
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
    } else {
#pragma unroll
      for (int i = 0; i < kVec; ++i) h[c][i] = rv[i] + dv[i];  // one rounding of an exact sum
    }
#pragma unroll
    for (int i = 0; i < kVec; ++i) {
      h[c][i] = live ? h[c][i] : 0.f;
      sq = fma((double)h[c][i], (double)h[c][i], sq);
    }
    if (a.residual_out && live)
      *reinterpret_cast<u32x4_t*>(static_cast<uint16_t*>(a.residual_out) + row + col) = pack8(h[c]);
  }
  if (a.gamma) {
    sq = wave_sum_f64(sq);
    if (lane == 0) part[tid / kWave] = sq;
    __syncthreads();
    double total = 0.0;
    for (int w = 0; w < (int)blockDim.x / kWave; ++w) total += part[w];
    const float rstd = (float)(1.0 / sqrt(total / (double)a.D + (double)a.eps));
#pragma unroll
    for (int c = 0; c < kChunks; ++c) {
      float gv[kVec];
      unpack8(g[c], gv);
#pragma unroll
      for (int i = 0; i < kVec; ++i) h[c][i] = (h[c][i] * rstd) * gv[i];
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

template <int kChunks>
void launch_norm(const moe_norm_args& a, int threads, hipStream_t stream) {
  if (a.k)
    hipLaunchKernelGGL((norm_kernel<kChunks, true>), dim3(a.T), dim3(threads), 0, stream, a);
  else
    hipLaunchKernelGGL((norm_kernel<kChunks, false>), dim3(a.T), dim3(threads), 0, stream, a);
}

}  // namespace
}  // namespace moe

extern "C" int moe_add_rmsnorm_quant(const moe_norm_args* args, void* stream) {
  using namespace moe;
  if (!args) return MOE_DECODE_ERR_INVALID_ARG;
  const moe_norm_args& a = *args;
  const int rc = check_norm(a);
  if (rc != MOE_DECODE_OK || a.T == 0) return rc;
  // Lanes for one chunk each: many, with all of a row's loads on their way at
  // once, for routed rows (whose positions come first: 4,096 tokens of eight
  // rows of 7168, 150 us against 171) and for few tokens (7168 columns: one
  // token 3.8 us against 4.6, 512 tokens 10.0 against 10.4); a quarter of
  // them, with more workgroups on a CU, for many plain rows (1,024 tokens
  // 14.9 against 16.5, 8,192 tokens 101 against 108).
  const int lanes = a.D / kVec;
  hipStream_t s = static_cast<hipStream_t>(stream);
  const auto waves = [](int n) { return (n + kWave - 1) / kWave * kWave; };
  const bool wide = a.k > 0 || a.T <= kFewTokens;
  if (lanes <= (wide ? 1024 : 256))
    launch_norm<1>(a, waves(lanes), s);
  else if (wide || lanes <= 512)
    launch_norm<2>(a, waves((lanes + 1) / 2), s);
  else
    launch_norm<4>(a, waves((lanes + 3) / 4), s);
  return hipGetLastError() == hipSuccess ? MOE_DECODE_OK : MOE_DECODE_ERR_HIP;
}

// The dense product for few rows: up to 16 kJ rows by 16 weight rows per workgroup,
// operands straight from memory into registers.
#include <hip/hip_runtime.h>

#include "dense_device.h"

namespace moe {
namespace {

constexpr int kWaves = 8;
constexpr int kBatch = 4;  // 32-wide steps requested at once

__device__ __forceinline__ bf16x8_t load8(const uint16_t* p) {
  return __builtin_bit_cast(bf16x8_t, *reinterpret_cast<const u32x4_t*>(p));
}

// The 64-wide blocks of K (128-byte lines of a row) go round the waves; a lane has
// row l % 16 and eight columns from 8 (l / 16) on of each 32-wide step.
template <int kJ>
__global__ __launch_bounds__(kWaves* kWave) void strip_kernel(DenseArgs a) {
  __shared__ float sums[kWaves][kJ][16][17];
  const int tid = threadIdx.x, lane = tid & (kWave - 1), wave = tid / kWave;
  const int r = lane & 15, k8 = (lane >> 4) * 8;
  const int n0 = blockIdx.x * 16, t0 = blockIdx.y * 16 * kJ;
  const uint16_t* wp = a.w + (size_t)min(n0 + r, a.N - 1) * a.ldw + k8;
  const uint16_t* xp[kJ];
#pragma unroll
  for (int j = 0; j < kJ; ++j) xp[j] = a.x + (size_t)min(t0 + 16 * j + r, a.T - 1) * a.ldx + k8;
  const bf16x8_t none = {};
  float4_t acc[kJ];
#pragma unroll
  for (int j = 0; j < kJ; ++j) acc[j] = float4_t{0.f, 0.f, 0.f, 0.f};
  for (int k0 = wave * 64; k0 < a.K; k0 += kWaves * 64 * (kBatch / 2)) {
    bf16x8_t w[kBatch], x[kBatch][kJ];
#pragma unroll
    for (int s = 0; s < kBatch; ++s) {
      const int k = k0 + (s >> 1) * kWaves * 64 + (s & 1) * 32;
      const bool in = k + k8 < a.K;
      w[s] = in ? load8(wp + k) : none;
#pragma unroll
      for (int j = 0; j < kJ; ++j) x[s][j] = in ? load8(xp[j] + k) : none;
    }
#pragma unroll
    for (int s = 0; s < kBatch; ++s)
#pragma unroll
      for (int j = 0; j < kJ; ++j) acc[j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(w[s], x[s][j], acc[j], 0, 0, 0);
  }
  // a lane's sums: row r of x, weight rows 4 (l / 16) + i
#pragma unroll
  for (int j = 0; j < kJ; ++j)
#pragma unroll
    for (int i = 0; i < 4; ++i) sums[wave][j][r][(lane >> 4) * 4 + i] = acc[j][i];
  __syncthreads();
  for (int q = tid; q < kJ * 256; q += kWaves * kWave) {
    const int j = q >> 8, t = t0 + 16 * j + ((q >> 4) & 15), n = n0 + (q & 15);
    float v = 0.f;
#pragma unroll
    for (int i = 0; i < kWaves; ++i) v += sums[i][j][(q >> 4) & 15][q & 15];
    if (t < a.T && n < a.N) finish(a, t, n, v);
  }
}

template <int kJ>
void launch(const DenseArgs& a, hipStream_t stream) {
  hipLaunchKernelGGL(strip_kernel<kJ>, dim3((a.N + 15) / 16, (a.T + 16 * kJ - 1) / (16 * kJ)), dim3(kWaves * kWave), 0, stream, a);
}

}  // namespace

void launch_dense_strip(const DenseArgs& a, hipStream_t stream) {
  if (a.T <= 16)
    launch<1>(a, stream);
  else if (a.T <= 32)
    launch<2>(a, stream);
  else
    launch<4>(a, stream);
}

}  // namespace moe

// Device pieces of the dense product (moe_dense_gemm in moe_block.h): operands,
// activations and the epilogue.
#pragma once

#include <type_traits>

#include "../../include/moe_block.h"
#include "dense_plan.h"
#include "grouped_device.h"
#include "rows_device.h"

namespace moe {

// Rows at most this far apart, so that the 256 rows of a tile lie within 2^32 bytes.
constexpr int64_t kDenseMaxStride = (1 << 23) - 1;

struct DenseArgs {
  const uint16_t* x;
  const uint16_t* w;
  const void* bias;      // or nullptr
  const void* residual;  // or nullptr
  void* out;
  int64_t ldx, ldw, ldr;
  int T, N, K;
  int act;
  bool out_f32, bias_f32, residual_f32;
  bool vector_io;  // eight neighbouring columns of out and of residual lie on 16-byte boundaries
  int splits;      // parts of K, one per workgroup
  float* partial;  // [splits][T][dense_pitch(N)] FP32 sums over a part of K each, where splits > 1
};

// Columns of a row of partial sums: whole groups of eight.
__host__ __device__ inline size_t dense_pitch(int N) { return ((size_t)N + 7) / 8 * 8; }

// 1 / (1 + exp(-v)) times u, from t = -v log2 e by the hardware's exp2 and reciprocal.
// What the rounding of t leaves of -v is made up for to first order, with ln 2 in two
// parts, so that the error does not grow with |v|: one step of 2^-23 each for the
// exponential and the reciprocal, half of one for three roundings; below -87 the first
// factor, under 2^-125, counts as 0. A NaN stays one. Without the correction (|v| 2^-23 of
// the value) 8,192 x 4,096 takes 109 us and not 114 for K = 2048 with SiLU, 359 and
// 363 for K = 7168 with the tanh form.
__device__ __forceinline__ float times_sigmoid(float v, float u) {
  constexpr float kLog2e = 0x1.715476p+0f, kLn2 = 0x1.62e43p-1f, kLn2Low = -0x1.05c61p-29f;  // ln 2 in two parts
  const bool none = v < -87.f;
  v = clamp_nan(v, -87.f, 87.f);  // neither t nor the exponential is infinite
  const float t = v * -kLog2e, e = __builtin_amdgcn_exp2f(t);
  return u * (none ? 0.f : __builtin_amdgcn_rcpf(fmaf(e, fmaf(t, -kLn2Low, fmaf(t, -kLn2, -v)), 1.f + e)));
}

template <int kAct>
__device__ __forceinline__ float activation(float v) {
  switch (kAct) {
    case MOE_ACT_RELU:
      return __builtin_elementwise_maximum(v, 0.f);
    case MOE_ACT_SILU:
      return times_sigmoid(v, v);
    case MOE_ACT_GELU:
      return 0.5f * v * (1.f + erff(v * 0.70710678118654752f));
    case MOE_ACT_GELU_TANH:  // (1 + tanh u) / 2 = 1 / (1 + exp(-2 u))
      return times_sigmoid(v * fmaf(v * v, 0.0713548162726009f, 1.5957691216057308f), v);
    case MOE_ACT_SIGMOID:
      return times_sigmoid(v, 1.f);
    default:
      return v;
  }
}

// One activation for all of v: the choice stands outside of the values.
template <int kN>
__device__ __forceinline__ void activate(const DenseArgs& a, float (&v)[kN]) {
  const auto all = [&](auto act) {
#pragma unroll
    for (int i = 0; i < kN; ++i) v[i] = activation<decltype(act)::value>(v[i]);
  };
  switch (a.act) {
    case MOE_ACT_RELU:
      return all(std::integral_constant<int, MOE_ACT_RELU>{});
    case MOE_ACT_SILU:
      return all(std::integral_constant<int, MOE_ACT_SILU>{});
    case MOE_ACT_GELU:
      return all(std::integral_constant<int, MOE_ACT_GELU>{});
    case MOE_ACT_GELU_TANH:
      return all(std::integral_constant<int, MOE_ACT_GELU_TANH>{});
    case MOE_ACT_SIGMOID:
      return all(std::integral_constant<int, MOE_ACT_SIGMOID>{});
  }
}

__device__ __forceinline__ float element(const void* p, size_t i, bool f32) {
  return f32 ? static_cast<const float*>(p)[i] : bf16_value(static_cast<const uint16_t*>(p)[i]);
}

// Bias, activation and residual of one value, and its store.
__device__ __forceinline__ void finish(const DenseArgs& a, int t, int n, float v) {
  if (a.bias) v += element(a.bias, n, a.bias_f32);
  float one[1] = {v};
  activate(a, one);
  v = one[0];
  if (a.residual) v += element(a.residual, (size_t)t * a.ldr + n, a.residual_f32);
  const size_t o = (size_t)t * a.N + n;
  if (a.out_f32)
    static_cast<float*>(a.out)[o] = v;
  else
    static_cast<uint16_t*>(a.out)[o] = (uint16_t)bf16x2_bits(v, 0.f);
}

// Eight neighbouring columns from n on: their bias, and how kRows rows' sums of them end.
template <int kRows>
struct Columns {
  int n, count;  // columns below N
  float bias[8];
  __device__ __forceinline__ Columns(const DenseArgs& a, int first) : n(first), count(min(8, a.N - first)) {
#pragma unroll
    for (int i = 0; i < 8; ++i) bias[i] = a.bias && i < count ? element(a.bias, n + i, a.bias_f32) : 0.f;
  }
  // Rows t, t + step, .. of those below T: v, eight values each, where eight columns of
  // `out` and of the residual lie on 16-byte boundaries. The residual's loads come first.
  __device__ __forceinline__ void finish(const DenseArgs& a, int t, int step, float (&v)[8 * kRows]) const {
    u32x4_t lo[kRows], hi[kRows];
    if (a.residual) {
#pragma unroll
      for (int r = 0; r < kRows; ++r) {
        const size_t at = (size_t)min(t + r * step, a.T - 1) * a.ldr + n;
        if (a.residual_f32) {
          const u32x4_t* p = reinterpret_cast<const u32x4_t*>(static_cast<const float*>(a.residual) + at);
          lo[r] = p[0];
          hi[r] = p[1];
        } else {
          lo[r] = load16(a.residual, at);
        }
      }
    }
    if (a.bias)
#pragma unroll
      for (int r = 0; r < kRows; ++r)
#pragma unroll
        for (int i = 0; i < 8; ++i) v[8 * r + i] += bias[i];
    activate(a, v);
    if (a.residual) {
#pragma unroll
      for (int r = 0; r < kRows; ++r) {
        float res[8];
        if (a.residual_f32) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            res[i] = __uint_as_float(lo[r][i]);
            res[4 + i] = __uint_as_float(hi[r][i]);
          }
        } else {
          unpack8(lo[r], res);
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) v[8 * r + i] += res[i];
      }
    }
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
      if (t + r * step >= a.T) continue;
      const size_t o = (size_t)(t + r * step) * a.N + n;
      const float(&w)[8] = *reinterpret_cast<const float(*)[8]>(&v[8 * r]);
      if (a.out_f32) {
        float4_t* p = reinterpret_cast<float4_t*>(static_cast<float*>(a.out) + o);
        p[0] = float4_t{w[0], w[1], w[2], w[3]};
        p[1] = float4_t{w[4], w[5], w[6], w[7]};
      } else {
        *reinterpret_cast<u32x4_t*>(static_cast<uint16_t*>(a.out) + o) = pack8(w);
      }
    }
  }
};

// What columns from K on are copied from.
alignas(16) static __device__ const uint32_t kNothing[4] = {};

void launch_dense_strip(const DenseArgs& a, int shape, hipStream_t stream);  // dense_strip.hip
void launch_dense_tile(const DenseArgs& a, int shape, hipStream_t stream);   // dense_tile.hip

}  // namespace moe

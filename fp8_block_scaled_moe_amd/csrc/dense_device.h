// Device pieces of the dense product (moe_dense_gemm in moe_block.h): operands,
// activations and the epilogue.
#pragma once

#include "../../include/moe_block.h"
#include "grouped_device.h"

namespace moe {

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
  float* partial;  // [splits][T][N] FP32 sums over a part of K each, where splits > 1
};

// 1 / (1 + exp(-v)) times u. The exponential by the hardware's exp2 of t =
// -v log2 e, with what the rounding of t leaves of -v made up for to first order, so
// that its error hardly grows with |v|. Below -87 v counts as -87 (the value is 2^-125
// then); a NaN stays one.
__device__ __forceinline__ float times_sigmoid(float v, float u) {
  constexpr float kLog2e = 0x1.715476p+0f, kLn2 = 0x1.62e43p-1f;
  v = clamp_nan(v, -87.f, 3.0e38f);
  const float t = v * -kLog2e, e = __builtin_amdgcn_exp2f(t);
  return u * __builtin_amdgcn_rcpf(fmaf(e, fmaf(t, -kLn2, -v), 1.f + e));
}

__device__ __forceinline__ float activation(float v, int act) {
  switch (act) {
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

__device__ __forceinline__ float element(const void* p, size_t i, bool f32) {
  return f32 ? static_cast<const float*>(p)[i] : bf16_value(static_cast<const uint16_t*>(p)[i]);
}

// Bias, activation and residual of one value, and its store.
__device__ __forceinline__ void finish(const DenseArgs& a, int t, int n, float v) {
  if (a.bias) v += element(a.bias, n, a.bias_f32);
  v = activation(v, a.act);
  if (a.residual) v += element(a.residual, (size_t)t * a.ldr + n, a.residual_f32);
  const size_t o = (size_t)t * a.N + n;
  if (a.out_f32)
    static_cast<float*>(a.out)[o] = v;
  else
    static_cast<uint16_t*>(a.out)[o] = (uint16_t)bf16x2_bits(v, 0.f);
}

void launch_dense_strip(const DenseArgs& a, hipStream_t stream);  // dense_strip.hip

}  // namespace moe

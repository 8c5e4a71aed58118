// Device pieces of the dense product (moe_dense_gemm in moe_block.h): operands,
// activations and the epilogue.
#pragma once

#include "../../include/moe_block.h"
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

// Eight neighbouring columns from n on: their bias, and how a row's sums of them end.
struct Columns {
  int n, count;  // columns below N
  float bias[8];
  __device__ __forceinline__ Columns(const DenseArgs& a, int first) : n(first), count(min(8, a.N - first)) {
#pragma unroll
    for (int i = 0; i < 8; ++i) bias[i] = a.bias && i < count ? element(a.bias, n + i, a.bias_f32) : 0.f;
  }
  // Row t's sums (of part `split` of K where there are several).
  __device__ __forceinline__ void finish(const DenseArgs& a, int t, int split, const float4_t& lo, const float4_t& hi) const {
    if (a.splits > 1) {
      float4_t* o = reinterpret_cast<float4_t*>(a.partial + ((size_t)split * a.T + t) * dense_pitch(a.N) + n);
      o[0] = lo;
      o[1] = hi;
      return;
    }
    float v[8] = {lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
    end(a, t, v);
  }
  __device__ __forceinline__ void end(const DenseArgs& a, int t, float (&v)[8]) const {
    const size_t r = (size_t)t * a.ldr + n;
    float res[8] = {};
    const bool whole = a.vector_io;  // N is a multiple of eight then
    if (a.residual) {
      if (!whole) {
#pragma unroll
        for (int i = 0; i < 8; ++i) res[i] = i < count ? element(a.residual, r + i, a.residual_f32) : 0.f;
      } else if (a.residual_f32) {
        const float4_t* p = reinterpret_cast<const float4_t*>(static_cast<const float*>(a.residual) + r);
        const float4_t lo = p[0], hi = p[1];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          res[i] = lo[i];
          res[4 + i] = hi[i];
        }
      } else {
        unpack8(load16(a.residual, r), res);
      }
    }
    if (a.bias)
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] += bias[i];
    if (a.act != MOE_ACT_NONE)
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = activation(v[i], a.act);
    if (a.residual)
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] += res[i];
    const size_t o = (size_t)t * a.N + n;
    if (whole) {
      if (a.out_f32) {
        float4_t* p = reinterpret_cast<float4_t*>(static_cast<float*>(a.out) + o);
        p[0] = float4_t{v[0], v[1], v[2], v[3]};
        p[1] = float4_t{v[4], v[5], v[6], v[7]};
      } else {
        *reinterpret_cast<u32x4_t*>(static_cast<uint16_t*>(a.out) + o) = pack8(v);
      }
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (i < count) {
          if (a.out_f32)
            static_cast<float*>(a.out)[o + i] = v[i];
          else
            static_cast<uint16_t*>(a.out)[o + i] = (uint16_t)bf16x2_bits(v[i], 0.f);
        }
    }
  }
};

// What columns from K on are copied from.
alignas(16) static __device__ const uint32_t kNothing[4] = {};

// Rows of x by weight rows of a workgroup, and how many workgroups a CU holds.
enum DenseShape {
  kDenseStrip4x4,
  kDenseStrip8x8,
  kDenseStrip16x16,
  kDenseStrip16x32,
  kDenseStrip32x32,
  kDenseStrip32x64,
  kDense64x128,
  kDense128x128,
  kDense128x128Two,  // two workgroups a CU
  kDense256x256,
  kDenseHalves,  // 256 x 256, the tiles past whole rounds of the CUs as 128 x 256
};

void launch_dense_strip(const DenseArgs& a, int shape, hipStream_t stream);// dense_strip.hip
void launch_dense_tile(const DenseArgs& a, int shape, hipStream_t stream);  // dense_tile.hip

}  // namespace moe

// Products grouped by expert over ragged rows (include/moe_rows.h): the calls
// moe_grouped_gemm and moe_grouped_swiglu, over the kernels of
// grouped_product.hip, grouped_product_fp8.hip and grouped_swiglu.hip, and the
// joining of split sums.
//
// A tile's K blocks come one after the other: 0.7 us and more each, whatever the
// number of tiles, since a CU takes in some 60 GB/s by these copies (a fourth block
// in LDS changes nothing). Where the tiles leave CUs idle, K is split over
// workgroups, whose FP32 sums go to the workspace and are added here in
// order (no atomics), before the rounding or the SwiGLU. Without and with it,
// calls in a graph, one token's 6 of 64 experts with 512 columns: product, K = 2048
// 15.9 and 10.1 us, 7168 44.7 and 12.4; SwiGLU 17.4 and 12.0, 46.6 and 18.0; 300
// tokens x 2 of 8: product 27.5 and 18.3, 85.4 and 26.0; SwiGLU 29.3 and 23.3, 88.7
// and 37.5; 1,000 tokens x 2 of 8: 31.7 and 23.8, 98.0 and 38.1, 33.1 and 31.9, 106
// and 70. K = 1024 takes 9.6 and 11.3 us unsplit and gains nothing in a graph; from
// Python, where the host needs 4 us for the second launch, it loses them. Parts of at
// least 2 to 8 blocks were alike.
#include <hip/hip_runtime.h>

#include "../../include/moe_rows.h"
#include "grouped_device.h"

namespace moe {
namespace {

constexpr int kJoinThreads = 256;

// Is row i one that an expert has?
__device__ __forceinline__ bool has_expert(const GroupedArgs& a, int i) {
  const uniform_ints o = as_uniform(a.offsets);
  return i >= o[0] && i < o[a.E];
}

// Eight neighbouring sums of row i from column n on, over all parts of K.
__device__ __forceinline__ void join8(const GroupedArgs& a, int i, int n, float (&v)[8]) {
  const float* p = a.partial + (size_t)i * a.N + n;
#pragma unroll
  for (int q = 0; q < 8; ++q) v[q] = 0.f;
#pragma unroll 4
  for (int s = 0; s < a.splits; ++s) {
    const float4_t lo = *reinterpret_cast<const float4_t*>(p), hi = *reinterpret_cast<const float4_t*>(p + 4);
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      v[q] += lo[q];
      v[4 + q] += hi[q];
    }
    p += (size_t)a.R * a.N;
  }
}

__global__ __launch_bounds__(kJoinThreads) void join_product_kernel(GroupedArgs a) {
  const int64_t at = ((int64_t)blockIdx.x * kJoinThreads + threadIdx.x) * 8;
  const int i = (int)(at / a.N), n = (int)(at % a.N);
  if (i >= a.R || !has_expert(a, i)) return;
  float v[8];
  join8(a, i, n, v);
  u32x4_t q = {bf16x2_bits(v[0], v[1]), bf16x2_bits(v[2], v[3]), bf16x2_bits(v[4], v[5]), bf16x2_bits(v[6], v[7])};
  if (x_row(a, i) < 0) q = u32x4_t{0u, 0u, 0u, 0u};
  *reinterpret_cast<u32x4_t*>(static_cast<uint16_t*>(a.out) + at) = q;
}

// Sixteen lanes have a block of 128 hidden values of a row.
__global__ __launch_bounds__(kJoinThreads) void join_swiglu_kernel(GroupedArgs a) {
  const int I = a.N / 2;
  const int64_t at = ((int64_t)blockIdx.x * kJoinThreads + threadIdx.x) * 8;
  const int i = (int)(at / I), n = (int)(at % I);
  if (i >= a.R || !has_expert(a, i)) return;
  float up[8], gate[8];
  join8(a, i, n, up);
  join8(a, i, I + n, gate);
  const bool none = x_row(a, i) < 0;
  float amax = kAmaxFloor;
#pragma unroll
  for (int q = 0; q < 8; ++q) {
    up[q] = none ? 0.f : swiglu(up[q], gate[q], a.limit);
    amax = fmaxf(amax, fabsf(up[q]));
  }
  amax = dpp_max16(amax);
  const float scale = amax / kFp8Max, inv = 1.0f / scale;
  u32x2_t codes;
#pragma unroll
  for (int q = 0; q < 2; ++q)
    codes[q] = e4m3x4_encode_nan(up[4 * q] * inv, up[4 * q + 1] * inv, up[4 * q + 2] * inv, up[4 * q + 3] * inv);
  *reinterpret_cast<u32x2_t*>(static_cast<uint8_t*>(a.out) + at) = codes;
  if ((threadIdx.x & 15) == 0) a.outs[(size_t)i * (I / 128) + n / 128] = scale;
}

void launch_join(void (*kernel)(GroupedArgs), const GroupedArgs& a, int64_t columns, hipStream_t stream) {
  const unsigned blocks = (unsigned)((a.R * columns / 8 + kJoinThreads - 1) / kJoinThreads);
  hipLaunchKernelGGL(kernel, dim3(blocks), dim3(kJoinThreads), 0, stream, a);
}

size_t workspace(int R, int E, int N, int K) {
  if (R <= 0 || E <= 0 || N <= 0 || K <= 0) return 0;
  const int splits = grouped_splits(R, E, N, K);
  return splits > 1 ? (size_t)splits * R * N * sizeof(float) : 0;
}

int check(const moe_grouped_args* p) {
  if (!p) return MOE_DECODE_ERR_INVALID_ARG;
  const moe_grouped_args& a = *p;
  if (a.R < 0 || a.X < 0 || a.E < 1 || a.N < 1 || a.K < 1) return MOE_DECODE_ERR_INVALID_ARG;
  if (a.E > MOE_DECODE_MAX_EXPERTS || a.N % 128 || a.K % 128 || a.N > MOE_ROWS_MAX_DIM || a.K > MOE_ROWS_MAX_DIM ||
      a.quant < MOE_QUANT_FP8 || a.quant > MOE_QUANT_MXFP8 || a.sums < MOE_SUMS_FP32 || a.sums > MOE_SUMS_FP8)
    return MOE_DECODE_ERR_UNSUPPORTED;
  if (a.R == 0) return MOE_DECODE_OK;
  if (a.X < (a.rows ? 1 : a.R)) return MOE_DECODE_ERR_INVALID_ARG;
  if (!a.x || !a.x_scale || !a.offsets || !a.w || !a.w_scale || !a.out) return MOE_DECODE_ERR_INVALID_ARG;
  if (misaligned(a.x, 16) || misaligned(a.w, 16) || misaligned(a.out, 16) || misaligned(a.w_scale, 4) ||
      misaligned(a.offsets, 4) || misaligned(a.rows, 4) || misaligned(a.x_scale, 4))
    return MOE_DECODE_ERR_INVALID_ARG;
  // a grid's limit, 2^32 threads of 512 a workgroup
  if (((int64_t)a.R / 128 + a.E) * ((a.N + 255) / 256) > (int64_t)(UINT32_MAX / 512) - 8) return MOE_DECODE_ERR_UNSUPPORTED;
  return MOE_DECODE_OK;
}

// With the workspace's errors: `need` bytes, or none at all (no parts of K then).
int check_workspace(const moe_grouped_args& a, size_t need) {
  if (!a.workspace || !need) return MOE_DECODE_OK;
  if (misaligned(a.workspace, 16)) return MOE_DECODE_ERR_INVALID_ARG;
  return a.workspace_bytes < need ? MOE_DECODE_ERR_SCRATCH_TOO_SMALL : MOE_DECODE_OK;
}

GroupedArgs kernel_args(const moe_grouped_args& a) {
  GroupedArgs g{};
  g.x = static_cast<const uint8_t*>(a.x);
  g.xs = a.x_scale;
  g.rows = a.rows;
  g.offsets = a.offsets;
  g.w = static_cast<const uint8_t*>(a.w);
  g.ws = a.w_scale;
  g.out = a.out;
  g.outs = a.out_scale;
  g.R = a.R;
  g.X = a.X;
  g.E = a.E;
  g.N = a.N;
  g.K = a.K;
  g.limit = fminf(a.limit, 0x1p127f);  // so that gate log2 e stays finite
  g.splits = a.workspace ? grouped_splits(a.R, a.E, a.N, a.K) : 1;
  g.partial = static_cast<float*>(a.workspace);
  return g;
}

}  // namespace
}  // namespace moe

extern "C" {

size_t moe_grouped_gemm_workspace(int32_t R, int32_t E, int32_t N, int32_t K) {
  return moe::workspace(R, E, N, K);
}

size_t moe_grouped_swiglu_workspace(int32_t R, int32_t E, int32_t N, int32_t K) {
  return moe::workspace(R, E, N, K);
}

int moe_grouped_gemm(const moe_grouped_args* args, void* stream) {
  using namespace moe;
  if (const int rc = check(args)) return rc;
  if (args->R == 0) return MOE_DECODE_OK;
  if (const int rc = check_workspace(*args, moe_grouped_gemm_workspace(args->R, args->E, args->N, args->K))) return rc;
  const GroupedArgs a = kernel_args(*args);
  hipStream_t s = static_cast<hipStream_t>(stream);
  const auto launch = args->sums == MOE_SUMS_FP8 ? launch_grouped_product_fp8 : launch_grouped_product;
  launch(args->quant == MOE_QUANT_MXFP8, a, s);
  if (a.splits > 1) launch_join(join_product_kernel, a, a.N, s);
  return hipGetLastError() == hipSuccess ? MOE_DECODE_OK : MOE_DECODE_ERR_HIP;
}

int moe_grouped_swiglu(const moe_grouped_args* args, void* stream) {
  using namespace moe;
  if (const int rc = check(args)) return rc;
  if (args->N % 256 || args->sums != MOE_SUMS_FP32) return MOE_DECODE_ERR_UNSUPPORTED;
  if (!(args->limit > 0.f)) return MOE_DECODE_ERR_INVALID_ARG;
  if (args->R == 0) return MOE_DECODE_OK;
  if (!args->out_scale || misaligned(args->out_scale, 4)) return MOE_DECODE_ERR_INVALID_ARG;
  if (const int rc = check_workspace(*args, moe_grouped_swiglu_workspace(args->R, args->E, args->N, args->K))) return rc;
  const GroupedArgs a = kernel_args(*args);
  hipStream_t s = static_cast<hipStream_t>(stream);
  launch_grouped_swiglu(args->quant == MOE_QUANT_MXFP8, a, s);
  if (a.splits > 1) launch_join(join_swiglu_kernel, a, a.N / 2, s);
  return hipGetLastError() == hipSuccess ? MOE_DECODE_OK : MOE_DECODE_ERR_HIP;
}

}  // extern "C"

// moe_dense_gemm (include/moe_block.h): checks and launches; dense_plan.h chooses the form.
#include <hip/hip_runtime.h>

#include "dense_device.h"

extern "C" {

size_t moe_dense_gemm_workspace(int32_t T, int32_t N, int32_t K) {
  if (T < 1 || N < 1 || K < 1) return 0;
  const moe::DensePlan p = moe::dense_plan(T, N, K, true);
  return p.splits > 1 ? (size_t)p.splits * T * moe::dense_pitch(N) * sizeof(float) : 0;
}

int moe_dense_gemm(const moe_dense_args* p, void* stream) {
  using namespace moe;
  if (!p) return MOE_DECODE_ERR_INVALID_ARG;
  const moe_dense_args& a = *p;
  if (a.T < 0 || a.N < 1 || a.K < 1) return MOE_DECODE_ERR_INVALID_ARG;
  if (a.T > MOE_ROWS_MAX_TOKENS || a.N > MOE_DENSE_MAX_DIM || a.K > MOE_DENSE_MAX_DIM || a.K % 8 || a.act < MOE_ACT_NONE ||
      a.act > MOE_ACT_SIGMOID)
    return MOE_DECODE_ERR_UNSUPPORTED;
  const auto other = [](int d) { return d != MOE_DTYPE_F32 && d != MOE_DTYPE_BF16; };
  if (other(a.out_dtype) || (a.bias && other(a.bias_dtype)) || (a.residual && other(a.residual_dtype)))
    return MOE_DECODE_ERR_UNSUPPORTED;
  if (a.T == 0) return MOE_DECODE_OK;
  if (!a.x || !a.w || !a.out) return MOE_DECODE_ERR_INVALID_ARG;
  const bool bias_f32 = a.bias && a.bias_dtype == MOE_DTYPE_F32, residual_f32 = a.residual && a.residual_dtype == MOE_DTYPE_F32;
  if (misaligned(a.x, 16) || misaligned(a.w, 16) || misaligned(a.out, 16) || misaligned(a.bias, bias_f32 ? 4 : 2) ||
      misaligned(a.residual, residual_f32 ? 4 : 2))
    return MOE_DECODE_ERR_INVALID_ARG;
  // strides of a single row mean nothing
  const int64_t ldx = a.T > 1 ? a.ldx : a.K, ldw = a.N > 1 ? a.ldw : a.K, ldr = a.T > 1 && a.residual ? a.ldr : a.N;
  if (ldx < a.K || ldw < a.K || ldr < a.N || ldx % 8 || ldw % 8) return MOE_DECODE_ERR_INVALID_ARG;
  if (ldx > kDenseMaxStride || ldw > kDenseMaxStride || ldr > kDenseMaxStride) return MOE_DECODE_ERR_UNSUPPORTED;
  if (misaligned(a.workspace, 16)) return MOE_DECODE_ERR_INVALID_ARG;
  const size_t need = moe_dense_gemm_workspace(a.T, a.N, a.K);
  if (a.workspace && a.workspace_bytes < need) return MOE_DECODE_ERR_SCRATCH_TOO_SMALL;

  DenseArgs d{};
  d.x = static_cast<const uint16_t*>(a.x);
  d.w = static_cast<const uint16_t*>(a.w);
  d.bias = a.bias;
  d.residual = a.residual;
  d.out = a.out;
  d.ldx = ldx;
  d.ldw = ldw;
  d.ldr = ldr;
  d.T = a.T;
  d.N = a.N;
  d.K = a.K;
  d.act = a.act;
  d.out_f32 = a.out_dtype == MOE_DTYPE_F32;
  d.bias_f32 = bias_f32;
  d.residual_f32 = residual_f32;
  d.vector_io = a.N % 8 == 0 && ldr % 8 == 0 && !misaligned(a.residual, 16);
  hipStream_t s = static_cast<hipStream_t>(stream);
  const DensePlan plan = dense_plan(a.T, a.N, a.K, a.workspace != nullptr);
  d.splits = plan.splits;
  d.partial = static_cast<float*>(a.workspace);
  if (plan.shape < kDense64x128)
    launch_dense_strip(d, plan.shape, s);
  else
    launch_dense_tile(d, plan.shape, s);
  return hipGetLastError() == hipSuccess ? MOE_DECODE_OK : MOE_DECODE_ERR_HIP;
}

}  // extern "C"

// Products grouped by expert over ragged rows (include/moe_rows.h): the calls
// moe_grouped_gemm and moe_grouped_swiglu, over the kernels of
// grouped_product.hip and grouped_swiglu.hip.
#include <hip/hip_runtime.h>

#include "../../include/moe_rows.h"
#include "grouped_device.h"

namespace moe {
namespace {

bool misaligned(const void* p, uintptr_t to) { return (reinterpret_cast<uintptr_t>(p) & (to - 1)) != 0; }

int check(const moe_grouped_args* p) {
  if (!p) return MOE_DECODE_ERR_INVALID_ARG;
  const moe_grouped_args& a = *p;
  if (a.R < 0 || a.X < 0 || a.E < 1 || a.N < 1 || a.K < 1) return MOE_DECODE_ERR_INVALID_ARG;
  if (a.E > MOE_DECODE_MAX_EXPERTS || a.N % 128 || a.K % 128 || a.N > MOE_ROWS_MAX_DIM || a.K > MOE_ROWS_MAX_DIM ||
      a.quant < MOE_QUANT_FP8 || a.quant > MOE_QUANT_MXFP8)
    return MOE_DECODE_ERR_UNSUPPORTED;
  if (a.R == 0) return MOE_DECODE_OK;
  if (a.X < (a.rows ? 1 : a.R)) return MOE_DECODE_ERR_INVALID_ARG;
  if (!a.x || !a.x_scale || !a.offsets || !a.w || !a.w_scale || !a.out) return MOE_DECODE_ERR_INVALID_ARG;
  if (misaligned(a.x, 16) || misaligned(a.w, 16) || misaligned(a.out, 16) || misaligned(a.w_scale, 4) ||
      misaligned(a.offsets, 4) || misaligned(a.rows, 4) || misaligned(a.x_scale, 4))
    return MOE_DECODE_ERR_INVALID_ARG;
  // a grid's limit, 2^32 threads (64-row tiles come with R <= 24 E only, far below it)
  if (((int64_t)a.R / 128 + a.E) * ((a.N + 255) / 256) > (int64_t)(UINT32_MAX / 512) - 8) return MOE_DECODE_ERR_UNSUPPORTED;
  return MOE_DECODE_OK;
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
  g.limit = a.limit;
  return g;
}

}  // namespace
}  // namespace moe

extern "C" {

int moe_grouped_gemm(const moe_grouped_args* args, void* stream) {
  using namespace moe;
  if (const int rc = check(args)) return rc;
  if (args->R == 0) return MOE_DECODE_OK;
  const GroupedArgs a = kernel_args(*args);
  hipStream_t s = static_cast<hipStream_t>(stream);
  launch_grouped_product(args->quant == MOE_QUANT_MXFP8, a, s);
  return hipGetLastError() == hipSuccess ? MOE_DECODE_OK : MOE_DECODE_ERR_HIP;
}

int moe_grouped_swiglu(const moe_grouped_args* args, void* stream) {
  using namespace moe;
  if (const int rc = check(args)) return rc;
  if (args->N % 256) return MOE_DECODE_ERR_UNSUPPORTED;
  if (!(args->limit > 0.f)) return MOE_DECODE_ERR_INVALID_ARG;
  if (args->R == 0) return MOE_DECODE_OK;
  if (!args->out_scale || misaligned(args->out_scale, 4)) return MOE_DECODE_ERR_INVALID_ARG;
  const GroupedArgs a = kernel_args(*args);
  hipStream_t s = static_cast<hipStream_t>(stream);
  launch_grouped_swiglu(args->quant == MOE_QUANT_MXFP8, a, s);
  return hipGetLastError() == hipSuccess ? MOE_DECODE_OK : MOE_DECODE_ERR_HIP;
}

}  // extern "C"

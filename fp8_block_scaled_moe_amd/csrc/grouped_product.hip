// moe_grouped_gemm with FP32 sums: up to 128 rows of an expert by 256 weight
// rows per workgroup, by grouped_tile.h's tile, rounded to BF16.
//
// Bounds, measured on MI355X. Few rows: the weights' bytes (one token, 8 experts,
// N = 7168, K = 2048: 20.1 us, 5.8 TB/s; 2,474 MXFP8 rows over 56 experts, N = 2048,
// K = 3584: 101 us, 4.1 TB/s). Many: as the SwiGLU (65,536 rows over 256 experts,
// N = 7168, K = 2048: 2.36 ms, 0.82 PFLOP/s; matrix instructions 41% of the cycles,
// vector instructions 46%, waves waiting for 35% of theirs; 6% of the rows
// multiplied are padding). grouped_product_fp8.hip takes 1.42 ms.
#include <hip/hip_runtime.h>

#include "grouped_tile.h"

namespace moe {
namespace {

template <bool kMx, bool kAll>
__global__ __launch_bounds__(kThreads, 2) void grouped_product_kernel(GroupedArgs a) {
  __shared__ Shared sm;
  grouped_tile<false, kMx, kAll>(a, sm);
}

}  // namespace

void launch_grouped_product(bool mx, GroupedArgs a, hipStream_t stream) {
  a.col_tiles = (a.N + 255) / 256 * a.splits;
  const auto kernel = all_of_k(a) ? mx ? grouped_product_kernel<true, true> : grouped_product_kernel<false, true>
                      : mx        ? grouped_product_kernel<true, false>
                                  : grouped_product_kernel<false, false>;
  hipLaunchKernelGGL(kernel, dim3(grouped_workgroups(a, a.R, kRows)), dim3(kThreads), 0, stream, a);
}

}  // namespace moe

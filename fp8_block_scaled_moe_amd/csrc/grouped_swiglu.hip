// moe_grouped_swiglu: up to 128 rows of an expert by 128 hidden columns (256
// weight rows, up and gate) per workgroup, by grouped_tile.h's tile: the hidden's
// codes and scales are decided from its sums, and sums of the FP8 instruction
// would move an FP32 scale by 1e-5, ten times what FP32 sums do.
//
// Bounds, measured on MI355X. Few rows: the weights' bytes (4 tokens x 8 of 256
// experts, K = 7168, I = 2048: 134 to 140 us, 6.7 TB/s and more). Many: no unit
// alone. 65,536 rows over 256 such experts take 4.6 ms, 0.83 PFLOP/s: matrix
// instructions are busy for 44% of the cycles and vector instructions (8.6 for each
// of them: widening, scaled sums) for 48%, at the 1.8-2.0 GHz that their power
// allows, and the waves wait for 35% of theirs, since all of a SIMD's are in the same
// phase of a block between two barriers. Dense rows (4,096 for each of 8 experts)
// reach 1.0 PFLOP/s, 1.23 without the copies; a loop of the same instructions on
// registers 1.3, a BF16 library product 1.22. MXFP8 rows 5.1 ms. Tiles of 32 rows with
// four blocks in LDS gained 1% below 5 rows an expert and lost 9% at 12, so there is
// one size.
#include <hip/hip_runtime.h>

#include "grouped_tile.h"

namespace moe {
namespace {

template <bool kMx, bool kAll>
__global__ __launch_bounds__(kThreads, 2) void grouped_swiglu_kernel(GroupedArgs a) {
  __shared__ Shared sm;
  grouped_tile<true, kMx, kAll>(a, sm);
}

}  // namespace

void launch_grouped_swiglu(bool mx, GroupedArgs a, hipStream_t stream) {
  a.col_tiles = a.N / 256 * a.splits;
  const auto kernel = all_of_k(a) ? mx ? grouped_swiglu_kernel<true, true> : grouped_swiglu_kernel<false, true>
                      : mx        ? grouped_swiglu_kernel<true, false>
                                  : grouped_swiglu_kernel<false, false>;
  hipLaunchKernelGGL(kernel, dim3(grouped_workgroups(a, a.R, kRows)), dim3(kThreads), 0, stream, a);
}

}  // namespace moe

// moe_dense_gemm (include/moe_block.h): checks, and the choice of a kernel by what its
// workgroups have to take in and to multiply.
#include <hip/hip_runtime.h>

#include <cmath>

#include "dense_device.h"

namespace moe {
namespace {

struct Plan {
  int shape, splits;
  double us;
};

// The shape and the parts of K with the least estimated time. Measured on MI355X (in a
// graph, N and K among 256, 896, 2048, 3584, 4096 and 7168):
//   strips: some 3 us, then what is copied: 140 KB a microsecond into one CU, 25 GB a
//     millisecond out of the caches in all (1 row, 7168 -> 256: 3.8 us with 4 x 4, 6.0 with
//     16 x 16; 32 rows, 2048 -> 7168: 6.4 with 32 x 32, 8.2 with 16 x 32, 11.1 with 16 x 16);
//   tiles: 3.5 us, then rounds of the CUs, each so long for a 64-column block of K (`block`;
//     `lone` where many CUs have none) and for a tile's beginning and end (`end`);
//   parts of K: a second launch (3 us) and the partial sums written and read.
// Over 60 sizes drawn from 1 to 16,384 rows the choice was 1.2% slower than the best of
// all shapes on average.
Plan dense_plan(int T, int N, int K, bool split) {
  Plan best{kDense64x128, 1, 1e300};
  const auto offer = [&](int shape, int splits, double us) {
    if (us < best.us) best = Plan{shape, splits, us};
  };
  const auto up = [](double a, double b) { return ceil(a / b); };
  const double cus = kCus, row = (double)K * 2;

  struct Strip {
    int shape, t, n, per;
    double rate, start;
  };
  for (const Strip& s : {Strip{kDenseStrip4x4, 4, 4, 2, 140e3, 3.1}, Strip{kDenseStrip8x8, 8, 8, 2, 140e3, 2.9},
                         Strip{kDenseStrip16x16, 16, 16, 1, 140e3, 2.8}, Strip{kDenseStrip16x32, 16, 32, 1, 140e3, 3.1},
                         Strip{kDenseStrip32x32, 32, 32, 1, 140e3, 3.2}, Strip{kDenseStrip32x64, 32, 64, 1, 110e3, 3.5}}) {
    const double wgs = up(T, s.t) * up(N, s.n), rounds = up(wgs, cus * s.per), bytes = (s.t + s.n) * row;
    const double cu = rounds * s.per * bytes / s.rate, caches = wgs * bytes / 25e6;
    if (wgs < 1 << 24) offer(s.shape, 1, s.start + (rounds - 1) * 4.0 + (cu > caches ? cu : caches));
  }

  struct Tile {
    int shape, t, n, per, splits;
    double block, lone, end;
  };
  for (const Tile& s : {Tile{kDense64x128, 64, 128, 1, 8, 0.29, 0.25, 2.7}, Tile{kDense128x128, 128, 128, 1, 4, 0.44, 0.36, 4.0},
                        Tile{kDense128x128Two, 128, 128, 2, 1, 0.785, 0.60, 6.0}, Tile{kDense256x256, 256, 256, 1, 1, 1.32, 1.09, 8.0}})
    for (int splits = 1; splits <= (split ? s.splits : 1); splits *= 2) {
      const double blocks = up(up(K, 64), splits);
      if (splits > 1 && blocks < 8) break;
      const double tiles = up(T, s.t) * up(N, s.n) * splits, slots = cus * s.per;
      const double full = floor(tiles / slots), rest = tiles - full * slots;
      const double last = rest == 0 ? 0.0 : blocks * (rest <= 0.75 * cus ? s.lone : s.block) + s.end;
      const double join = splits > 1 ? 3.0 + splits * (double)T * N * 4 / 3e6 : 0.0;
      offer(s.shape, splits, 3.5 + full * (blocks * s.block + s.end) + last + join);
      if (s.shape == kDense256x256 && rest > 0 && rest <= cus / 2)
        offer(kDenseHalves, 1, 3.5 + full * (blocks * s.block + s.end) + blocks * 0.70 + 6.0);
    }
  return best;
}

}  // namespace
}  // namespace moe

extern "C" {

size_t moe_dense_gemm_workspace(int32_t T, int32_t N, int32_t K) {
  if (T < 1 || N < 1 || K < 1) return 0;
  const moe::Plan p = moe::dense_plan(T, N, K, true);
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
  const Plan plan = dense_plan(a.T, a.N, a.K, a.workspace != nullptr);
  d.splits = plan.splits;
  d.partial = static_cast<float*>(a.workspace);
  if (plan.shape < kDense64x128)
    launch_dense_strip(d, plan.shape, s);
  else
    launch_dense_tile(d, plan.shape, s);
  return hipGetLastError() == hipSuccess ? MOE_DECODE_OK : MOE_DECODE_ERR_HIP;
}

}  // extern "C"

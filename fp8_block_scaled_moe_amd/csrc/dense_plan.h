// Which form of the dense product (moe_dense_gemm in moe_block.h) a call of given sizes
// takes. Host code without HIP.
#pragma once

#include <cmath>
#include <initializer_list>

namespace moe {

constexpr int kCus = 256;

// Rows of x by weight rows of a workgroup, and how many workgroups a CU holds.
enum DenseShape {
  kDenseStrip4x4,
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

struct DensePlan {
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
// Over 60 sizes drawn from 1 to 16,384 rows the choice was 1.5% slower than the best of
// all shapes on average, 1.3 times at worst (16,054 rows, K = 88, N = 1).
inline DensePlan dense_plan(int T, int N, int K, bool split) {
  DensePlan best{kDense64x128, 1, 1e300};
  const auto offer = [&](int shape, int splits, double us) {
    if (us < best.us) best = DensePlan{shape, splits, us};
  };
  const auto up = [](double a, double b) { return ceil(a / b); };
  const double cus = kCus, row = (double)K * 2;

  struct Strip {
    int shape, t, n, per;
    double rate, start;
  };
  for (const Strip& s : {Strip{kDenseStrip4x4, 4, 4, 2, 140e3, 3.1}, Strip{kDenseStrip16x16, 16, 16, 1, 140e3, 2.8},
                         Strip{kDenseStrip16x32, 16, 32, 1, 140e3, 3.1}, Strip{kDenseStrip32x32, 32, 32, 1, 140e3, 3.2},
                         Strip{kDenseStrip32x64, 32, 64, 1, 110e3, 3.5}}) {
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

}  // namespace moe

// The dense product for few rows: every wave has K blocks of its own.
//
// Bound by how fast a CU takes in the weights (some 140 KB a microsecond through LDS) and by
// a launch's beginning and end, some 3 us: 1 row, 7168 -> 256 3.8 us in 64 workgroups of 4 x 4
// (6.0 in 16 of 16 x 16); 32 rows, 2048 -> 7168 6.4 us, 30.4 MB at 4.8 TB/s, most of it out of
// the caches. A wave's own stages and K blocks need no barrier before the sums are added.
#include <hip/hip_runtime.h>

#include <type_traits>

#include "dense_device.h"

namespace moe {
namespace {

// A workgroup has 16 kI / kS weight rows by 16 kJ / kS rows of x; its waves take the
// blocks of K in turn, each through LDS of its own, so that no wave waits for
// another before the end. The 16 rows of an operand of the matrix instruction are 16 /
// kS rows by kS neighbouring pieces of 64 columns each; of the products only those of
// a piece with itself count. A block is 64 kS columns, kDepth of them are on their way.
template <int kI, int kJ, int kS, int kWaves, int kDepth>
__global__ __launch_bounds__(kWaves* kWave) void strip_kernel(DenseArgs a, int row_tiles, int tiles) {
  constexpr int kBlock = 64 * kS, kN = 16 * kI / kS, kT = 16 * kJ / kS, kStage = (kI + kJ) * 2048, kCopies = 2 * (kI + kJ);
  constexpr int kSumBytes = kWaves * kJ * kI * 16 * 20 * 4, kLds = kWaves * kDepth * kStage;
  __shared__ alignas(16) uint8_t sm[kLds > kSumBytes ? kLds : kSumBytes];
  const int tid = threadIdx.x, lane = tid & (kWave - 1);
  const int wave = __builtin_amdgcn_readfirstlane(tid / kWave);
  // each XCD (workgroup id mod 8) takes a contiguous eighth of the tiles, those of the same weights next to each other
  const int share = (tiles + 7) / 8, tile = (int)(blockIdx.x & 7) * share + (int)(blockIdx.x >> 3);
  if ((int)(blockIdx.x >> 3) >= share || tile >= tiles) return;
  const int n0 = tile / row_tiles * kN, t0 = tile % row_tiles * kT;
  // A copy: eight operand rows of 128 bytes; row L keeps 16-byte chunk c at place c ^ (L /
  // 2 % 8).
  const uint8_t* const xbase = reinterpret_cast<const uint8_t*>(a.x + (size_t)t0 * a.ldx);
  const uint8_t* const wbase = reinterpret_cast<const uint8_t*>(a.w + (size_t)n0 * a.ldw);
  const int piece = lane & 7;
  uint32_t off[kCopies];
  int col[2];  // first column of the lane's 16 bytes in a block, by the copy's parity
#pragma unroll
  for (int i = 0; i < kCopies; ++i) {
    const int L = (i & 1) * 8 + (lane >> 3), row = L / kS, c = L % kS * 64 + (piece ^ (L >> 1 & 7)) * 8;
    col[i & 1] = c;
    const int f = i / 2;  // operand: x's first
    off[i] = f < kJ ? (uint32_t)(min(f * (16 / kS) + row, a.T - 1 - t0) * (int)a.ldx + c) * 2u
                    : (uint32_t)(min((f - kJ) * (16 / kS) + row, a.N - 1 - n0) * (int)a.ldw + c) * 2u;
  }
  const uint32_t lds = lds_offset(sm) + wave * kDepth * kStage;
  const auto issue = [&](int st, int b) {
    const uint32_t to = lds + st * kStage;
    const size_t k = (size_t)b * kBlock * 2;
    if ((b + 1) * kBlock <= a.K) {
#pragma unroll
      for (int i = 0; i < kCopies; ++i) copy16_to_lds<false>(i / 2 < kJ ? xbase + k : wbase + k, off[i], to + i * 1024);
    } else {
#pragma unroll
      for (int i = 0; i < kCopies; ++i)
        copy16_to_lds(b * kBlock + col[i & 1] < a.K ? (i / 2 < kJ ? xbase : wbase) + k + off[i] : reinterpret_cast<const uint8_t*>(kNothing),
                      to + i * 1024);
    }
  };
  const int r = lane & 15, quarter = lane >> 4;
  float4_t acc[kJ][kI];
#pragma unroll
  for (int j = 0; j < kJ; ++j)
#pragma unroll
    for (int i = 0; i < kI; ++i) acc[j][i] = float4_t{0.f, 0.f, 0.f, 0.f};
  const int blocks = (a.K + kBlock - 1) / kBlock, mine = wave < blocks ? (blocks - wave + kWaves - 1) / kWaves : 0;
  // Block i's products; its copies have ended. Behind its reads the next block goes into its place.
  const auto step = [&](int st, int i, auto more) {
    bf16x8_t w[2][kI], x[2][kJ];
    const uint8_t* from = sm + (wave * kDepth + st) * kStage + r * 128;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int at = ((quarter + 4 * h) ^ (r >> 1)) * 16;
#pragma unroll
      for (int j = 0; j < kJ; ++j) x[h][j] = *reinterpret_cast<const bf16x8_t*>(from + j * 2048 + at);
#pragma unroll
      for (int q = 0; q < kI; ++q) w[h][q] = *reinterpret_cast<const bf16x8_t*>(from + (kJ + q) * 2048 + at);
    }
    if (decltype(more)::value) {
      asm volatile("s_waitcnt lgkmcnt(0)" ::"v"(sm) : "memory");
      issue(st, wave + (i + kDepth) * kWaves);
    }
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int j = 0; j < kJ; ++j)
#pragma unroll
        for (int q = 0; q < kI; ++q) acc[j][q] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(w[h][q], x[h][j], acc[j][q], 0, 0, 0);
  };
#pragma unroll
  for (int d = 0; d < kDepth; ++d)
    if (d < mine) issue(d, wave + d * kWaves);
  int i = 0, st = 0;
  for (; i + kDepth < mine; ++i) {
    copies_left<(kDepth - 1) * kCopies>(sm);
    step(st, i, std::true_type{});
    st = st == kDepth - 1 ? 0 : st + 1;
  }
  for (; i < mine; ++i) {
    const int left = mine - 1 - i;  // blocks behind it, all on their way
    if (kDepth > 3 && left == 3) copies_left<3 * kCopies>(sm);
    if (kDepth > 2 && left == 2) copies_left<2 * kCopies>(sm);
    if (left == 1) copies_left<kCopies>(sm);
    if (left == 0) copies_left<0>(sm);
    step(st, i, std::false_type{});
    st = st == kDepth - 1 ? 0 : st + 1;
  }
  __syncthreads();
  // a lane's sums: row r of x's operand, rows 4 (l / 16) + q of the weights'
  float(*const sums)[kJ][kI][16][20] = reinterpret_cast<float(*)[kJ][kI][16][20]>(sm);
#pragma unroll
  for (int j = 0; j < kJ; ++j)
#pragma unroll
    for (int q = 0; q < kI; ++q) *reinterpret_cast<float4_t*>(&sums[wave][j][q][r][quarter * 4]) = acc[j][q];
  __syncthreads();
  for (int q = tid; q < kT * kN; q += kWaves * kWave) {
    const int t = q / kN, n = q % kN, j = t * kS / 16, i2 = n * kS / 16, tr = t * kS % 16, nr = n * kS % 16;
    float v = 0.f;
#pragma unroll
    for (int p = 0; p < kWaves; ++p)
#pragma unroll
      for (int s = 0; s < kS; ++s) v += sums[p][j][i2][tr + s][nr + s];
    if (t0 + t < a.T && n0 + n < a.N) finish(a, t0 + t, n0 + n, v);
  }
}

template <int kI, int kJ, int kS, int kWaves, int kDepth>
void launch(const DenseArgs& a, hipStream_t stream) {
  static_assert(kDepth >= 2 && kDepth <= 4, "the waits");
  const int rows = (a.T + 16 * kJ / kS - 1) / (16 * kJ / kS), tiles = rows * ((a.N + 16 * kI / kS - 1) / (16 * kI / kS));
  hipLaunchKernelGGL((strip_kernel<kI, kJ, kS, kWaves, kDepth>), dim3((tiles + 7) / 8 * 8), dim3(kWaves * kWave), 0, stream, a, rows, tiles);
}

}  // namespace

void launch_dense_strip(const DenseArgs& a, int shape, hipStream_t stream) {
  switch (shape) {
    case kDenseStrip4x4:
      return launch<1, 1, 4, 8, 2>(a, stream);
    case kDenseStrip16x16:
      return launch<1, 1, 1, 8, 4>(a, stream);
    case kDenseStrip16x32:
      return launch<2, 1, 1, 8, 3>(a, stream);
    case kDenseStrip32x32:
      return launch<2, 2, 1, 8, 2>(a, stream);
    default:
      return launch<4, 2, 1, 4, 3>(a, stream);
  }
}

}  // namespace moe

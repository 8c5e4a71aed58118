// The dense product in tiles through LDS.
//
// K blocks of 64 columns of the tile's rows and weight rows are copied into LDS (two to
// five of them at a time) and multiplied by the 16x16x32 instruction, the reads of the
// next 32 columns and the copies of a block ahead placed between the matrix
// instructions. What bounds a large product is power: taking out every wait and barrier
// of the loop does not change its time, and the 16x16x32 instruction is faster than
// 32x32x16 at the same rate per cycle (8,192 x 4,096, K = 7168: 326 and 359 us), since it
// moves its sums half as often. 256 x 256 tiles: 1.47 PFLOP/s at that size on the same
// inputs again (1.41 with bias and the tanh form, 1.30 on changing inputs); eight waves of
// 64 x 128, two a SIMD (four of 128 x 128 leave a SIMD idle at every wait: 393 us). A tile
// ends in 8 us (8,192 x 4,096, K = 64: 21 us, 67 MB of them stored); workgroups that stay
// for their next tile and request its blocks before they store were slower (8,192 x 7,168,
// K = 2048: 197 and 187 us). Short prompts are bound by a block's own chain: at 509 x 7168
// -> 3584, 64 x 128 tiles, 36 us, a wave has eight matrix instructions between two barriers;
// of the cycles of a CU the matrix cores are busy for 37%, LDS for 38% (a 16-byte read of a
// wave takes it four cycles), and the waves wait for 45%.
#include <hip/hip_runtime.h>

#include "dense_device.h"

namespace moe {
namespace {

// A wave's product: 16 kMJ rows of x by 16 kNJ weight rows; a workgroup's: kWM by
// kWN of them. A K block of the tile is 64 columns (128 bytes a row), kStages of them
// in LDS.
template <int kMJ_, int kNJ_, int kWM_, int kWN_, int kBlock_, int kStages_, int kWgs_>
struct Shape {
  static constexpr int kMJ = kMJ_, kNJ = kNJ_, kWM = kWM_, kWN = kWN_, kBlock = kBlock_, kStages = kStages_, kWgs = kWgs_;
  static constexpr int kRow = 2 * kBlock, kPieces = kRow / 16, kCopyRows = kWave / kPieces, kSteps = kBlock / 32;
  static constexpr int kWaves = kWM * kWN, kThreads = kWaves * kWave;
  static constexpr int kM = 16 * kMJ * kWM, kN = 16 * kNJ * kWN;
  static constexpr int kStageBytes = (kM + kN) * kRow;
  static constexpr int kXCopies = kM / kCopyRows / kWaves, kWCopies = kN / kCopyRows / kWaves, kCopies = kXCopies + kWCopies;
  // Behind the products: FP32 sums of some of a wave's rows by up to 64 columns at a time
  static constexpr int kMostLds = 160 * 1024 / kWgs;
  static constexpr int kOutCols = kNJ % 4 == 0 ? 64 : kNJ % 2 == 0 ? 32 : 16, kOutPitch = kOutCols + 4;
  static constexpr int out_bytes(int j) { return 16 * j * kOutPitch * 4; }
  static constexpr int kOutJ = kWaves * out_bytes(kMJ) <= kMostLds ? kMJ : kMJ % 2 == 0 && kWaves * out_bytes(kMJ / 2) <= kMostLds ? kMJ / 2 : 1;
  static constexpr int kOutBytes = out_bytes(kOutJ);
  static constexpr int kLds = kStages * kStageBytes > kWaves * kOutBytes ? kStages * kStageBytes : kWaves * kOutBytes;
  static_assert(kLds <= kMostLds && kOutJ >= 1, "LDS of the workgroups of a CU");
  static_assert(kM % (kCopyRows * kWaves) == 0 && kN % (kCopyRows * kWaves) == 0, "whole copies");
};

// A workgroup's tile: rows from t0, columns from n0 on, part `split` of K.
template <typename S>
__device__ __forceinline__ void dense_tile(const DenseArgs& a, uint8_t* sm, int t0, int n0, int split) {
  constexpr int kMJ = S::kMJ, kNJ = S::kNJ;
  const int tid = threadIdx.x, lane = tid & (kWave - 1);
  const int wave = __builtin_amdgcn_readfirstlane(tid / kWave);
  const int r16 = lane & 15, quarter = lane >> 4, wm = wave / S::kWN, wn = wave % S::kWN;
  const int all_blocks = (a.K + S::kBlock - 1) / S::kBlock;
  const int first = (int)((int64_t)all_blocks * split / a.splits), KB = (int)((int64_t)all_blocks * (split + 1) / a.splits) - first;

  // What a lane copies of a block: 16 bytes of a row each. LDS row L keeps 16-byte
  // chunk c of its row at place c ^ (L / 2 % 8) (64-column blocks), so that the 16 rows
  // of a read phase differ in bank.
  constexpr int kRow = S::kRow;
  const int lr = lane / S::kPieces, piece = lane % S::kPieces;
  const auto swizzle = [](int L) { return L / (256 / kRow) % S::kPieces; };
  const uint8_t* const xbase = reinterpret_cast<const uint8_t*>(a.x) + ((size_t)t0 * a.ldx + (size_t)first * S::kBlock) * 2;
  const uint8_t* const wbase = reinterpret_cast<const uint8_t*>(a.w) + ((size_t)n0 * a.ldw + (size_t)first * S::kBlock) * 2;
  uint32_t xoff[S::kXCopies], woff[S::kWCopies];
#pragma unroll
  for (int i = 0; i < S::kXCopies; ++i) {
    const int L = (wave * S::kXCopies + i) * S::kCopyRows + lr;
    xoff[i] = (uint32_t)(min(L, a.T - 1 - t0) * (int)a.ldx) * 2u + (piece ^ swizzle(L)) * 16;
  }
#pragma unroll
  for (int i = 0; i < S::kWCopies; ++i) {
    const int L = (wave * S::kWCopies + i) * S::kCopyRows + lr;
    woff[i] = (uint32_t)(min(L, a.N - 1 - n0) * (int)a.ldw) * 2u + (piece ^ swizzle(L)) * 16;
  }
  const uint32_t lds = lds_offset(sm);
  const auto copy = [&](int i, int st, int b) {  // one of the wave's copies of a whole block
    const uint32_t to = lds + st * S::kStageBytes;
    if (i < S::kXCopies)
      copy16_to_lds<false>(xbase + (size_t)b * kRow, xoff[i], to + (wave * S::kXCopies + i) * 1024);
    else
      copy16_to_lds<false>(wbase + (size_t)b * kRow, woff[i - S::kXCopies], to + S::kM * kRow + (wave * S::kWCopies + i - S::kXCopies) * 1024);
  };
  const auto issue = [&](int st, int b) {  // all of them, of any block
    const int left = a.K - (first + b) * S::kBlock;  // columns of the block
    if (left >= S::kBlock) {
#pragma unroll
      for (int i = 0; i < S::kCopies; ++i) copy(i, st, b);
    } else {
      const uint32_t to = lds + st * S::kStageBytes;
      const uint8_t *xp = xbase + (size_t)b * kRow, *wp = wbase + (size_t)b * kRow;
      const uint8_t* const nothing = reinterpret_cast<const uint8_t*>(kNothing);
#pragma unroll
      for (int i = 0; i < S::kXCopies; ++i)
        copy16_to_lds((piece ^ swizzle((wave * S::kXCopies + i) * S::kCopyRows + lr)) * 8 < left ? xp + xoff[i] : nothing,
                      to + (wave * S::kXCopies + i) * 1024);
#pragma unroll
      for (int i = 0; i < S::kWCopies; ++i)
        copy16_to_lds((piece ^ swizzle((wave * S::kWCopies + i) * S::kCopyRows + lr)) * 8 < left ? wp + woff[i] : nothing,
                      to + S::kM * kRow + (wave * S::kWCopies + i) * 1024);
    }
  };

  // 32 columns of every row (16-byte chunk l / 16 + 4 c of row l % 16) at a time, read
  // while the matrix instructions of the 32 before run: the weights' into other
  // registers, the rows of x into the ones that the last instruction is done with.
  int off[S::kSteps];
#pragma unroll
  for (int c = 0; c < S::kSteps; ++c) off[c] = r16 * kRow + ((quarter + 4 * c) ^ swizzle(r16)) * 16;
  bf16x8_t x[kMJ], w[2][kNJ];  // [step parity]
  float4_t acc[kMJ][kNJ];
#pragma unroll
  for (int j = 0; j < kMJ; ++j)
#pragma unroll
    for (int t = 0; t < kNJ; ++t) acc[j][t] = float4_t{0.f, 0.f, 0.f, 0.f};
  const auto read_x = [&](int j, int st, int c) {
    x[j] = *reinterpret_cast<const bf16x8_t*>(sm + st * S::kStageBytes + off[c] + (wm * kMJ + j) * 16 * kRow);
  };
  const auto read_w = [&](int t, int st, int c) {
    w[c & 1][t] = *reinterpret_cast<const bf16x8_t*>(sm + st * S::kStageBytes + S::kM * kRow + off[c] + (wn * kNJ + t) * 16 * kRow);
  };
  // The products of step c, the reads of step `next` of stage `st` and, with kCopy, the
  // copies of block `b` into stage `to` between them. Neighbouring instructions share an operand.
  constexpr int kOps = kMJ * kNJ, kReadEvery = kMJ >= 4 ? kMJ / 2 : 1;
  constexpr int kCopyAtOnce = (S::kCopies + kOps - 1) / kOps, kCopyEvery = kOps * kCopyAtOnce / S::kCopies;
  const auto chunk = [&](auto reads, auto copies, int c, int st, int next, int to, int b) {
#pragma unroll
    for (int i = 0; i < kOps; ++i) {
      const int j = i / kNJ, t = j % 2 ? kNJ - 1 - i % kNJ : i % kNJ;
      acc[j][t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(w[c & 1][t], x[j], acc[j][t], 0, 0, 0);
      if (decltype(reads)::value) {
        if (i % kReadEvery == 0 && i / kReadEvery < kNJ) read_w(i / kReadEvery, st, next);
        if (i % kNJ == kNJ - 1) read_x(j, st, next);
      }
      if (decltype(copies)::value && i % kCopyEvery == 0)
#pragma unroll
        for (int q = 0; q < kCopyAtOnce; ++q)
          if (i / kCopyEvery * kCopyAtOnce + q < S::kCopies) copy(i / kCopyEvery * kCopyAtOnce + q, to, b);
      if (kOps <= 16 || i % 2) __builtin_amdgcn_sched_barrier(0);
    }
  };
  constexpr std::true_type yes{};
  constexpr std::false_type no{};
  // Block b's copies have ended, in every wave, and every wave has read all of the
  // block before. The copies of kStages - 2 blocks behind may be on their way.
  const auto ready = [&](int b) {
    if (b + S::kStages - 2 < KB)
      copies_left<(S::kStages - 2) * S::kCopies>(sm);
    else
      copies_left<0>(sm);
    workgroup_barrier();
  };

#pragma unroll
  for (int b = 0; b < S::kStages - 1; ++b)
    if (b < KB) issue(b, b);
  ready(0);
  if (S::kStages - 1 < KB) issue(S::kStages - 1, S::kStages - 1);
#pragma unroll
  for (int j = 0; j < kMJ; ++j) read_x(j, 0, 0);
#pragma unroll
  for (int t = 0; t < kNJ; ++t) read_w(t, 0, 0);
  int st = 0;
  const auto all_but_last = [&] {
#pragma unroll
    for (int c = 0; c + 1 < S::kSteps; ++c) chunk(yes, no, c, st, c + 1, 0, 0);
  };
  constexpr int kLast = S::kSteps - 1;
  const auto after = [&](int s) { return s == S::kStages - 1 ? 0 : s + 1; };
  int b = 0;
  for (; b + S::kStages + 1 < KB; ++b) {  // the block to copy is whole
    all_but_last();
    ready(b + 1);
    chunk(yes, yes, kLast, after(st), 0, st, b + S::kStages);
    st = after(st);
  }
  for (; b + 1 < KB; ++b) {
    all_but_last();
    ready(b + 1);
    if (b + S::kStages < KB) issue(st, b + S::kStages);
    st = after(st);
    chunk(yes, no, kLast, st, 0, 0, 0);
  }
  all_but_last();
  chunk(no, no, kLast, 0, 0, 0, 0);

  // The sums go through LDS, so that a row's columns are finished and stored by
  // neighbouring lanes, eight each, in a loop (the activations' code stands once).
  __syncthreads();
  constexpr int kCols = S::kOutCols, kPitch = S::kOutPitch, kT = kCols / 16, kLanes = kCols / 8;
  float* const mine = reinterpret_cast<float*>(sm + wave * S::kOutBytes);
#pragma unroll
  for (int g = 0; g < kNJ / kT * (kMJ / S::kOutJ); ++g) {
    const int t = g % (kNJ / kT) * kT, j0 = g / (kNJ / kT) * S::kOutJ;
#pragma unroll
    for (int j = 0; j < S::kOutJ; ++j)
#pragma unroll
      for (int u = 0; u < kT; ++u)
        *reinterpret_cast<float4_t*>(mine + (j * 16 + r16) * kPitch + u * 16 + 4 * quarter) = acc[j0 + j][t + u];
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
    const int from = n0 + (wn * kNJ + t) * 16, below = t0 + (wm * kMJ + j0) * 16;
    const int c = lane % kLanes * 8, r0 = lane / kLanes;
    constexpr int kStep = kWave / kLanes, kRows = 16 * S::kOutJ, kAtOnce = kRows / kStep < 4 ? kRows / kStep : 4;
    if (a.splits > 1) {
      if (from + c < a.N)
#pragma unroll 4
        for (int r = r0; r < kRows && below + r < a.T; r += kStep) {
          const float4_t* v = reinterpret_cast<const float4_t*>(mine + r * kPitch + c);
          float4_t* o = reinterpret_cast<float4_t*>(a.partial + ((size_t)split * a.T + below + r) * dense_pitch(a.N) + from + c);
          o[0] = v[0];
          o[1] = v[1];
        }
    } else if (a.vector_io) {
      const Columns<kAtOnce> cols(a, from + c);
      if (from + c < a.N)
#pragma unroll 1
        for (int r = r0; r < kRows && below + r < a.T; r += kAtOnce * kStep) {
          float v[8 * kAtOnce];
#pragma unroll
          for (int q = 0; q < kAtOnce; ++q)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              const float4_t u = *reinterpret_cast<const float4_t*>(mine + (r + q * kStep) * kPitch + c + 4 * i);
#pragma unroll
              for (int k = 0; k < 4; ++k) v[8 * q + 4 * i + k] = u[k];
            }
          cols.finish(a, below + r, kStep, v);
        }
    } else {  // rows that begin anywhere: neighbouring lanes store neighbouring columns
      const int one = lane % kCols;
      for (int r = lane / kCols; r < kRows; r += kWave / kCols)
        if (below + r < a.T && from + one < a.N) finish(a, below + r, from + one, mine[r * kPitch + one]);
    }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
  }
}

// Tiles are numbered in bands of kBand row tiles, in a band column tile by column tile;
// of `count` pieces of work from `first` on each XCD (workgroup id mod 8) takes a
// contiguous eighth, so that what neighbours share meets in one L2.
constexpr int kBand = 8;
__device__ __forceinline__ int64_t dense_piece(int64_t count, int block) {
  const int64_t share = (count + 7) / 8, i = (int64_t)(block & 7) * share + (block >> 3);
  return (block >> 3) < share && i < count ? i : -1;
}
struct TilePlace {
  int row, col;
};
__device__ __forceinline__ TilePlace dense_place(int64_t tile, int row_tiles, int col_tiles) {
  const int64_t band = (int64_t)kBand * col_tiles;
  const int first = (int)(tile / band) * kBand, rows = min(kBand, row_tiles - first), in = (int)(tile % band);
  return TilePlace{first + in % rows, in / rows};
}

// The parts of a tile's K are next to each other.
template <typename S>
__global__ __launch_bounds__(S::kThreads, S::kWaves* S::kWgs / 4) void dense_tile_kernel(DenseArgs a, int row_tiles, int col_tiles) {
  __shared__ alignas(16) uint8_t sm[S::kLds];
  const int64_t i = dense_piece((int64_t)row_tiles * col_tiles * a.splits, blockIdx.x);
  if (i < 0) return;
  const TilePlace at = dense_place(i / a.splits, row_tiles, col_tiles);
  dense_tile<S>(a, sm, at.row * S::kM, at.col * S::kN, (int)(i % a.splits));
}

// The first `whole` tiles of S, the others as two halves of their rows, tiles of H.
template <typename S, typename H>
__global__ __launch_bounds__(S::kThreads, S::kWaves* S::kWgs / 4) void dense_halves_kernel(DenseArgs a, int row_tiles, int col_tiles, int whole) {
  static_assert(S::kM == 2 * H::kM && S::kN == H::kN && S::kThreads == H::kThreads, "halves");
  __shared__ alignas(16) uint8_t sm[S::kLds > H::kLds ? S::kLds : H::kLds];
  const int whole_blocks = (whole + 7) / 8 * 8;
  if ((int)blockIdx.x < whole_blocks) {
    const int64_t i = dense_piece(whole, blockIdx.x);
    if (i < 0) return;
    const TilePlace at = dense_place(i, row_tiles, col_tiles);
    dense_tile<S>(a, sm, at.row * S::kM, at.col * S::kN, 0);
    return;
  }
  const int64_t i = dense_piece(2 * ((int64_t)row_tiles * col_tiles - whole), blockIdx.x - whole_blocks);
  if (i < 0) return;
  const TilePlace at = dense_place(whole + i / 2, row_tiles, col_tiles);
  const int t0 = at.row * S::kM + (int)(i & 1) * H::kM;
  if (t0 < a.T) dense_tile<H>(a, sm, t0, at.col * S::kN, 0);
}

// The parts of K, added in order: eight columns a thread.
constexpr int kJoinThreads = 256;
__global__ __launch_bounds__(kJoinThreads) void dense_join_kernel(DenseArgs a, int groups) {
  const int64_t i = (int64_t)blockIdx.x * kJoinThreads + threadIdx.x;
  const int t = (int)(i / groups);
  if (t >= a.T) return;
  const int n = (int)(i % groups) * 8;
  const size_t pitch = dense_pitch(a.N), step = (size_t)a.T * pitch;
  const float* p = a.partial + (size_t)t * pitch + n;
  float v[8] = {};
#pragma unroll 4
  for (int s = 0; s < a.splits; ++s) {
    const float4_t lo = *reinterpret_cast<const float4_t*>(p + s * step), hi = *reinterpret_cast<const float4_t*>(p + s * step + 4);
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      v[q] += lo[q];
      v[4 + q] += hi[q];
    }
  }
  if (a.vector_io) {
    const Columns<1> cols(a, n);
    cols.finish(a, t, 0, v);
  } else {
#pragma unroll 1
    for (int q = 0; q < 8; ++q) {
      if (n + q < a.N) finish(a, t, n + q, v[0]);
#pragma unroll
      for (int k = 0; k < 7; ++k) v[k] = v[k + 1];
    }
  }
}

template <typename S>
void launch(const DenseArgs& a, hipStream_t stream) {
  const int rows = (a.T + S::kM - 1) / S::kM, cols = (a.N + S::kN - 1) / S::kN;
  const int64_t all = (int64_t)rows * cols * a.splits;
  hipLaunchKernelGGL(dense_tile_kernel<S>, dim3((unsigned)((all + 7) / 8 * 8)), dim3(S::kThreads), 0, stream, a, rows, cols);
  if (a.splits > 1) {
    const int groups = (a.N + 7) / 8;
    hipLaunchKernelGGL(dense_join_kernel, dim3((unsigned)(((int64_t)a.T * groups + kJoinThreads - 1) / kJoinThreads)), dim3(kJoinThreads), 0, stream, a, groups);
  }
}

template <typename S, typename H>
void launch_halves(const DenseArgs& a, hipStream_t stream) {
  const int rows = (a.T + S::kM - 1) / S::kM, cols = (a.N + S::kN - 1) / S::kN;
  const int64_t all = (int64_t)rows * cols, rest = all % kCus, whole = all - rest;
  hipLaunchKernelGGL((dense_halves_kernel<S, H>), dim3((unsigned)(whole + (2 * rest + 7) / 8 * 8)), dim3(S::kThreads), 0, stream, a, rows, cols,
                     (int)whole);
}

}  // namespace

void launch_dense_tile(const DenseArgs& a, int shape, hipStream_t stream) {
  using Big = Shape<4, 8, 4, 2, 64, 2, 1>;
  switch (shape) {
    case kDenseHalves:
      return launch_halves<Big, Shape<4, 4, 2, 4, 64, 3, 1>>(a, stream);
    case kDense256x256:
      return launch<Big>(a, stream);
    case kDense128x128Two:
      return launch<Shape<4, 4, 2, 2, 64, 2, 2>>(a, stream);
    case kDense128x128:
      return launch<Shape<2, 4, 4, 2, 64, 4, 1>>(a, stream);
    default:
      return launch<Shape<2, 2, 2, 4, 64, 5, 1>>(a, stream);
  }
}

}  // namespace moe

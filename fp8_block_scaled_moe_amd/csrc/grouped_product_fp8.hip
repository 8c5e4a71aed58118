// moe_grouped_gemm with the sums of the FP8 matrix instructions, where the
// caller asks for them: up to 256 rows of an expert by 256 weight rows per
// workgroup.
//
// Every 128-wide K block of the tile's activations and weights is copied into
// LDS, read from there by eight waves, up to 128 rows by 64 weight rows each,
// and multiplied by the 16x16x128 instruction, a block's product per
// instruction; its FP32 sums are multiplied by the block's scales when they are
// added. The instruction adds eight products at a time, each cut off 14 bits
// below the power of two of the largest (measured one product at a time), and
// these sums in FP32: 2^-16 of a result on average, a hundredth of what the
// rounding of the rows to BF16 moves, but all of it where large products cancel.
// It runs at three times the rate of the BF16 instruction, which needs its operands
// widened too (grouped_product.hip: 2.36 ms where this one takes 1.42, for 65,536 rows
// over 256 experts, N = 7168, K = 2048).
//
// The weights of a block are in registers from its beginning on, so their
// place in LDS is refilled at once and the activations' place when they have
// been read; the two halves of the waves share the tile's 16-row groups evenly
// and a SIMD has a wave of each. A tile of up to 128 rows has three blocks in
// LDS, a larger one two, and copies no more activation rows than its waves
// read.
//
// Bounds, measured on MI355X. Few rows: the weights' bytes (one token, 8 experts,
// N = 7168, K = 2048: 19.5 us, 6.0 TB/s; 2 rows for each of 64 experts: 6.1, 16:
// 5.8, 28: 5.3, 64: 4.7). Many: 1.6 PFLOP/s for 512 rows for each of 64 experts, 1.9
// without the copies into LDS; an FP8 library product without block scales
// reaches 2.7. For the 65,536 rows above the matrix instructions are busy for 37% of
// the cycles and the waves wait for 36% of theirs: a workgroup fills its CU's LDS, so
// that a tile's start (16 blocks follow it) and its stores overlap with nothing, and
// 17% of the instructions are padding, since a wave has 1, 2, 4, 6 or 8 groups. Tiles
// of at most 128 rows throughout: 3% faster for some 44 rows an expert, 5% slower for
// 110.
#include <hip/hip_runtime.h>

#include <type_traits>

#include "grouped_device.h"

namespace moe {
namespace {

constexpr int kThreads = 512;
constexpr int kGroup = 16;  // rows of a matrix instruction
constexpr int kRows = 256;
constexpr int kCols = 256;  // weight rows of a tile

// A K block in LDS, for waves of up to kJ 16-row groups.
template <int kJ>
struct Stage {
  static constexpr int kRows = 2 * kJ * kGroup;
  uint8_t x[kRows * 128];
  uint8_t w[kCols * 128];
  uint32_t xs[kRows < 64 ? 64 : kRows];  // FP32 scales, or four E8M0 bytes
};
// Blocks in LDS: one read, the others on their way.
template <int kJ>
constexpr int kStages = kJ <= 4 ? 3 : 2;
constexpr size_t kShared = kStages<4> * sizeof(Stage<4>);
static_assert(kStages<8> * sizeof(Stage<8>) <= kShared && kShared <= 160 * 1024, "all forms fit");

__device__ __forceinline__ int8v_t read_operand(const uint8_t* p, int lo, int hi) {
  const u32x4_t a = *reinterpret_cast<const u32x4_t*>(p + lo), b = *reinterpret_cast<const u32x4_t*>(p + hi);
  return int8v_t{(int)a[0], (int)a[1], (int)a[2], (int)a[3], (int)b[0], (int)b[1], (int)b[2], (int)b[3]};
}

// A 16 x 16 product of one block: lane 16 g + r gives bytes 16 g .. 16 g + 15
// and 64 + 16 g .. of weight row r and of activation row r, and gets activation
// row r by weight rows 4 g .. 4 g + 3. kMx: the instruction applies the
// activations' E8M0 scales; lane 16 g + r gives that of positions 32 g .. of
// row r.
template <bool kMx>
__device__ __forceinline__ float4_t product(const int8v_t& w, const int8v_t& x, int e8m0) {
  const float4_t zero = {0.f, 0.f, 0.f, 0.f};
  if (kMx) return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(w, x, zero, 0, 0, 0, 127, 0, e8m0);
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(w, x, zero, 0, 0, 0, 0, 0, 0);
}

// kJ: the most 16-row groups of a wave; `first`: those of the first four waves.
template <bool kMx, bool kWhole, int kJ>
__device__ __forceinline__ void tile(const GroupedArgs& a, const TileAt& at, uint8_t* shared, int groups) {
  Stage<kJ>* const sm = reinterpret_cast<Stage<kJ>*>(shared);
  constexpr int kHalf = kJ * kGroup;  // LDS rows of a half of the waves
  const int tid = threadIdx.x, lane = tid & (kWave - 1);
  const int wave = __builtin_amdgcn_readfirstlane(tid / kWave);
  const int r16 = lane & 15, g = lane >> 4;
  const int wn = wave & 3, wm = wave >> 2;
  const int first = (groups + 1) / 2, tile_col = kWhole ? at.col : at.col / a.splits;
  const KPart part = k_part<kWhole>(a, at, kRows);
  const int KB = part.blocks;

  // What this wave copies of a block: 32 LDS rows of the weights, 4 kJ of the
  // activations (8 for kJ = 1, the same ones by two waves), 64 scales (the same ones by several waves, so that every
  // wave has as many copies on its way). LDS row L keeps 16-byte chunk c of
  // its row at place c ^ (L / 2 % 8), so that the 16 rows of a read phase
  // differ in bank. A lane's results of instructions s = 0, 1 (2, 3) of a
  // block and group are eight neighbouring columns and those of a row's four
  // lanes 32: instruction s has weight rows r of columns 32 (s / 2) +
  // 8 (r / 4) + 4 (s % 2) + r % 4.
  constexpr int kXCopies = (kJ + 1) / 2, kCopies = 4 + kXCopies + 1;
  static_assert(kJ == 1 || kJ % 2 == 0, "whole copies of eight rows for each of eight waves (kJ = 1: for four)");
  const int wx = kJ == 1 ? wave & 3 : wave * kXCopies;  // in eights of LDS rows
  const int lr = lane >> 3;
  const auto x_of = [&](int L) {  // activation row of LDS row L
    const int m = L % kHalf + L / kHalf * kGroup * first;
    return (size_t)max(x_row(a, min(at.row + m, at.end - 1)), 0);
  };
  const uint8_t* xp[kXCopies];
#pragma unroll
  for (int i = 0; i < kXCopies; ++i) {
    const int L = (wx + i) * 8 + lr;
    xp[i] = a.x + x_of(L) * a.K + (size_t)part.first * 128 + ((lane & 7) ^ ((L >> 1) & 7)) * 16;
  }
  // its weight rows: 32 of the 64 columns of one wave; eight i begins at column
  // 16 (i % 2) + 4 (i / 2) and, where i is odd, at the other half's chunks
  const int col = min(tile_col * kCols + (wave >> 1) * 64, a.N - 64) + (wave & 1) * 32;
  const uint8_t* wp = a.w + ((size_t)at.e * a.N + col) * a.K + (size_t)part.first * 128;
  const uint32_t wrow = (uint32_t)((lr >> 2) * 8 + (lr & 3)) * (uint32_t)a.K, chunk = ((lane & 7) ^ (lr >> 1)) * 16;
  const uint32_t woff[2] = {wrow + chunk, wrow + (chunk ^ 64)};
  const int sl = wave % kXCopies * 64;
  const uint8_t* sp = static_cast<const uint8_t*>(a.xs) + (x_of(sl + lane) * (a.K / 128) + part.first) * 4;
  const uint32_t lds = lds_offset(shared);
  constexpr int kWCopies = 4;
  const auto issue_w = [&](int st, int b) {
    const int kb = part.at<kWhole>(b);
    const uint32_t to = lds + st * (uint32_t)sizeof(Stage<kJ>);
    const size_t k0 = (size_t)kb * 128;
    const auto all = [&](auto once) {
#pragma unroll
      for (int i = 0; i < kWCopies; ++i)
        copy16_to_lds<decltype(once)::value>(wp + k0 + (size_t)((i & 1) * 16 + (i >> 1) * 4) * a.K, woff[i & 1],
                                             to + (uint32_t)offsetof(Stage<kJ>, w) + (wave * 32 + i * 8) * 128);
    };
    if (at.only)
      all(std::true_type{});
    else
      all(std::false_type{});
  };
  const auto issue_x = [&](int st, int b) {
    const int kb = part.at<kWhole>(b);
    const uint32_t to = lds + st * (uint32_t)sizeof(Stage<kJ>);
#pragma unroll
    for (int i = 0; i < kXCopies; ++i) copy16_to_lds(xp[i] + (size_t)kb * 128, to + (wx + i) * 1024);
    copy4_to_lds(sp + (size_t)kb * 4, to + (uint32_t)offsetof(Stage<kJ>, xs) + sl * 4);
  };

  const int n0 = tile_col * kCols + wn * 64;
  const uniform_floats sw = as_uniform(a.ws) + ((size_t)at.e * (a.N / 128) + min(n0, a.N - 1) / 128) * (a.K / 128) + part.first;
  const int swz = (g ^ (r16 >> 1)) * 16;
  const int w_lo = (wn * 64 + r16) * 128 + swz, x_lo = (wm * kHalf + r16) * 128 + swz;

  float4_t acc[kJ][4];
#pragma unroll
  for (int j = 0; j < kJ; ++j)
#pragma unroll
    for (int s = 0; s < 4; ++s) acc[j][s] = float4_t{0.f, 0.f, 0.f, 0.f};

  // The copies of blocks b .. b + kStages - 1 go on while block b is worked on:
  // its weights are in registers from its beginning on, so their place is
  // filled anew at once; its activations' place when they have all been read.
#pragma unroll
  for (int b = 0; b < kStages<kJ>; ++b)
    if (b < KB) {
      issue_w(b, b);
      issue_x(b, b);
    }
  if (kStages<kJ> - 1 < KB)
    copies_left<(kStages<kJ> - 1) * kCopies>(shared);
  else
    copies_left<0>(shared);
  workgroup_barrier();

  int8v_t w[4], x[2];
  uint32_t sx[2];
  const auto load_w = [&](int st) {
#pragma unroll
    for (int s = 0; s < 4; ++s) w[s] = read_operand(sm[st].w + s * 2048, w_lo, w_lo ^ 64);
  };
  const auto load_x = [&](int st, int j) {
    x[j & 1] = read_operand(sm[st].x + j * 2048, x_lo, x_lo ^ 64);
    sx[j & 1] = sm[st].xs[wm * kHalf + j * 16 + r16];
  };
  float4_t p[2][4];
  float sc[2];
  const auto multiply = [&](int j, float s0) {
    sc[j & 1] = kMx ? s0 : __uint_as_float(sx[j & 1]) * s0;
#pragma unroll
    for (int s = 0; s < 4; ++s) p[j & 1][s] = product<kMx>(w[s], x[j & 1], (int)((sx[j & 1] >> (8 * g)) & 0xFFu));
  };
  const auto add = [&](int j) {
#pragma unroll
    for (int s = 0; s < 4; ++s) {
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[j][s][i] = fmaf(p[j & 1][s][i], sc[j & 1], acc[j][s][i]);
      asm volatile("" : "+v"(acc[j][s]));  // here, not behind the loop's body, where every p would have to live until then
    }
  };
  load_w(0);
  load_x(0, 0);
  int st = 0;
  for (int b = 0; b < KB; ++b) {
    const float s0 = sw[part.at<kWhole>(b)];
    if (b + kStages<kJ> < KB) {
      asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
      workgroup_barrier();  // every wave has read the block's weights
      issue_w(st, b + kStages<kJ>);
    }
    // a group's scaled sums are added while the next group's instructions
    // run; the fences keep the compiler from loading further ahead than the
    // registers reach
#pragma unroll
    for (int j = 0; j + 1 < kJ; ++j) {
      load_x(st, j + 1);
      multiply(j, s0);
      if (j) add(j - 1);
      __builtin_amdgcn_sched_barrier(0);
    }
    if (b + 1 < KB) {
      // the next block is there, in every wave, and every wave has read all of this one
      if (b + kStages<kJ> < KB)
        copies_left<(kStages<kJ> - 2) * kCopies + kWCopies>(shared);
      else
        copies_left<0>(shared);
      workgroup_barrier();
      if (b + kStages<kJ> < KB) issue_x(st, b + kStages<kJ>);
    }
    multiply(kJ - 1, s0);
    if (kJ > 1) add(kJ - 2);
    __builtin_amdgcn_sched_barrier(0);
    st = st == kStages<kJ> - 1 ? 0 : st + 1;
    if (b + 1 < KB) {
      load_w(st);
      load_x(st, 0);
    }
    add(kJ - 1);
  }

  if (n0 >= a.N) return;
#pragma unroll
  for (int j = 0; j < kJ; ++j) {
    const int i = at.row + (wm * first + j) * kGroup + r16;
    if (j < (wm ? groups - first : first) && i < at.end) {
      if (!kWhole && a.splits > 1) {
        float* o = a.partial + ((size_t)part.split * a.R + i) * a.N + n0 + g * 8;
#pragma unroll
        for (int s = 0; s < 4; ++s) *reinterpret_cast<float4_t*>(o + 32 * (s >> 1) + 4 * (s & 1)) = acc[j][s];
        continue;
      }
      const bool none = x_row(a, i) < 0;
      uint16_t* o = static_cast<uint16_t*>(a.out) + (size_t)i * a.N + n0 + g * 8;
#pragma unroll
      for (int s = 0; s < 4; s += 2) {
        const float4_t u = acc[j][s], v = acc[j][s + 1];
        u32x4_t q = {bf16x2_bits(u[0], u[1]), bf16x2_bits(u[2], u[3]), bf16x2_bits(v[0], v[1]), bf16x2_bits(v[2], v[3])};
        if (none) q = u32x4_t{0u, 0u, 0u, 0u};
        *reinterpret_cast<u32x4_t*>(o + 16 * s) = q;
      }
    }
  }
}

template <bool kMx, bool kWhole>
__device__ __forceinline__ void any_tile(const GroupedArgs& a, const TileAt& at, uint8_t* shared) {
  const int groups = (at.end - at.row + kGroup - 1) / kGroup;
  const int need = (groups + 1) / 2;  // of the first half of the waves; the other half has the rest
  if (need > 6)
    tile<kMx, kWhole, 8>(a, at, shared, groups);
  else if (need > 4)
    tile<kMx, kWhole, 6>(a, at, shared, groups);
  else if (need > 2)
    tile<kMx, kWhole, 4>(a, at, shared, groups);
  else if (need > 1)
    tile<kMx, kWhole, 2>(a, at, shared, groups);
  else
    tile<kMx, kWhole, 1>(a, at, shared, groups);
}

template <bool kMx>
__global__ __launch_bounds__(kThreads, 2) void grouped_product_fp8_kernel(GroupedArgs a) {
  __shared__ alignas(16) uint8_t shared[kShared];
  const TileAt at = find_tile<kRows, kGroup, kThreads>(a, blockIdx.x);
  if (at.e < 0) return;
  if (whole_k(a, at, kRows))
    any_tile<kMx, true>(a, at, shared);
  else
    any_tile<kMx, false>(a, at, shared);
}

}  // namespace

void launch_grouped_product_fp8(bool mx, GroupedArgs a, hipStream_t stream) {
  a.col_tiles = (a.N + kCols - 1) / kCols * a.splits;
  const auto kernel = mx ? grouped_product_fp8_kernel<true> : grouped_product_fp8_kernel<false>;
  hipLaunchKernelGGL(kernel, dim3(grouped_workgroups(a, a.R, kRows)), dim3(kThreads), 0, stream, a);
}

}  // namespace moe

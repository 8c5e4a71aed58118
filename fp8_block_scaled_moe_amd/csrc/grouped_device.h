// Device pieces shared by the grouped products (moe_rows.h): which rows a
// workgroup has, where an activation row lies, and the block product.
#pragma once

#include "rows_device.h"

namespace moe {

struct GroupedArgs {
  const uint8_t* x;
  const void* xs;
  const int32_t* rows;
  const int32_t* offsets;
  const uint8_t* w;
  const float* ws;
  void* out;
  float* outs;
  int R, X, E, N, K;
  float limit;
  int splits;      // parts of K, one per workgroup
  float* partial;  // [splits][R][N] FP32 sums over a part of K each, where splits > 1
  int col_tiles;   // column tiles of an expert's output times `splits`
};

constexpr int kTileRows = 128;  // of a tile with FP32 sums, at most

// Parts of K for so few tiles (of up to 128 rows by 256 weight rows) that
// they leave CUs idle: as many as give every CU a part, of four 128-wide blocks
// and more, from 16 blocks on (below, the second launch costs what it saves). See
// grouped_gemm.hip.
inline int grouped_splits(int R, int E, int N, int K) {
  const int64_t full = (int64_t)R / kTileRows + E, tiles = (full < R ? full : R) * ((N + 255) / 256);
  const int64_t most = K / 128 / 4, wanted = tiles > 0 ? 256 / tiles : 1;
  return (int)(wanted < 2 || most < 4 ? 1 : wanted < most ? wanted : most);
}

// Workgroups that find_tile's tiles need at most for R grouped rows (each
// expert's rows rounded up, no tile without a row), a multiple of the XCDs.
__host__ __device__ inline unsigned grouped_workgroups(const GroupedArgs& a, int R, int rows) {
  const int64_t full = (int64_t)R / rows + a.E, tiles = (full < R ? full : R) * a.col_tiles;
  return (unsigned)((tiles + 7) / 8 * 8);
}

// Read-only data at addresses that are the same for the whole wave, through
// the scalar cache (loads that the vector memory counter does not wait for).
typedef const __attribute__((address_space(4))) float* uniform_floats;
typedef const __attribute__((address_space(4))) int32_t* uniform_ints;
__device__ __forceinline__ uniform_floats as_uniform(const float* p) { return (uniform_floats)(uintptr_t)p; }
__device__ __forceinline__ uniform_ints as_uniform(const int32_t* p) { return (uniform_ints)(uintptr_t)p; }

void launch_grouped_product(bool mx, GroupedArgs a, hipStream_t stream);      // grouped_product.hip
void launch_grouped_product_fp8(bool mx, GroupedArgs a, hipStream_t stream);  // grouped_product_fp8.hip
void launch_grouped_swiglu(bool mx, GroupedArgs a, hipStream_t stream);       // grouped_swiglu.hip

// A workgroup's tile: grouped rows [row, end) of expert e, column tile and
// part of K `col`;
// only: these are all of the expert's rows, so nobody else reads the tile's
// weights. e < 0: no tile is left for it.
struct TileAt {
  int e, row, end, col, only;
};

// A workgroup's part of K, in 128-wide blocks, and the block of it that the
// workgroup begins with (at() wraps round). A tile with all of K from its beginning
// on (whole_k) has code of its own: the others' costs it 2%.
//
// Where K is a multiple of 4096, the blocks of one index of all rows lie in few
// memory channels, so tiles with weights of their own (an expert's only row tile)
// begin at different blocks. Measured with N = 2048, without and with it: 16 rows
// for each of 32 experts, K = 4096 61 and 43 us, 8192 115 and 80, 12288 160 and 119,
// 16384 162 and 158; of 64, 120 and 84, 164 and 164, 285 and 243, 323 and 321; of
// 128, 171 and 174, 331 and 331, 504 and 487; of 15 with K split, 27 and 28, 57 and
// 45, 66 and 63, 102 and 80. Where K is another multiple of 1024 it costs up to 14%
// and gains 3 at most (K = 2048, 23 and 26 us; 6144, 64 and 62; 7168, 71 and 72;
// 10240, 101 and 102). With FP32 sums it pays up to 64 rows in a tile (32 experts:
// 64 rows, K = 4096 64 and 58 us, 8192 122 and 112; 48 or 64 experts, 8192, up to 9%
// the other way) and costs 1 to 5% beyond (100 rows, 8192: 157 and 160), where the
// matrix instructions bind; the FP8 instruction's tiles gain at any height (100
// rows, K = 8192: 123 and 101 us; 64 experts of 100 rows lose 7%).
struct KPart {
  int split, first, blocks, start;
  template <bool kWhole>
  __device__ __forceinline__ int at(int b) const {
    return kWhole ? b : b + start - (b + start >= blocks ? blocks : 0);
  }
};
__device__ __forceinline__ bool turned(const GroupedArgs& a, const TileAt& at, int most_rows) {
  return at.only && a.K % 4096 == 0 && at.end - at.row <= most_rows;
}
__device__ __forceinline__ bool whole_k(const GroupedArgs& a, const TileAt& at, int most_rows) {
  return a.splits == 1 && !turned(a, at, most_rows);
}
// True of every tile: such calls have kernels of their own, since with the other
// tiles' code beside it the SwiGLU's (8,192 tokens x 8 of 256, K = 7168) took 4.62 ms
// where it takes 4.58.
inline bool all_of_k(const GroupedArgs& a) { return a.splits == 1 && a.K % 4096 != 0; }
template <bool kWhole>
__device__ __forceinline__ KPart k_part(const GroupedArgs& a, const TileAt& at, int most_rows) {
  if (kWhole) return KPart{0, 0, a.K / 128, 0};
  const int KB = a.K / 128, split = at.col % a.splits;
  const int lo = KB * split / a.splits, n = KB * (split + 1) / a.splits - lo;
  int start = 0;
  if (turned(a, at, most_rows)) start = (at.e * (a.col_tiles / a.splits) + at.col / a.splits) % n;
  return KPart{split, lo, n, start};
}

// The workgroup's tile when every expert's rows are cut into as few tiles of
// at most kRows (a multiple of kGroup) as can be, even but for kGroup rows.
// The row tiles are counted anew by every workgroup (offsets are on the
// device; E + 1 of them from L2 and one sum over the workgroup, about 1 us).
// Tiles are numbered expert by expert, inside an expert column tile by column
// tile, the expert's row tiles fastest, so that neighbours share weights; and
// each XCD (workgroup id mod 8) takes a contiguous eighth of the numbers, so
// that what neighbours share meets in one L2. Every thread calls it; barriers
// inside.
template <int kRows, int kGroup, int kThreadsWg>
__device__ __forceinline__ TileAt find_tile(const GroupedArgs& a, int block) {
  constexpr int kWavesWg = kThreadsWg / kWave;
  constexpr int kPer = 1024 / kThreadsWg;  // experts per thread: E <= 1024
  static_assert(kPer >= 1, "every expert has a thread");
  __shared__ int wave_sum[kWavesWg];
  __shared__ int found[5];
  // R may be far more than the rows that are there (one GPU's share of the
  // experts): workgroups that these cannot need leave at once
  if ((unsigned)block >= grouped_workgroups(a, min(max(as_uniform(a.offsets)[a.E], 0), a.R), kRows))
    return TileAt{-1, 0, 0, 0, 0};
  const int tid = threadIdx.x, lane = tid & (kWave - 1), wave = tid / kWave;
  const int per = (a.E + kThreadsWg - 1) / kThreadsWg;
  const auto clamped = [&](int e) { return min(max(a.offsets[min(e, a.E)], 0), a.R); };
  int lo[kPer], tiles[kPer], sum = 0;
#pragma unroll
  for (int q = 0; q < kPer; ++q) {
    const int e = tid * per + q;
    lo[q] = tiles[q] = 0;
    if (q < per && e < a.E) {
      lo[q] = clamped(e);
      tiles[q] = (max(clamped(e + 1) - lo[q], 0) + kRows - 1) / kRows;
    }
    sum += tiles[q];
  }
  int incl = sum;
#pragma unroll
  for (int o = 1; o < kWave; o <<= 1) {
    const int up = __shfl_up(incl, o, kWave);
    incl += lane >= o ? up : 0;
  }
  if (lane == kWave - 1) wave_sum[wave] = incl;
  if (tid == 0) found[0] = -1;
  __syncthreads();
  int before = incl - sum, total = 0;
#pragma unroll
  for (int w = 0; w < kWavesWg; ++w) {
    before += w < wave ? wave_sum[w] : 0;
    total += wave_sum[w];
  }
  const int64_t all = (int64_t)total * a.col_tiles;
  const int64_t share = (all + 7) / 8;
  const int64_t at = (int64_t)(block & 7) * share + (block >> 3);
  if ((block >> 3) < share && at < all) {
    const int t = (int)(at / a.col_tiles);  // lies in its expert's range of row tiles
#pragma unroll
    for (int q = 0; q < kPer; ++q) {
      if (t >= before && t < before + tiles[q]) {
        const int mine = (int)(at - (int64_t)before * a.col_tiles);
        found[0] = tid * per + q;
        // the expert's groups of kGroup rows, evenly over its tiles
        const int end = clamped(tid * per + q + 1), i = mine % tiles[q];
        const int groups = (end - lo[q] + kGroup - 1) / kGroup;
        found[1] = lo[q] + kGroup * (int)((int64_t)groups * i / tiles[q]);
        found[2] = min(lo[q] + kGroup * (int)((int64_t)groups * (i + 1) / tiles[q]), end);
        found[3] = mine / tiles[q];
        found[4] = tiles[q] == 1;
      }
      before += tiles[q];
    }
  }
  __syncthreads();
  TileAt r;
  r.e = __builtin_amdgcn_readfirstlane(found[0]);
  r.row = __builtin_amdgcn_readfirstlane(found[1]);
  r.end = __builtin_amdgcn_readfirstlane(found[2]);
  r.col = __builtin_amdgcn_readfirstlane(found[3]);
  r.only = __builtin_amdgcn_readfirstlane(found[4]);
  return r;
}

// The activation row of grouped row i, -1 where its index is out of range.
__device__ __forceinline__ int x_row(const GroupedArgs& a, int i) {
  const int r = a.rows ? a.rows[i] : i;
  return r >= 0 && r < a.X ? r : -1;
}

// Copies from memory straight into LDS: lane l's 16 (or 4) bytes go to byte
// 16 l (4 l) behind `to`, the same for the whole wave. In assembly, since the
// compiler waits for its own form of them before every later read of LDS,
// whichever buffer it reads; no register is written but M0, and copies_left()
// waits until at most n of the wave's are on their way (they end in order). A
// workgroup barrier behind it makes all waves' copies visible.
__device__ __forceinline__ uint32_t lds_offset(const void* p) {
  return (uint32_t)(uintptr_t)(const __attribute__((address_space(3))) char*)p;
}
__device__ __forceinline__ uint32_t uniform(uint32_t v) { return (uint32_t)__builtin_amdgcn_readfirstlane((int)v); }
__device__ __forceinline__ const uint8_t* uniform(const uint8_t* p) {
  const uint64_t v = reinterpret_cast<uint64_t>(p);
  return reinterpret_cast<const uint8_t*>(((uint64_t)uniform((uint32_t)(v >> 32)) << 32) | uniform((uint32_t)v));
}
// M0 is reserved from the allocator, of which the compiler warns; named, the
// statements keep their place among its own uses of it.
#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"
__device__ __forceinline__ void copy16_to_lds(const uint8_t* from, uint32_t to) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, off" ::"s"(uniform(to)), "v"(from) : "m0");
}
__device__ __forceinline__ void copy4_to_lds(const uint8_t* from, uint32_t to) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dword %1, off" ::"s"(uniform(to)), "v"(from) : "m0");
}
// The same from a uniform address plus the lane's offset. kOnce: with the
// non-temporal hint, for data that is read once: weights of an expert's only
// row tile (16 rows for each of 64 experts of 4096 x 7168, 288 us with it and
// 318 without; where row tiles share them it costs: 65,536 rows over 256 such
// experts, 4.92 ms with it and 4.69 without).
template <bool kOnce>
__device__ __forceinline__ void copy16_to_lds(const uint8_t* base, uint32_t offset, uint32_t to) {
  if (kOnce)
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, %2 nt" ::"s"(uniform(to)), "v"(offset),
                 "s"(uniform(base)) : "m0");
  else
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, %2" ::"s"(uniform(to)), "v"(offset),
                 "s"(uniform(base)) : "m0");
}
#pragma clang diagnostic pop
// At most kLeft copies are left, and all reads of LDS have returned.
template <int kLeft>
__device__ __forceinline__ void copies_left(const void* lds) {
  asm volatile("s_waitcnt vmcnt(%1) lgkmcnt(0)" ::"v"(lds), "n"(kLeft) : "memory");
}
__device__ __forceinline__ void workgroup_barrier() {
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));

// Eight e4m3 codes as BF16 values times a power of two: exact, down to 2^-117.
__device__ __forceinline__ bf16x8_t widen8_scaled(uint32_t w0, uint32_t w1, float scale) {
  const bf16x2_t a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w0, scale, false);
  const bf16x2_t b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w0, scale, true);
  const bf16x2_t c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w1, scale, false);
  const bf16x2_t d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w1, scale, true);
  return bf16x8_t{a.x, a.y, b.x, b.y, c.x, c.y, d.x, d.y};
}

// 2^(byte - 127) of E8M0 byte c of a row's four of a block (32 positions each).
__device__ __forceinline__ int e8m0_byte(uint32_t bytes, int c) { return (int)((bytes >> (8 * c)) & 0xFFu); }
__device__ __forceinline__ float e8m0_value(int byte) { return __uint_as_float(byte ? (uint32_t)byte << 23 : 0x400000u); }

// MXFP8 scales of a row's block: the largest as the block's own scale, the four
// relative to it, so that no product is larger than FP32's range allows while
// its result is not. A product of two codes is a multiple of 2^-18, so down to a
// relative scale of 2^-96 every operand is a normal BF16 value and no bit of a
// product falls out of FP32; and a scale of 2^63 times w_scale is finite up to
// 2^64. Beyond either (`far`), each 32 positions are to be summed and scaled by
// themselves (scale_apart); the relative scales and the block's own are 1 and 0 then.
constexpr int kMxApart = 96, kMxTop = 127 + 63;
__device__ __forceinline__ float mx_scales(uint32_t bytes, float (&rel)[4], bool& far) {
  int top = 0, bottom = 255;
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    top = max(top, e8m0_byte(bytes, c));
    bottom = min(bottom, e8m0_byte(bytes, c));
  }
  far = top - bottom > kMxApart || top > kMxTop;
#pragma unroll
  for (int c = 0; c < 4; ++c) rel[c] = far ? 1.f : __uint_as_float((uint32_t)(127 + e8m0_byte(bytes, c) - top) << 23);
  return far ? 0.f : e8m0_value(top);
}

// s * 2^(byte - 127) in two factors, the second 2^up with up >= 0, so that the
// first is finite and a sum scaled by both is what it would be without FP32's
// limits.
__device__ __forceinline__ float scale_apart(float s, int byte, int& up) {
  const int e = (int)((__float_as_uint(s) >> 23) & 0xFFu) - 127;
  up = max(byte - 127 + e - 126, 0);
  return ldexpf(s, byte - 127 - up);
}

// gate / (1 + exp(-gate)) * up with both clamped; a NaN stays one (the median
// instruction would not keep it). The exponential by the hardware's exp2 of
// t = -gate log2 e, with what the rounding of t leaves of -gate made up for to
// first order, so that its error hardly grows with |gate| (by a unit of 2^-23 for
// 42 of it, that of ln 2); below -87 a gate counts as -87, whose SiLU is 2^-119.
__device__ __forceinline__ float clamp_nan(float v, float lo, float hi) {
  return __builtin_elementwise_minimum(__builtin_elementwise_maximum(v, lo), hi);
}

__device__ __forceinline__ float swiglu(float up, float gate, float limit) {
  constexpr float kLog2e = 0x1.715476p+0f, kLn2 = 0x1.62e43p-1f;
  up = clamp_nan(up, -limit, limit);
  gate = clamp_nan(gate, -87.f, limit);
  const float t = gate * -kLog2e, e = __builtin_amdgcn_exp2f(t);
  return gate * __builtin_amdgcn_rcpf(fmaf(e, fmaf(t, -kLn2, -gate), 1.f + e)) * up;
}

}  // namespace moe

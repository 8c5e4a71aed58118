// The tile of the grouped products with FP32 sums (grouped_swiglu.hip,
// grouped_product.hip): up to 128 rows of an expert by 256 weight rows per
// workgroup.
//
// Every 128-wide K block of the tile's activations and weights is copied into
// LDS (up to 48 KB, three blocks at a time), read from there by eight waves, 64
// rows by 64 weight rows each (SwiGLU: 32 up and 32 gate), widened to BF16
// (exact) and multiplied by the 32x32x16 instruction; the block's FP32 sums are
// multiplied by its scales when they are added. BF16 and not the FP8
// instruction, which adds eight products at a time cut off 14 bits below the
// power of two of the largest (measured; 2^-16 of a result on average, and
// products that cancel leave nothing of small ones beside them). F16 is as exact
// (both keep 23 bits below the largest), but a hundredth slower (4.61 and 4.56 ms
// for the SwiGLU of 65,536 rows over 256 experts, K = 7168, I = 2048) and too
// narrow for MXFP8 scales that lie 2^15 and more apart.
// The two halves of the waves share the tile's 32-row groups evenly, a SIMD has
// one wave of each, and row tiles of an expert are alike in size.
#pragma once

#include <type_traits>

#include "grouped_device.h"

namespace moe {

constexpr int kThreads = 512;
constexpr int kGroup = 32;  // rows of a matrix instruction
constexpr int kRows = kTileRows;
constexpr int kTurnRows = 64;  // see KPart
constexpr int kStages = 3;  // K blocks in LDS: one read, the others on their way

// A K block in LDS, for waves of up to kFirst 32-row groups.
template <int kFirst>
struct Stage {
  uint8_t x[2 * kFirst * kGroup * 128];
  uint8_t w[256 * 128];
  uint32_t xs[2 * kFirst * kGroup];  // FP32 scales, or four E8M0 bytes
};
struct Shared {
  alignas(16) uint8_t st[kStages * sizeof(Stage<2>)];
  float amax[4][kRows];
};

typedef float float16_t __attribute__((ext_vector_type(16)));

// Sixteen codes of a row in BF16, two instructions' worth.
struct Wide16 {
  bf16x8_t v[2];
};
__device__ __forceinline__ Wide16 widen16(const u32x4_t& q, float scale) {
  return Wide16{{widen8_scaled(q[0], q[1], scale), widen8_scaled(q[2], q[3], scale)}};
}

// kGlu: the SwiGLU of 128 hidden columns; else the product of 256 columns.
// kJ: the 32-row groups of this wave; kFirst: those of the first four waves.
template <bool kGlu, bool kMx, bool kWhole, int kFirst, int kJ>
__device__ __forceinline__ void tile(const GroupedArgs& a, const TileAt& at, Shared& sm) {
  constexpr int kHalf = kFirst * kGroup;  // LDS rows of a half of the waves
  const Stage<kFirst>* const stage = reinterpret_cast<const Stage<kFirst>*>(sm.st);
  constexpr int kN = kJ ? kJ : 1;
  const int tid = threadIdx.x, lane = tid & (kWave - 1);
  const int wave = __builtin_amdgcn_readfirstlane(tid / kWave);
  const int r32 = lane & 31, h = lane >> 5;
  const int wn = wave & 3, wm = wave >> 2;
  const int I = a.N / 2, tile_col = kWhole ? at.col : at.col / a.splits;
  const KPart part = k_part<kWhole>(a, at, kTurnRows);
  const int KB = part.blocks;

  // What this wave copies of a block: 32 LDS rows of the weights, 8 kFirst
  // of the activations and 64 scales (the same ones by several waves, so that
  // every wave has as many copies on its way). LDS row L keeps 16-byte chunk c of its
  // row at place c ^ (L / 2 % 8), so that the 16 rows of a read phase differ in
  // bank. A lane's results of an instruction are weight rows 8 a + 4 h + b (a,
  // b = 0..3) of its 32. SwiGLU: these are columns 16 h + 4 a + b, so that a
  // lane's 16 codes are neighbours. Product: 16 (a / 2) + 8 h + 4 (a % 2) + b,
  // so that eight values of a lane are, and those of a row's two lanes.
  constexpr int kXCopies = kFirst, kCopies = 4 + kXCopies + 1;
  const int lr = lane >> 3;
  const auto x_of = [&](int L) {  // activation row of LDS row L
    return (size_t)max(x_row(a, min(at.row + L, at.end - 1)), 0);
  };
  const uint8_t* xp[kXCopies];
#pragma unroll
  for (int i = 0; i < kXCopies; ++i) {
    const int L = (wave * kXCopies + i) * 8 + lr;
    xp[i] = a.x + x_of(L) * a.K + (size_t)part.first * 128 + ((lane & 7) ^ ((L >> 1) & 7)) * 16;
  }
  // SwiGLU: up rows for even waves, the same columns' gate rows for odd ones.
  // Its eight LDS rows i (a = i) are at the other half's chunks where i is odd.
  const int wfirst = kGlu ? tile_col * 128 + (wave >> 1) * 32 + (wave & 1) * I : min(tile_col * 256 + wave * 32, a.N - 32);
  const uint8_t* wp = a.w + ((size_t)at.e * a.N + wfirst) * a.K + (size_t)part.first * 128;
  const uint32_t wrow = (uint32_t)((lr >> 2) * (kGlu ? 16 : 8) + (lr & 3)) * (uint32_t)a.K, chunk = ((lane & 7) ^ (lr >> 1)) * 16;
  const uint32_t woff[2] = {wrow + chunk, wrow + (chunk ^ 64)};
  const int sl = wave % kFirst * 64;  // its first scale
  const uint8_t* sp = static_cast<const uint8_t*>(a.xs) + (x_of(sl + lane) * (a.K / 128) + part.first) * 4;
  const uint32_t lds = lds_offset(sm.st);
  const auto issue = [&](int st, int b) {
    const int kb = part.at<kWhole>(b);
    const uint32_t to = lds + st * (uint32_t)sizeof(Stage<kFirst>);
    const size_t k0 = (size_t)kb * 128;
    const auto weights = [&](auto once) {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        copy16_to_lds<decltype(once)::value>(wp + k0 + (size_t)(kGlu ? 4 * i : 16 * (i >> 1) + 4 * (i & 1)) * a.K, woff[i & 1],
                                             to + (uint32_t)offsetof(Stage<kFirst>, w) + (wave * 32 + i * 8) * 128);
    };
    if (at.only)
      weights(std::true_type{});
    else
      weights(std::false_type{});
#pragma unroll
    for (int i = 0; i < kXCopies; ++i) copy16_to_lds(xp[i] + k0, to + (wave * kXCopies + i) * 1024);
    copy4_to_lds(sp + (size_t)kb * 4, to + (uint32_t)offsetof(Stage<kFirst>, xs) + sl * 4);
  };

  const int n0 = tile_col * 256 + wn * 64;  // product: the wave's first column; it has none from N on
  const uniform_floats su =
      as_uniform(a.ws) + ((size_t)at.e * (a.N / 128) + (kGlu ? tile_col : min(n0, a.N - 1) / 128)) * (a.K / 128) + part.first;
  const uniform_floats sg = kGlu ? su + (size_t)(I / 128) * (a.K / 128) : su;

  // Sixteen bytes of every row (chunk h + 2 c of the lane's row) at a time,
  // widened while the matrix instructions of the chunk before run. Of a
  // wave's two products [t], 0 is up and 1 gate (product: 32 columns each).
  const float16_t zero = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  int off[4];
#pragma unroll
  for (int c = 0; c < 4; ++c) off[c] = r32 * 128 + (((h + 2 * c) ^ (r32 >> 1)) & 7) * 16;
  Wide16 w[2][2], x[2][kN];  // [chunk parity]
  float rel[kN][4], xs[kN];
  uint32_t sx[kN];                     // MXFP8: the four scales of the lane's row,
  bool far[kN] = {}, any_far = false;  // whether they lie far apart, and whether those of any row of the wave do
  float16_t acc[kN][2], p[kN][2];
#pragma unroll
  for (int j = 0; j < kJ; ++j) acc[j][0] = acc[j][1] = zero;
  const auto scales = [&](int st) {
    bool f = false;
#pragma unroll
    for (int j = 0; j < kJ; ++j) {
      sx[j] = stage[st].xs[wm * kHalf + j * 32 + r32];
#pragma unroll
      for (int c = 0; c < 4; ++c) rel[j][c] = 1.f;
      xs[j] = kMx ? mx_scales(sx[j], rel[j], far[j]) : __uint_as_float(sx[j]);
      f |= far[j];
    }
    if (kMx) any_far = __ballot(f) != 0;
  };
  const auto load = [&](int st, int c) {
    if (!kJ) return;
    const uint8_t *wb = stage[st].w + wn * 64 * 128, *xb = stage[st].x + wm * kHalf * 128;
#pragma unroll
    for (int t = 0; t < 2; ++t) w[c & 1][t] = widen16(*reinterpret_cast<const u32x4_t*>(wb + t * 4096 + off[c]), 1.f);
#pragma unroll
    for (int j = 0; j < kJ; ++j)
      x[c & 1][j] = widen16(*reinterpret_cast<const u32x4_t*>(xb + j * 4096 + off[c]), rel[j][c]);
  };
  const auto multiply = [&](int c) {
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int j = 0; j < kJ; ++j)
#pragma unroll
        for (int t = 0; t < 2; ++t)
          p[j][t] =
              __builtin_amdgcn_mfma_f32_32x32x16_bf16(w[c & 1][t].v[i], x[c & 1][j].v[i], c || i ? p[j][t] : zero, 0, 0, 0);
  };
  // The block's products of rows whose scales lie far apart: each 32 positions (a
  // chunk c) summed and scaled by themselves. The block's own scale of such rows
  // is 0, so that the rest of the loop adds nothing to them; other rows are left
  // alone. Beside the loop's own body, not in it: four passes of the body over such
  // a block, with the other codes read as zeros, cost MXFP8 rows without any 7 to
  // 12%, where this costs 0 to 3 (8,192 tokens x 8 of 256, K = 7168: 5.00 -> 5.12 ms).
  const auto add_far = [&](int st, float s0, float s1) {
    const uint8_t *wb = stage[st].w + wn * 64 * 128, *xb = stage[st].x + wm * kHalf * 128;
#pragma unroll 1
    for (int c = 0; c < 4; ++c) {
      const int o = r32 * 128 + (((h + 2 * c) ^ (r32 >> 1)) & 7) * 16;
#pragma unroll
      for (int j = 0; j < kJ; ++j) {
        const Wide16 xc = widen16(*reinterpret_cast<const u32x4_t*>(xb + j * 4096 + o), 1.f);
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          const Wide16 wc = widen16(*reinterpret_cast<const u32x4_t*>(wb + t * 4096 + o), 1.f);
          float16_t q = __builtin_amdgcn_mfma_f32_32x32x16_bf16(wc.v[0], xc.v[0], zero, 0, 0, 0);
          q = __builtin_amdgcn_mfma_f32_32x32x16_bf16(wc.v[1], xc.v[1], q, 0, 0, 0);
          int up;
          const float f = scale_apart(t ? s1 : s0, e8m0_byte(sx[j], c), up);
#pragma unroll
          for (int i = 0; i < 16; ++i) acc[j][t][i] = far[j] ? fmaf(ldexpf(q[i], up), f, acc[j][t][i]) : acc[j][t][i];
        }
      }
    }
  };
  // Block b's copies have ended, in every wave, and every wave has read all
  // of the block before. The copies of kStages - 2 blocks behind may be on
  // their way.
  const auto ready = [&](int b) {
    if (b + kStages - 2 < KB)
      copies_left<(kStages - 2) * kCopies>(&sm);
    else
      copies_left<0>(&sm);
    workgroup_barrier();
  };

#pragma unroll
  for (int b = 0; b < kStages - 1; ++b)
    if (b < KB) issue(b, b);
  ready(0);
  if (kStages - 1 < KB) issue(kStages - 1, kStages - 1);
  scales(0);
  load(0, 0);
  int st = 0;
  for (int b = 0; b < KB; ++b) {
    const float s0 = su[part.at<kWhole>(b)], s1 = sg[part.at<kWhole>(b)];
    if (kMx && any_far) add_far(st, s0, s1);
    load(st, 1);
    multiply(0);
    load(st, 2);
    multiply(1);
    load(st, 3);
    multiply(2);
    float sc[kN][2];
#pragma unroll
    for (int j = 0; j < kJ; ++j) {
      sc[j][0] = xs[j] * s0;
      sc[j][1] = xs[j] * s1;
    }
    if (b + 1 < KB) {
      ready(b + 1);
      if (b + kStages < KB) issue(st, b + kStages);
      st = st == kStages - 1 ? 0 : st + 1;
      scales(st);
      load(st, 0);
    }
    multiply(3);
#pragma unroll
    for (int j = 0; j < kJ; ++j)
#pragma unroll
      for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int i = 0; i < 16; ++i) acc[j][t][i] = fmaf(p[j][t][i], sc[j][t], acc[j][t][i]);
  }

  if (!kGlu && n0 >= a.N) return;
  if (!kWhole && a.splits > 1) {
#pragma unroll
    for (int j = 0; j < kJ; ++j) {
      const int i = at.row + (wm * kFirst + j) * kGroup + r32;
      if (i < at.end) {
        float* o = a.partial + ((size_t)part.split * a.R + i) * a.N + (kGlu ? tile_col * 128 + wn * 32 + h * 16 : n0 + h * 8);
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
          for (int q = 0; q < 4; ++q)
            *reinterpret_cast<float4_t*>(o + (kGlu ? t * I + 4 * q : t * 32 + 16 * (q >> 1) + 4 * (q & 1))) =
                float4_t{acc[j][t][4 * q], acc[j][t][4 * q + 1], acc[j][t][4 * q + 2], acc[j][t][4 * q + 3]};
      }
    }
    return;
  }
  if (!kGlu) {
#pragma unroll
    for (int j = 0; j < kJ; ++j) {
      const int i = at.row + (wm * kFirst + j) * kGroup + r32;
      if (i < at.end) {
        const bool none = x_row(a, i) < 0;
        uint16_t* o = static_cast<uint16_t*>(a.out) + (size_t)i * a.N + n0 + h * 8;
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
          for (int q = 0; q < 2; ++q) {
            u32x4_t v;
#pragma unroll
            for (int p = 0; p < 4; ++p) v[p] = none ? 0u : bf16x2_bits(acc[j][t][8 * q + 2 * p], acc[j][t][8 * q + 2 * p + 1]);
            *reinterpret_cast<u32x4_t*>(o + t * 32 + q * 16) = v;
          }
      }
    }
    return;
  }

  // SwiGLU: a lane's 16 hidden values of a row, the row's maximum over the 128
  // columns (the row's other lane, then the four waves), the codes
#pragma unroll
  for (int j = 0; j < kJ; ++j) {
    float amax = kAmaxFloor;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const float v = swiglu(acc[j][0][i], acc[j][1][i], a.limit);
      acc[j][0][i] = v;
      amax = fmaxf(amax, fabsf(v));
    }
    amax = fmaxf(amax, __shfl_xor(amax, 32, kWave));
    if (h == 0) sm.amax[wn][wm * kHalf + j * 32 + r32] = amax;
  }
  __syncthreads();
#pragma unroll
  for (int j = 0; j < kJ; ++j) {
    const int i = at.row + (wm * kFirst + j) * kGroup + r32;
    if (i < at.end) {
      float amax = kAmaxFloor;
#pragma unroll
      for (int q = 0; q < 4; ++q) amax = fmaxf(amax, sm.amax[q][wm * kHalf + j * 32 + r32]);
      const bool none = x_row(a, i) < 0;
      if (none) amax = kAmaxFloor;
      const float scale = amax / kFp8Max, inv = 1.0f / scale;
      u32x4_t codes;
#pragma unroll
      for (int q = 0; q < 4; ++q)
        codes[q] = none ? 0u
                        : e4m3x4_encode_nan(acc[j][0][4 * q] * inv, acc[j][0][4 * q + 1] * inv, acc[j][0][4 * q + 2] * inv,
                                            acc[j][0][4 * q + 3] * inv);
      *reinterpret_cast<u32x4_t*>(static_cast<uint8_t*>(a.out) + (size_t)i * I + tile_col * 128 + wn * 32 + h * 16) = codes;
      if (wn == 0 && h == 0) a.outs[(size_t)i * (I / 128) + tile_col] = scale;
    }
  }
}

template <bool kGlu, bool kMx, bool kWhole>
__device__ __forceinline__ void any_tile(const GroupedArgs& a, const TileAt& at, Shared& sm) {
  // the first half of the waves takes half of the 32-row groups, rounded up,
  // the other the rest; all branches meet the same barriers
  const int groups = (at.end - at.row + kGroup - 1) / kGroup, first = (groups + 1) / 2;
  const bool half = threadIdx.x < kThreads / 2;
  if (first == 2) {
    if (half || groups == 4)
      tile<kGlu, kMx, kWhole, 2, 2>(a, at, sm);
    else
      tile<kGlu, kMx, kWhole, 2, 1>(a, at, sm);
  } else if (half || groups == 2) {
    tile<kGlu, kMx, kWhole, 1, 1>(a, at, sm);
  } else {
    tile<kGlu, kMx, kWhole, 1, 0>(a, at, sm);
  }
}

// The whole kernel of a workgroup. kAll: every tile has all of K from its
// beginning on.
template <bool kGlu, bool kMx, bool kAll>
__device__ __forceinline__ void grouped_tile(const GroupedArgs& a, Shared& sm) {
  const TileAt at = find_tile<kRows, kGroup, kThreads>(a, blockIdx.x);
  if (at.e < 0) return;
  if (kAll || whole_k(a, at, kTurnRows))
    any_tile<kGlu, kMx, true>(a, at, sm);
  else
    any_tile<kGlu, kMx, false>(a, at, sm);
}

}  // namespace moe

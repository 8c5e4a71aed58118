// moe_grouped_swiglu: tiles of up to 128 rows by 128 hidden columns (256 weight
// rows) through LDS and the F16 matrix instructions.
#include <hip/hip_runtime.h>

#include "grouped_device.h"

namespace moe {
namespace {

constexpr int kThreads = 512;
constexpr int kGroup = 32;     // rows of a matrix instruction

template <int kRows>
struct Stage {
  uint8_t x[kRows * 128];
  uint8_t w[256 * 128];
  uint32_t xs[kRows < 64 ? 64 : kRows];  // FP32 scales, or four E8M0 bytes
};
template <int kRows, int kStages>
struct Shared {
  Stage<kRows> st[kStages];  // K blocks: one read, the others on their way
  float amax[4][kRows];
};

typedef float float16_t __attribute__((ext_vector_type(16)));

// Sixteen codes of a row in F16, two instructions' worth.
struct Wide16 {
  half8_t v[2];
};
__device__ __forceinline__ Wide16 widen16(const u32x4_t& q, float scale) {
  return Wide16{{widen8_scaled(q[0], q[1], scale), widen8_scaled(q[2], q[3], scale)}};
}

// kJ: the 32-row groups of this wave; `first`: those of the first four waves.
template <bool kMx, int kRows, int kStages, int kJ>
__device__ __forceinline__ void tile(const GroupedArgs& a, const TileAt& at, Shared<kRows, kStages>& sm, int first) {
  constexpr int kN = kJ ? kJ : 1, kHalf = kRows < 64 ? 32 : kRows / 2;
  const int tid = threadIdx.x, lane = tid & (kWave - 1);
  const int wave = __builtin_amdgcn_readfirstlane(tid / kWave);
  const int r32 = lane & 31, h = lane >> 5;
  const int wn = wave & 3, wm = wave >> 2;
  const int KB = a.K / 128, I = a.N / 2;

  // What this wave copies of a block: 32 LDS rows of the weights, 16 of the
  // activations and 64 scales (fewer where a tile has fewer rows: then several
  // waves copy the same, so that every wave has as many copies on its way).
  // LDS row L keeps 16-byte chunk c of its row at place c ^ (L / 2 % 8), so
  // that the 16 rows of a read phase differ in bank. A wave's results of an
  // instruction are weight rows 8 a + 4 h + b (a, b = 0..3) of its 32: these
  // are columns 16 h + 4 a + b, so that a lane's 16 are neighbours.
  constexpr int kXCopies = kRows / 64 ? kRows / 64 : 1, kCopies = 4 + kXCopies + 1;
  const int lr = lane >> 3;
  const auto x_of = [&](int L) {  // activation row of LDS row L
    const int m = L % kHalf + L / kHalf * kGroup * first;
    return (size_t)max(x_row(a, min(at.row + m, at.end - 1)), 0);
  };
  const int xl = kXCopies > 1 ? wave * 8 * kXCopies : (wave & (kRows / 8 - 1)) * 8;  // its first LDS row of the activations
  const uint8_t* xp[kXCopies];
#pragma unroll
  for (int i = 0; i < kXCopies; ++i) {
    const int L = xl + i * 8 + lr;
    xp[i] = a.x + x_of(L) * a.K + ((lane & 7) ^ ((L >> 1) & 7)) * 16;
  }
  // up rows for even waves, the same columns' gate rows for odd ones; its
  // eight LDS rows i begin 4 i columns further, at the other half's chunks
  // where i is odd
  const uint8_t* wp = a.w + ((size_t)at.e * a.N + at.col * 128 + (wave >> 1) * 32 + (wave & 1) * I) * a.K;
  const uint32_t wrow = (uint32_t)((lr >> 2) * 16 + (lr & 3)) * (uint32_t)a.K, chunk = ((lane & 7) ^ (lr >> 1)) * 16;
  const uint32_t woff[2] = {wrow + chunk, wrow + (chunk ^ 64)};
  const int sl = kRows < 64 ? 0 : wave % (kRows / 64) * 64;  // its first scale
  const uint8_t* sp = static_cast<const uint8_t*>(a.xs) + x_of(min(sl + lane, kRows - 1)) * KB * 4;
  const uint32_t lds = lds_offset(&sm);
  const auto issue = [&](int st, int kb) {
    const uint32_t to = lds + st * (uint32_t)sizeof(Stage<kRows>);
    const size_t k0 = (size_t)kb * 128;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      copy16_to_lds(wp + k0 + (size_t)(4 * i) * a.K, woff[i & 1],
                    to + (uint32_t)offsetof(Stage<kRows>, w) + (wave * 32 + i * 8) * 128);
#pragma unroll
    for (int i = 0; i < kXCopies; ++i) copy16_to_lds(xp[i] + k0, to + (xl + i * 8) * 128);
    copy4_to_lds(sp + (size_t)kb * 4, to + (uint32_t)offsetof(Stage<kRows>, xs) + sl * 4);
  };

  const uniform_floats su = as_uniform(a.ws) + ((size_t)at.e * (a.N / 128) + at.col) * KB;
  const uniform_floats sg = su + (size_t)(I / 128) * KB;

  // Sixteen bytes of every row (chunk h + 2 c of the lane's row) at a time,
  // widened while the matrix instructions of the chunk before run. Of a
  // wave's two products [t], 0 is up and 1 gate.
  const float16_t zero = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  int off[4];
#pragma unroll
  for (int c = 0; c < 4; ++c) off[c] = r32 * 128 + (((h + 2 * c) ^ (r32 >> 1)) & 7) * 16;
  Wide16 w[2][2], x[2][kN];  // [chunk parity]
  float rel[kN][4], xs[kN];
  float16_t acc[kN][2], p[kN][2];
#pragma unroll
  for (int j = 0; j < kJ; ++j) acc[j][0] = acc[j][1] = zero;
  const auto scales = [&](int st) {
#pragma unroll
    for (int j = 0; j < kJ; ++j) {
      const uint32_t sx = sm.st[st].xs[wm * kHalf + j * 32 + r32];
#pragma unroll
      for (int c = 0; c < 4; ++c) rel[j][c] = 1.f;
      xs[j] = kMx ? mx_scales(sx, rel[j]) : __uint_as_float(sx);
    }
  };
  const auto load = [&](int st, int c) {
    if (!kJ) return;
    const uint8_t *wb = sm.st[st].w + wn * 64 * 128, *xb = sm.st[st].x + wm * kHalf * 128;
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
              __builtin_amdgcn_mfma_f32_32x32x16_f16(w[c & 1][t].v[i], x[c & 1][j].v[i], c || i ? p[j][t] : zero, 0, 0, 0);
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
    const float s0 = su[b], s1 = sg[b];
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
    const int i = at.row + (wm * first + j) * kGroup + r32;
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
      *reinterpret_cast<u32x4_t*>(static_cast<uint8_t*>(a.out) + (size_t)i * I + at.col * 128 + wn * 32 + h * 16) = codes;
      if (wn == 0 && h == 0) a.outs[(size_t)i * (I / 128) + at.col] = scale;
    }
  }
}

template <bool kMx, int kRows, int kStages>
__global__ __launch_bounds__(kThreads, 2) void grouped_swiglu_kernel(GroupedArgs a) {
  __shared__ Shared<kRows, kStages> sm;
  const TileAt at = find_tile<kRows, kGroup, kThreads>(a, blockIdx.x);
  if (at.e < 0) return;
  // 32-row groups: the first half of the waves takes `first` of them, the
  // second half the rest, so that each SIMD has a wave of both. All branches
  // meet the same barriers.
  const int groups = (at.end - at.row + kGroup - 1) / kGroup, first = (groups + 1) / 2;
  const int mine = threadIdx.x < kThreads / 2 ? first : groups - first;
  if (kRows > 64 && mine == 2)
    tile<kMx, kRows, kStages, kRows / 64 ? kRows / 64 : 1>(a, at, sm, first);
  else if (mine == 1)
    tile<kMx, kRows, kStages, 1>(a, at, sm, first);
  else
    tile<kMx, kRows, kStages, 0>(a, at, sm, first);
}

template <bool kMx, int kRows, int kStages>
void launch(const GroupedArgs& a, hipStream_t stream) {
  const int64_t tiles = std::min<int64_t>(a.R, (int64_t)a.R / kRows + a.E) * a.col_tiles;
  hipLaunchKernelGGL((grouped_swiglu_kernel<kMx, kRows, kStages>), dim3((unsigned)((tiles + 7) / 8 * 8)), dim3(kThreads), 0,
                     stream, a);
}

}  // namespace

void launch_grouped_swiglu(bool mx, GroupedArgs a, hipStream_t stream) {
  a.col_tiles = a.N / 256;
  if ((int64_t)a.R <= (int64_t)a.E * 24)
    mx ? launch<true, 32, 4>(a, stream) : launch<false, 32, 4>(a, stream);
  else
    mx ? launch<true, 128, 3>(a, stream) : launch<false, 128, 3>(a, stream);
}

}  // namespace moe

// Products grouped by expert: tiles of up to 128 rows by 256 weight rows through
// LDS and the F16 matrix instructions.
#include <hip/hip_runtime.h>

#include "grouped_device.h"

namespace moe {
namespace {

constexpr int kThreads = 512;
constexpr int kWaves = kThreads / kWave;
constexpr int kRows = 128;   // activation rows of a tile
constexpr int kCols = 256;   // weight rows of a tile
constexpr int kStages = 3;   // K blocks in LDS: one read, two on their way

// Copies from memory straight into LDS: lane l's 16 (or 4) bytes go to byte
// 16 l (4 l) behind `to`, the same for the whole wave. In assembly, since the
// compiler waits for its own form of them before every later read of LDS,
// whichever buffer it reads; no register is written, and copies_left() waits
// until at most n of the wave's are on their way (they end in order). A
// workgroup barrier behind it makes all waves' copies visible.
__device__ __forceinline__ uint32_t lds_offset(const void* p) {
  return (uint32_t)(uintptr_t)(const __attribute__((address_space(3))) char*)p;
}
__device__ __forceinline__ void copy16_to_lds(const void* from, uint32_t to) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, off" ::"s"(to), "v"(from) : "m0");
}
__device__ __forceinline__ void copy4_to_lds(const void* from, uint32_t to) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dword %1, off" ::"s"(to), "v"(from) : "m0");
}
template <int kLeft>
__device__ __forceinline__ void copies_left(const void* lds) {
  asm volatile("s_waitcnt vmcnt(%1)" ::"v"(lds), "n"(kLeft) : "memory");
}

struct Stage {
  uint8_t x[kRows * 128];
  uint8_t w[kCols * 128];
  uint32_t xs[kRows];  // FP32 scales, or four E8M0 bytes
};
struct Shared {
  Stage st[kStages];
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

template <int kEpi, bool kMx, int kJ>
__device__ __forceinline__ void tile(const GroupedArgs& a, const TileAt& at, Shared& sm, int first) {
  constexpr int kN = kJ ? kJ : 1;
  constexpr bool kGlu = kEpi == kOutSwiglu;
  const int tid = threadIdx.x, lane = tid & (kWave - 1);
  const int wave = __builtin_amdgcn_readfirstlane(tid / kWave);
  const int r32 = lane & 31, h = lane >> 5;
  const int wn = wave & 3, wm = wave >> 2;
  const int KB = a.K / 128, I = a.N / 2;
  const int last = at.end - 1;

  // What this wave copies of a block: 16 LDS rows of the activations, 32 of
  // the weights, 64 scales. LDS row L keeps 16-byte chunk c of its row at
  // place c ^ (L / 2 % 8), so that the 16 rows of a read phase differ in bank.
  // A wave's results of an instruction are weight rows 8 a + 4 h + b (a, b =
  // 0..3) of its 32: these are columns 16 h + 4 a + b, so that a lane's 16
  // are neighbours.
  const uint8_t *xp[2], *wp[4];
  const int lr = lane >> 3;
  const auto chunk = [&](int L) { return ((lane & 7) ^ ((L >> 1) & 7)) * 16; };
  const auto x_of = [&](int L) {  // activation row of LDS row L
    const int m = (L & 63) + (L >> 6) * 32 * first;
    return (size_t)max(x_row(a, min(at.row + m, last)), 0);
  };
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int L = wave * 16 + i * 8 + lr;
    xp[i] = a.x + x_of(L) * a.K + chunk(L);
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int L = wave * 32 + i * 8 + lr, r = L & 31;
    const int c = ((r >> 2) & 1) * 16 + (r >> 3) * 4 + (r & 3);
    int n;
    if (kGlu)
      n = at.col * 128 + (L >> 6) * 32 + c + ((L >> 5) & 1) * I;
    else
      n = min(at.col * kCols + (L >> 5) * 32 + c, a.N - 1);
    wp[i] = a.w + ((size_t)at.e * a.N + n) * a.K + chunk(L);
  }
  const uint8_t* sp = static_cast<const uint8_t*>(a.xs) + x_of((wave & 1) * 64 + lane) * KB * 4;
  const uint32_t lds = lds_offset(&sm);
  constexpr int kCopies = 7;
  const auto issue = [&](int st, int kb) {
    const uint32_t to = lds + st * (uint32_t)sizeof(Stage);
#pragma unroll
    for (int i = 0; i < 4; ++i)
      copy16_to_lds(wp[i] + (size_t)kb * 128, to + (uint32_t)offsetof(Stage, w) + (wave * 32 + i * 8) * 128);
#pragma unroll
    for (int i = 0; i < 2; ++i) copy16_to_lds(xp[i] + (size_t)kb * 128, to + (wave * 16 + i * 8) * 128);
    // every wave copies scales, the same ones by four waves each: as many copies in every wave
    copy4_to_lds(sp + (size_t)kb * 4, to + (uint32_t)offsetof(Stage, xs) + (wave & 1) * 256);
  };

  const int n0 = kGlu ? at.col * 128 : at.col * kCols + wn * 64;
  const uniform_floats sw0 = as_uniform(a.ws) + ((size_t)at.e * (a.N / 128) + min(n0, a.N - 1) / 128) * KB;
  const uniform_floats sw1 = kGlu ? sw0 + (size_t)(I / 128) * KB : sw0;

  float16_t acc[kN][2];
#pragma unroll
  for (int j = 0; j < kJ; ++j)
#pragma unroll
    for (int t = 0; t < 2; ++t)
#pragma unroll
      for (int i = 0; i < 16; ++i) acc[j][t][i] = 0.f;

  int off[4];
#pragma unroll
  for (int c = 0; c < 4; ++c) off[c] = r32 * 128 + (((h + 2 * c) ^ (r32 >> 1)) & 7) * 16;

  if (wm) __builtin_amdgcn_s_setprio(1);
  // Sixteen bytes of every row (chunk h + 2 c of the lane's row) at a time,
  // widened while the matrix instructions of the chunk before run; the scaled
  // sums of a block are added while the next block's first ones run.
  Wide16 w[2][2], x[2][kN];  // [chunk parity]
  float rel[kN][4], sc[kN][2];
  const auto scales = [&](int st, int kb, float (&xs)[kN]) {
#pragma unroll
    for (int j = 0; j < kJ; ++j) {
      const uint32_t sx = sm.st[st].xs[wm * 64 + j * 32 + r32];
#pragma unroll
      for (int c = 0; c < 4; ++c) rel[j][c] = 1.f;
      xs[j] = kMx ? mx_scales(sx, rel[j]) : __uint_as_float(sx);
    }
  };
  const auto load = [&](int st, int c) {
    if (!kJ) return;
    const uint8_t *wb = sm.st[st].w + wn * 64 * 128, *xb = sm.st[st].x + wm * 64 * 128;
#pragma unroll
    for (int t = 0; t < 2; ++t) w[c & 1][t] = widen16(*reinterpret_cast<const u32x4_t*>(wb + t * 4096 + off[c]), 1.f);
#pragma unroll
    for (int j = 0; j < kJ; ++j)
      x[c & 1][j] = widen16(*reinterpret_cast<const u32x4_t*>(xb + j * 4096 + off[c]), rel[j][c]);
  };
  float16_t p[kN][2];
  const float16_t zero = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  const auto add = [&](int j, int t) {
#pragma unroll
    for (int i = 0; i < 16; ++i) acc[j][t][i] = fmaf(p[j][t][i], sc[j][t], acc[j][t][i]);
  };
  const auto multiply = [&](int c, bool first) {
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int j = 0; j < kJ; ++j)
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          p[j][t] = __builtin_amdgcn_mfma_f32_32x32x16_f16(w[c & 1][t].v[i], x[c & 1][j].v[i],
                                                           first && i == 0 ? zero : p[j][t], 0, 0, 0);
        }
  };
  const auto ready = [&](bool more) {  // block kb's copies have ended, in every wave
    if (more)
      copies_left<kCopies>(&sm);
    else
      copies_left<0>(&sm);
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
  };

  issue(0, 0);
  if (KB > 1) issue(1, 1);
  ready(KB > 1);
  if (KB > 2) issue(2, 2);
  float xs[kN];
  scales(0, 0, xs);
  load(0, 0);
  int st = 0;
  for (int kb = 0; kb < KB; ++kb) {
    const float s0 = sw0[kb], s1 = kGlu ? sw1[kb] : s0;
    load(st, 1);
    multiply(0, true);
    load(st, 2);
    multiply(1, false);
    load(st, 3);
    multiply(2, false);
#pragma unroll
    for (int j = 0; j < kJ; ++j)
#pragma unroll
      for (int t = 0; t < 2; ++t) sc[j][t] = xs[j] * (t ? s1 : s0);
    if (kb + 1 < KB) {
      ready(kb + 2 < KB);  // and every wave has read all of block kb
      if (kb + 3 < KB) issue(st, kb + 3);
      st = st == 2 ? 0 : st + 1;
      scales(st, kb + 1, xs);
      load(st, 0);
    }
    multiply(3, false);
#pragma unroll
    for (int j = 0; j < kJ; ++j)
#pragma unroll
      for (int t = 0; t < 2; ++t) add(j, t);
  }

  if (!kGlu) {
    if (n0 >= a.N) return;
#pragma unroll
    for (int j = 0; j < kJ; ++j) {
      const int i = at.row + (wm * first + j) * 32 + r32;
      if (i <= last) {
        const bool none = x_row(a, i) < 0;
        uint16_t* o = static_cast<uint16_t*>(a.out) + (size_t)i * a.N + n0 + h * 16;
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
          for (int q = 0; q < 2; ++q) {
            u32x4_t v;
#pragma unroll
            for (int b = 0; b < 4; ++b) v[b] = none ? 0u : bf16x2_bits(acc[j][t][8 * q + 2 * b], acc[j][t][8 * q + 2 * b + 1]);
            *reinterpret_cast<u32x4_t*>(o + t * 32 + q * 8) = v;
          }
      }
    }
    return;
  }
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
    if (h == 0) sm.amax[wn][wm * 64 + j * 32 + r32] = amax;
  }
  __syncthreads();
#pragma unroll
  for (int j = 0; j < kJ; ++j) {
    const int i = at.row + (wm * first + j) * 32 + r32;
    if (i <= last) {
      float amax = kAmaxFloor;
#pragma unroll
      for (int w = 0; w < 4; ++w) amax = fmaxf(amax, sm.amax[w][wm * 64 + j * 32 + r32]);
      const bool none = x_row(a, i) < 0;
      if (none) amax = kAmaxFloor;
      const float scale = amax / kFp8Max, inv = 1.0f / scale;
      u32x4_t codes;
#pragma unroll
      for (int q = 0; q < 4; ++q)
        codes[q] = none ? 0u
                        : e4m3x4_encode_nan(acc[j][0][4 * q] * inv, acc[j][0][4 * q + 1] * inv, acc[j][0][4 * q + 2] * inv,
                                            acc[j][0][4 * q + 3] * inv);
      *reinterpret_cast<u32x4_t*>(static_cast<uint8_t*>(a.out) + (size_t)i * I + n0 + wn * 32 + h * 16) = codes;
      if (wn == 0 && h == 0) a.outs[(size_t)i * (I / 128) + at.col] = scale;
    }
  }
}

template <int kEpi, bool kMx>
__global__ __launch_bounds__(kThreads, 2) void grouped_tile_kernel(GroupedArgs a) {
  __shared__ Shared sm;
  const TileAt at = find_tile<kRows, 32, kThreads>(a, blockIdx.x);
  if (at.e < 0) return;
  // 32-row groups: the first half of the waves takes `first` of them, the
  // second half the rest, so that each SIMD has a wave of both. All branches
  // meet the same barriers.
  const int groups = (at.end - at.row + 31) / 32, first = (groups + 1) / 2;
  const int mine = threadIdx.x < kThreads / 2 ? first : groups - first;
  if (mine == 2)
    tile<kEpi, kMx, 2>(a, at, sm, first);
  else if (mine == 1)
    tile<kEpi, kMx, 1>(a, at, sm, first);
  else
    tile<kEpi, kMx, 0>(a, at, sm, first);
}

template <int kEpi, bool kMx>
void launch(const GroupedArgs& a, int64_t tiles, hipStream_t stream) {
  hipLaunchKernelGGL((grouped_tile_kernel<kEpi, kMx>), dim3((unsigned)((tiles + 7) / 8 * 8)), dim3(kThreads), 0, stream, a);
}

}  // namespace

void launch_grouped_tile(Epilogue epi, bool mx, GroupedArgs a, hipStream_t stream) {
  a.col_tiles = (a.N + kCols - 1) / kCols;  // a SwiGLU tile: 128 up and 128 gate rows
  const int64_t tiles = std::min<int64_t>(a.R, (int64_t)a.R / kRows + a.E) * a.col_tiles;
  if (epi == kOutSwiglu)
    mx ? launch<kOutSwiglu, true>(a, tiles, stream) : launch<kOutSwiglu, false>(a, tiles, stream);
  else
    mx ? launch<kOutBf16, true>(a, tiles, stream) : launch<kOutBf16, false>(a, tiles, stream);
}

}  // namespace moe

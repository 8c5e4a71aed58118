// Products grouped by expert over ragged rows (include/moe_rows.h):
// moe_grouped_gemm and moe_grouped_swiglu.
#include <hip/hip_runtime.h>

#include <algorithm>

#include "../../include/moe_rows.h"
#include "grouped_device.h"

namespace moe {
namespace {

constexpr int kThreads = 256;
constexpr int kWaves = kThreads / kWave;

// Few rows per expert: the weights' bytes bound it. A workgroup takes up to
// 16 * kJ rows of one expert and kWaves * 16 * kS weight rows over all of K;
// each wave streams its 16 * kS weight rows from memory into registers, kDepth
// K blocks ahead, in the layout of the matrix instruction, and reads the
// activations from the caches in the same layout. The codes are widened to
// F16 (exact) and multiplied by the F16 instructions, whose sums are FP32
// throughout; at this few rows their lower rate is hidden behind memory. Each
// 128-wide block's partial is multiplied by its scales when it is added.
//
// A lane's results of the kS instructions of a block are 4 * kS neighbouring
// columns: instruction s takes weight rows (r / 4) * 4 * kS + 4 * s + r % 4.
// For the SwiGLU the wave's rows are 32 up and the 32 gate rows of the same
// hidden columns, so a lane holds both of a pair, and the four waves make one
// 128-wide block of the hidden.
template <int kEpi, bool kMx, int kJ, int kS, int kDepth>
__global__ __launch_bounds__(kThreads, 2) void grouped_stream_kernel(GroupedArgs a) {
  constexpr bool kGlu = kEpi == kOutSwiglu;
  static_assert(!kGlu || kS == 4, "two instructions of up rows and two of gate rows");
  __shared__ float amax_lds[kGlu ? kWaves : 1][16 * kJ];
  const TileAt at = find_tile<16 * kJ, kThreads>(a, blockIdx.x);
  if (at.e < 0) return;
  const int lane = threadIdx.x & (kWave - 1), wave = threadIdx.x / kWave;
  const int m = lane & 15, g = lane >> 4;
  const int KB = a.K / 128;
  const int subs = min((at.end - at.row + 15) / 16, kJ);

  // weight rows: gemm: columns n0 .. n0 + 16 kS - 1; SwiGLU: hidden columns
  // n0 .. n0 + 31, up and gate
  const int I = a.N / 2;
  const int n0 = kGlu ? at.col * 128 + wave * 32 : (at.col * kWaves + wave) * 16 * kS;
  if (!kGlu && n0 >= a.N) return;
  constexpr int kWide = kGlu ? 8 : 4 * kS;  // neighbouring columns per lane
  const uint8_t* wp[kS];
#pragma unroll
  for (int s = 0; s < kS; ++s) {
    const int gate = kGlu ? s / 2 : 0, t = kGlu ? s % 2 : s;
    const int n = n0 + (m / 4) * kWide + t * 4 + (m & 3) + gate * I;
    wp[s] = a.w + ((size_t)at.e * a.N + n) * a.K + g * 16;
  }
  const uniform_floats sw0 = as_uniform(a.ws) + ((size_t)at.e * (a.N / 128) + n0 / 128) * KB;
  const uniform_floats sw1 = kGlu ? sw0 + (size_t)(I / 128) * KB : sw0;

  const uint8_t* xp[kJ];
  const uint8_t* xsp[kJ];
#pragma unroll
  for (int j = 0; j < kJ; ++j) {
    const int r = max(x_row(a, min(at.row + 16 * j + m, at.end - 1)), 0);  // row 0 stands in where there is none
    xp[j] = a.x + (size_t)r * a.K + g * 16;
    xsp[j] = static_cast<const uint8_t*>(a.xs) + (size_t)r * KB * 4;
  }

  float4_t acc[kJ][kS];
#pragma unroll
  for (int j = 0; j < kJ; ++j)
#pragma unroll
    for (int s = 0; s < kS; ++s) acc[j][s] = float4_t{0.f, 0.f, 0.f, 0.f};

  u32x4_t wr[kDepth][kS][2], xr[kDepth][kJ][2];
  uint32_t xsr[kDepth][kJ];
  const auto request = [&](int d, int kb) {
    kb = min(kb, KB - 1);
#pragma unroll
    for (int s = 0; s < kS; ++s) {
      wr[d][s][0] = load_stream16(wp[s] + (size_t)kb * 128);
      wr[d][s][1] = load_stream16(wp[s] + (size_t)kb * 128 + 64);
    }
#pragma unroll
    for (int j = 0; j < kJ; ++j) {
      if (j < subs) {
        xr[d][j][0] = *reinterpret_cast<const u32x4_t*>(xp[j] + (size_t)kb * 128);
        xr[d][j][1] = *reinterpret_cast<const u32x4_t*>(xp[j] + (size_t)kb * 128 + 64);
        xsr[d][j] = *reinterpret_cast<const uint32_t*>(xsp[j] + (size_t)kb * 4);  // an FP32 scale or four E8M0 bytes
      }
    }
  };
#pragma unroll
  for (int d = 0; d < kDepth; ++d) request(d, d);
  for (int kb0 = 0; kb0 < KB; kb0 += kDepth) {
#pragma unroll
    for (int d = 0; d < kDepth; ++d) {
      const int kb = kb0 + d;
      if (kb < KB) {
        const float s0 = sw0[kb], s1 = kGlu ? sw1[kb] : s0;
        Wide xw[kJ];
        float xs[kJ];
#pragma unroll
        for (int j = 0; j < kJ; ++j) {
          if (j < subs) {
            if (kMx) {
              float rel[4];  // bytes 16g .. 16g+15 lie in block g / 2, 64 further in block 2 + g / 2
              xs[j] = mx_scales(xsr[d][j], rel);
              xw[j] = widen(xr[d][j][0], xr[d][j][1], g < 2 ? rel[0] : rel[1], g < 2 ? rel[2] : rel[3]);
            } else {
              xs[j] = __uint_as_float(xsr[d][j]);
              xw[j] = widen(xr[d][j][0], xr[d][j][1]);
            }
          }
        }
#pragma unroll
        for (int s = 0; s < kS; ++s) {
          const Wide ww = widen(wr[d][s][0], wr[d][s][1]);
#pragma unroll
          for (int j = 0; j < kJ; ++j) {
            if (j < subs) {
              const float4_t p = product_f16(ww, xw[j]);
              const float sc = xs[j] * (kGlu && s >= 2 ? s1 : s0);
#pragma unroll
              for (int i = 0; i < 4; ++i) acc[j][s][i] = fmaf(p[i], sc, acc[j][s][i]);
            }
          }
        }
        request(d, kb + kDepth);
      }
    }
  }

  if (!kGlu) {
#pragma unroll
    for (int j = 0; j < kJ; ++j) {
      const int i = at.row + 16 * j + m;
      if (i < at.end) {
        const bool none = x_row(a, i) < 0;
        const size_t o = (size_t)i * a.N + n0 + g * kWide;
#pragma unroll
        for (int s = 0; s < kS; ++s) {
          float4_t v = acc[j][s];
          if (none) v = float4_t{0.f, 0.f, 0.f, 0.f};
          *reinterpret_cast<u32x2_t*>(static_cast<uint16_t*>(a.out) + o + 4 * s) =
              u32x2_t{bf16x2_bits(v[0], v[1]), bf16x2_bits(v[2], v[3])};
        }
      }
    }
    return;
  }

  // SwiGLU: a lane's eight hidden values of a row, the row's maximum over the
  // 128 columns (lanes of the row, then the waves), the codes
#pragma unroll
  for (int j = 0; j < kJ; ++j) {
    float amax = kAmaxFloor;
#pragma unroll
    for (int t = 0; t < 2; ++t)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float v = swiglu(acc[j][t][i], acc[j][2 + t][i], a.limit);
        acc[j][t][i] = v;
        amax = fmaxf(amax, fabsf(v));
      }
    amax = fmaxf(amax, __shfl_xor(amax, 16, kWave));
    amax = fmaxf(amax, __shfl_xor(amax, 32, kWave));
    if (g == 0) amax_lds[kGlu ? wave : 0][16 * j + m] = amax;
  }
  __syncthreads();
#pragma unroll
  for (int j = 0; j < kJ; ++j) {
    const int i = at.row + 16 * j + m;
    if (i < at.end) {
      float amax = kAmaxFloor;
#pragma unroll
      for (int w = 0; w < (kGlu ? kWaves : 1); ++w) amax = fmaxf(amax, amax_lds[w][16 * j + m]);
      const bool none = x_row(a, i) < 0;
      if (none) amax = kAmaxFloor;
      const float scale = amax / kFp8Max, inv = 1.0f / scale;
      u32x2_t codes;
#pragma unroll
      for (int t = 0; t < 2; ++t)
        codes[t] = none ? 0u
                        : e4m3x4_encode_nan(acc[j][t][0] * inv, acc[j][t][1] * inv, acc[j][t][2] * inv,
                                            acc[j][t][3] * inv);
      *reinterpret_cast<u32x2_t*>(static_cast<uint8_t*>(a.out) + (size_t)i * I + n0 + g * 8) = codes;
      if (wave == 0 && g == 0) a.outs[(size_t)i * (I / 128) + at.col] = scale;
    }
  }
}

template <int kEpi, bool kMx, int kJ, int kS, int kDepth>
void launch_stream(GroupedArgs a, hipStream_t stream) {
  a.col_tiles = kEpi == kOutSwiglu ? a.N / 256 : (a.N + kWaves * 16 * kS - 1) / (kWaves * 16 * kS);
  // row tiles: each expert's rows rounded up, at most one tile per row
  const int64_t tiles = std::min<int64_t>(a.R, (int64_t)a.R / (16 * kJ) + a.E) * a.col_tiles;
  hipLaunchKernelGGL((grouped_stream_kernel<kEpi, kMx, kJ, kS, kDepth>), dim3((unsigned)((tiles + 7) / 8 * 8)),
                     dim3(kThreads), 0, stream, a);
}

template <Epilogue kEpi, bool kMx>
void launch(const GroupedArgs& a, hipStream_t stream) {
  if ((int64_t)a.R <= (int64_t)a.E * 8)
    launch_stream<kEpi, kMx, 1, 4, 4>(a, stream);
  else if ((int64_t)a.R > (int64_t)a.E * 32)
    launch_grouped_tile(kEpi, kMx, a, stream);
  else
    launch_stream<kEpi, kMx, 2, 4, 2>(a, stream);
}

bool misaligned(const void* p, uintptr_t to) { return (reinterpret_cast<uintptr_t>(p) & (to - 1)) != 0; }

int check(const moe_grouped_args* p) {
  if (!p) return MOE_DECODE_ERR_INVALID_ARG;
  const moe_grouped_args& a = *p;
  if (a.R < 0 || a.X < 0 || a.E < 1 || a.N < 1 || a.K < 1) return MOE_DECODE_ERR_INVALID_ARG;
  if (a.E > MOE_DECODE_MAX_EXPERTS || a.N % 128 || a.K % 128 || a.N > MOE_ROWS_MAX_DIM || a.K > MOE_ROWS_MAX_DIM ||
      a.quant < MOE_QUANT_FP8 || a.quant > MOE_QUANT_MXFP8)
    return MOE_DECODE_ERR_UNSUPPORTED;
  if (a.R == 0) return MOE_DECODE_OK;
  if (a.X < (a.rows ? 1 : a.R)) return MOE_DECODE_ERR_INVALID_ARG;
  if (!a.x || !a.x_scale || !a.offsets || !a.w || !a.w_scale || !a.out) return MOE_DECODE_ERR_INVALID_ARG;
  if (misaligned(a.x, 16) || misaligned(a.w, 16) || misaligned(a.out, 16) || misaligned(a.w_scale, 4) ||
      misaligned(a.offsets, 4) || misaligned(a.rows, 4) || misaligned(a.x_scale, 4))
    return MOE_DECODE_ERR_INVALID_ARG;
  // workgroups of any form of the kernels: a grid's limit
  if (((int64_t)a.R / 16 + a.E) * ((a.N + 255) / 256) > INT32_MAX - 8) return MOE_DECODE_ERR_UNSUPPORTED;
  return MOE_DECODE_OK;
}

GroupedArgs kernel_args(const moe_grouped_args& a) {
  GroupedArgs g{};
  g.x = static_cast<const uint8_t*>(a.x);
  g.xs = a.x_scale;
  g.rows = a.rows;
  g.offsets = a.offsets;
  g.w = static_cast<const uint8_t*>(a.w);
  g.ws = a.w_scale;
  g.out = a.out;
  g.outs = a.out_scale;
  g.R = a.R;
  g.X = a.X;
  g.E = a.E;
  g.N = a.N;
  g.K = a.K;
  g.limit = a.limit;
  return g;
}

}  // namespace
}  // namespace moe

extern "C" {

int moe_grouped_gemm(const moe_grouped_args* args, void* stream) {
  using namespace moe;
  if (const int rc = check(args)) return rc;
  if (args->R == 0) return MOE_DECODE_OK;
  const GroupedArgs a = kernel_args(*args);
  hipStream_t s = static_cast<hipStream_t>(stream);
  if (args->quant == MOE_QUANT_MXFP8)
    launch<kOutBf16, true>(a, s);
  else
    launch<kOutBf16, false>(a, s);
  return hipGetLastError() == hipSuccess ? MOE_DECODE_OK : MOE_DECODE_ERR_HIP;
}

int moe_grouped_swiglu(const moe_grouped_args* args, void* stream) {
  using namespace moe;
  if (const int rc = check(args)) return rc;
  if (args->N % 256) return MOE_DECODE_ERR_UNSUPPORTED;
  if (!(args->limit > 0.f)) return MOE_DECODE_ERR_INVALID_ARG;
  if (args->R == 0) return MOE_DECODE_OK;
  if (!args->out_scale || misaligned(args->out_scale, 4)) return MOE_DECODE_ERR_INVALID_ARG;
  const GroupedArgs a = kernel_args(*args);
  hipStream_t s = static_cast<hipStream_t>(stream);
  if (args->quant == MOE_QUANT_MXFP8)
    launch<kOutSwiglu, true>(a, s);
  else
    launch<kOutSwiglu, false>(a, s);
  return hipGetLastError() == hipSuccess ? MOE_DECODE_OK : MOE_DECODE_ERR_HIP;
}

}  // extern "C"

// moe_add_rmsnorm_quant (include/moe_rows.h): residual + addend + weighted
// expert rows, RMSNorm, BF16 and 8-bit outputs with scales, in one pass.
//
// One workgroup per token holds the whole row in registers, eight columns a
// lane and chunk, so every input is read once and every output written once:
// the bound is HBM (8,191 rows of 3584 with an addend, MXFP8: 54 us, 4.9 TB/s;
// 4,096 rows of 7168 with eight routed rows each: 142 us, 4.8 TB/s; a large copy
// runs at 4.9). The sum and the sum of squares are taken in FP64 (two
// more instructions per value, hidden behind memory): residual, addend, then the
// picks in their order, rounded to FP32. That is the correctly rounded sum but
// next to a rounding border and where terms of 2^29 times the result and more
// cancel; the same call gives the same bits every time. The sum of squares is
// joined over a workgroup's lanes, so the last bit of rstd may differ, next to a
// rounding border, between the workgroup sizes of the launch below.
#include <hip/hip_runtime.h>

#include "../../include/moe_rows.h"
#include "rows_device.h"

namespace moe {
namespace {

constexpr int kVec = 8;        // columns per lane and chunk (16 bytes of BF16)
constexpr int kBatch = 8;      // expert rows requested before they are added
constexpr int kMaxPicks = 32;
constexpr int kFewTokens = 512;  // see the launch

__device__ __forceinline__ void unpack8(const u32x4_t& w, float (&v)[kVec]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = bf16_value(w[i] & 0xFFFFu);
    v[2 * i + 1] = bf16_value(w[i] >> 16);
  }
}

__device__ __forceinline__ u32x4_t pack8(const float (&v)[kVec]) {
  return u32x4_t{bf16x2_bits(v[0], v[1]), bf16x2_bits(v[2], v[3]), bf16x2_bits(v[4], v[5]), bf16x2_bits(v[6], v[7])};
}

__device__ __forceinline__ u32x4_t load16(const void* p, size_t at) {
  return *reinterpret_cast<const u32x4_t*>(static_cast<const uint16_t*>(p) + at);
}

__device__ __forceinline__ double wave_sum_f64(double v) {
#pragma unroll
  for (int o = 1; o < kWave; o <<= 1) v += __shfl_xor(v, o, kWave);
  return v;
}

// The 8-bit form of a lane's eight values of row t from column col on; the
// lanes of a block (16 for 128 values, 4 for 32) hold neighbouring columns.
// Lanes past the row (live false) take part in the permutations only.
__device__ __forceinline__ void store_quant(const moe_norm_args& a, const float (&v)[kVec], int t, int col, bool live) {
  float amax = a.quant == MOE_QUANT_MXFP8 ? 0.f : kAmaxFloor;
#pragma unroll
  for (int i = 0; i < kVec; ++i) amax = fmaxf(amax, fabsf(v[i]));
  u32x2_t codes;
  if (a.quant == MOE_QUANT_MXFP8) {
    amax = dpp_max4(amax);
    const uint32_t u = __float_as_uint(amax);
    int shared = -127;
    if (u) shared = (u >> 23) ? (int)(u >> 23) - 127 - 8 : 31 - __builtin_clz(u) - 149 - 8;
    shared = max(shared, -127);
    float w[kVec];
#pragma unroll
    for (int i = 0; i < kVec; ++i) w[i] = ldexpf(v[i], -shared);
    codes[0] = e4m3x4_encode_nan(w[0], w[1], w[2], w[3]);
    codes[1] = e4m3x4_encode_nan(w[4], w[5], w[6], w[7]);
    if (live && (threadIdx.x & 3) == 0)
      static_cast<uint8_t*>(a.scale)[(size_t)t * (a.D / 32) + col / 32] = (uint8_t)(shared + 127);
  } else {
    amax = dpp_max16(amax);
    float s = amax / kFp8Max;
    if (a.quant == MOE_QUANT_FP8_P2) {
      const uint32_t b = __float_as_uint(fmaxf(s, kAmaxFloor));
      s = __uint_as_float(((b >> 23) + ((b & 0x7FFFFFu) != 0u)) << 23);
    }
    const float inv = 1.0f / s;
    codes[0] = e4m3x4_encode_nan(v[0] * inv, v[1] * inv, v[2] * inv, v[3] * inv);
    codes[1] = e4m3x4_encode_nan(v[4] * inv, v[5] * inv, v[6] * inv, v[7] * inv);
    if (live && (threadIdx.x & 15) == 0) static_cast<float*>(a.scale)[(size_t)t * (a.D / 128) + col / 128] = s;
  }
  if (live) *reinterpret_cast<u32x2_t*>(static_cast<uint8_t*>(a.q) + (size_t)t * a.D + col) = codes;
}

template <int kChunks, bool kRouted>
__global__ __launch_bounds__(1024) void norm_kernel(moe_norm_args a) {
  __shared__ double part[16];
  const int t = blockIdx.x, tid = threadIdx.x, lane = tid & (kWave - 1);
  const size_t row = (size_t)t * a.D;
  float h[kChunks][kVec];
  u32x4_t r[kChunks], d[kChunks], g[kChunks];
  const u32x4_t zero = {0u, 0u, 0u, 0u};
#pragma unroll
  for (int c = 0; c < kChunks; ++c) {  // lanes past the row read its start and drop it
    const int col = (c * (int)blockDim.x + tid) * kVec;
    const int at = col < a.D ? col : 0;
    r[c] = a.residual ? load16(a.residual, row + at) : zero;
    d[c] = a.delta ? load16(a.delta, row + at) : zero;
    g[c] = a.gamma ? load16(a.gamma, at) : zero;
  }
  double sq = 0.0;
#pragma unroll
  for (int c = 0; c < kChunks; ++c) {
    const int col = (c * (int)blockDim.x + tid) * kVec;
    const bool live = col < a.D;
    float rv[kVec], dv[kVec];
    unpack8(r[c], rv);
    unpack8(d[c], dv);
    if (kRouted) {
      const int at = live ? col : 0;
      double acc[kVec];
#pragma unroll
      for (int i = 0; i < kVec; ++i) acc[i] = (double)rv[i] + (double)dv[i];
      for (int j0 = 0; j0 < a.k; j0 += kBatch) {
        u32x4_t y[kBatch];
        double w[kBatch];
#pragma unroll
        for (int j = 0; j < kBatch; ++j) {
          w[j] = 0.0;
          y[j] = zero;
          if (j0 + j < a.k) {  // uniform: the token's own positions and weights
            const int p = a.pos[(size_t)t * a.k + j0 + j];
            if (p >= 0 && p < a.R) {
              w[j] = (double)a.weights[(size_t)t * a.k + j0 + j];
              y[j] = load16(a.y, (size_t)p * a.D + at);
            }
          }
        }
#pragma unroll
        for (int j = 0; j < kBatch; ++j) {
          float yv[kVec];
          unpack8(y[j], yv);
#pragma unroll
          for (int i = 0; i < kVec; ++i) acc[i] = fma(w[j], (double)yv[i], acc[i]);
        }
      }
#pragma unroll
      for (int i = 0; i < kVec; ++i) h[c][i] = (float)acc[i];
    } else {
#pragma unroll
      for (int i = 0; i < kVec; ++i) h[c][i] = rv[i] + dv[i];  // one rounding of an exact sum
    }
#pragma unroll
    for (int i = 0; i < kVec; ++i) {
      h[c][i] = live ? h[c][i] : 0.f;
      sq = fma((double)h[c][i], (double)h[c][i], sq);
    }
    if (a.residual_out && live)
      *reinterpret_cast<u32x4_t*>(static_cast<uint16_t*>(a.residual_out) + row + col) = pack8(h[c]);
  }
  if (a.gamma) {
    sq = wave_sum_f64(sq);
    if (lane == 0) part[tid / kWave] = sq;
    __syncthreads();
    double total = 0.0;
    for (int w = 0; w < (int)blockDim.x / kWave; ++w) total += part[w];
    const float rstd = (float)(1.0 / sqrt(total / (double)a.D + (double)a.eps));
#pragma unroll
    for (int c = 0; c < kChunks; ++c) {
      float gv[kVec];
      unpack8(g[c], gv);
#pragma unroll
      for (int i = 0; i < kVec; ++i) h[c][i] = (h[c][i] * rstd) * gv[i];
    }
  }
#pragma unroll
  for (int c = 0; c < kChunks; ++c) {
    const int col = (c * (int)blockDim.x + tid) * kVec;
    const bool live = col < a.D;
    if (a.out && live) *reinterpret_cast<u32x4_t*>(static_cast<uint16_t*>(a.out) + row + col) = pack8(h[c]);
    if (a.quant != MOE_QUANT_NONE) store_quant(a, h[c], t, col, live);
  }
}

template <int kChunks>
void launch_norm(const moe_norm_args& a, int threads, hipStream_t stream) {
  if (a.k)
    hipLaunchKernelGGL((norm_kernel<kChunks, true>), dim3(a.T), dim3(threads), 0, stream, a);
  else
    hipLaunchKernelGGL((norm_kernel<kChunks, false>), dim3(a.T), dim3(threads), 0, stream, a);
}

bool misaligned(const void* p, uintptr_t to) { return (reinterpret_cast<uintptr_t>(p) & (to - 1)) != 0; }

}  // namespace
}  // namespace moe

extern "C" int moe_add_rmsnorm_quant(const moe_norm_args* args, void* stream) {
  using namespace moe;
  if (!args) return MOE_DECODE_ERR_INVALID_ARG;
  const moe_norm_args& a = *args;
  if (a.T == 0) return MOE_DECODE_OK;
  if (a.T < 0 || a.R < 0 || a.k < 0 || !(a.eps >= 0.f) || !(a.eps <= 3.4e38f)) return MOE_DECODE_ERR_INVALID_ARG;
  if (a.quant < MOE_QUANT_NONE || a.quant > MOE_QUANT_MXFP8 || a.k > kMaxPicks || a.T > MOE_ROWS_MAX_TOKENS)
    return MOE_DECODE_ERR_UNSUPPORTED;
  const int unit = a.quant == MOE_QUANT_NONE ? kVec : a.quant == MOE_QUANT_MXFP8 ? 32 : 128;
  if (a.D <= 0 || a.D % unit || a.D > MOE_ROWS_MAX_D) return MOE_DECODE_ERR_UNSUPPORTED;
  if (!a.residual && !a.delta && !a.y) return MOE_DECODE_ERR_INVALID_ARG;
  if (!a.residual_out && !a.out && !a.q) return MOE_DECODE_ERR_INVALID_ARG;
  const bool routed = a.k > 0;
  if (routed != (a.y != nullptr) || routed != (a.pos != nullptr) || routed != (a.weights != nullptr))
    return MOE_DECODE_ERR_INVALID_ARG;
  const bool quant = a.quant != MOE_QUANT_NONE;
  if (quant != (a.q != nullptr) || quant != (a.scale != nullptr)) return MOE_DECODE_ERR_INVALID_ARG;
  if (misaligned(a.residual, 16) || misaligned(a.delta, 16) || misaligned(a.y, 16) || misaligned(a.gamma, 16) ||
      misaligned(a.residual_out, 16) || misaligned(a.out, 16) || misaligned(a.q, 16) || misaligned(a.pos, 4) ||
      misaligned(a.weights, 4) || (a.quant != MOE_QUANT_MXFP8 && misaligned(a.scale, 4)))
    return MOE_DECODE_ERR_INVALID_ARG;
  // Lanes for one chunk each: many, with all of a row's loads on their way at
  // once, for routed rows (whose positions come first: 4,096 tokens of eight
  // rows of 7168, 150 us against 171) and for few tokens (7168 columns: one
  // token 3.8 us against 4.6, 512 tokens 10.0 against 10.4); a quarter of
  // them, with more workgroups on a CU, for many plain rows (1,024 tokens
  // 14.9 against 16.5, 8,192 tokens 101 against 108).
  const int lanes = a.D / kVec;
  hipStream_t s = static_cast<hipStream_t>(stream);
  const auto waves = [](int n) { return (n + kWave - 1) / kWave * kWave; };
  const bool wide = routed || a.T <= kFewTokens;
  if (lanes <= (wide ? 1024 : 256))
    launch_norm<1>(a, waves(lanes), s);
  else if (wide || lanes <= 512)
    launch_norm<2>(a, waves((lanes + 1) / 2), s);
  else
    launch_norm<4>(a, waves((lanes + 3) / 4), s);
  return hipGetLastError() == hipSuccess ? MOE_DECODE_OK : MOE_DECODE_ERR_HIP;
}

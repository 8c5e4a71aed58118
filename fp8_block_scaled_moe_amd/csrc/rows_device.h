// Device pieces of the operators over any number of tokens (moe_rows.h, moe_block.h).
#pragma once

#include "../../include/moe_rows.h"
#include "device_common.h"

namespace moe {

// e4m3 codes of four values, nearest even, saturating, NaN kept as NaN (the
// median instruction that clamps would turn a NaN into -448).
__device__ __forceinline__ float clamp_fp8(float v) {
  return v != v ? v : __builtin_amdgcn_fmed3f(v, -kFp8Max, kFp8Max);
}

__device__ __forceinline__ uint32_t e4m3x4_encode_nan(float a, float b, float c, float d) {
  int w = __builtin_amdgcn_cvt_pk_fp8_f32(clamp_fp8(a), clamp_fp8(b), 0, false);
  w = __builtin_amdgcn_cvt_pk_fp8_f32(clamp_fp8(c), clamp_fp8(d), w, true);
  return (uint32_t)w;
}

typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));
typedef float float2_t __attribute__((ext_vector_type(2)));
typedef uint32_t u32x2_t __attribute__((ext_vector_type(2)));

// Two BF16 values, nearest even, NaN and infinities kept, low half first.
__device__ __forceinline__ uint32_t bf16x2_bits(float a, float b) {
  return __builtin_bit_cast(uint32_t, __builtin_convertvector(float2_t{a, b}, bf16x2_t));
}

// Maximum over aligned groups of 4 or 16 lanes, in every lane, by lane
// permutations inside a row of 16. A NaN takes no part.
__device__ __forceinline__ float dpp_max4(float v) {
  v = fmaxf(v, __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(v), 0xB1, 0xF, 0xF, false)));  // swap neighbours
  return fmaxf(v, __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(v), 0x4E, 0xF, 0xF, false)));  // swap pairs
}

__device__ __forceinline__ float dpp_max16(float v) {
  v = dpp_max4(v);
  v = fmaxf(v, __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(v), 0x141, 0xF, 0xF, false)));  // half-row mirror
  return fmaxf(v, __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(v), 0x140, 0xF, 0xF, false)));  // row mirror
}

constexpr int kVec = 8;  // columns per lane and chunk of a norm's row (16 bytes of BF16)

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

constexpr int kMaxPicks = 32;

inline bool misaligned(const void* p, uintptr_t to) { return (reinterpret_cast<uintptr_t>(p) & (to - 1)) != 0; }

// The checks of a norm call (T = 0: an empty one, whatever the rest).
inline int check_norm(const moe_norm_args& a) {
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
  return MOE_DECODE_OK;
}

}  // namespace moe

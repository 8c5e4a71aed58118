// Device pieces of the operators over any number of tokens (moe_rows.h).
#pragma once

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

}  // namespace moe

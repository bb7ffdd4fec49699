// Weights held in fewer bits, back to bf16 for the matrix cores: every conversion here is exact.
#pragma once

#include "device_common.h"

typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));

namespace moe {

// 8 codes -> 8 bf16 weights (code * scale, exact unless it overflows).
__device__ __forceinline__ bf16x8_t decode_w4(uint32_t q, float scale) {
  const bf16x2_t a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(q, scale, 0);
  const bf16x2_t b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(q, scale, 1);
  const bf16x2_t c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(q, scale, 2);
  const bf16x2_t d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(q, scale, 3);
  return bf16x8_t{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
}

// 8 E4M3 codes -> 8 bf16 weights.
__device__ __forceinline__ bf16x8_t decode_e4m3(uint32_t q0, uint32_t q1) {
  const bf16x2_t a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(q0, 1.0f, false);
  const bf16x2_t b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(q0, 1.0f, true);
  const bf16x2_t c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(q1, 1.0f, false);
  const bf16x2_t d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(q1, 1.0f, true);
  return bf16x8_t{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
}

// 8 int8 codes -> 8 bf16 weights: an integer of 8 bits as f32 has its bits in the upper half.
__device__ __forceinline__ bf16x8_t decode_i8(uint32_t q0, uint32_t q1) {
  u32x4 o;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t q = i < 2 ? q0 : q1;
    const int sh = 16 * (i & 1);
    const uint32_t lo = __float_as_uint((float)(int8_t)(q >> sh)), hi = __float_as_uint((float)(int8_t)(q >> (sh + 8)));
    o[i] = __builtin_amdgcn_perm(hi, lo, 0x07060302u);
  }
  return __builtin_bit_cast(bf16x8_t, o);
}

}  // namespace moe

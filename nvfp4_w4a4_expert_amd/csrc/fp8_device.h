// Device-side 8-bit helpers of the dense operators: OCP E4M3 codes with one
// fp32 scale per row, or one UE8M0 (power-of-two) scale per 32 elements.
//
// Row form:  scale = fl32(amax / 448), code = E4M3(fl32(y * inv)) with
//            inv = min(fl32(1 / scale), FLT_MAX), 0 for a row without a
//            nonzero finite element.
// Block form: scale = the smallest power of two P with amax <= 448 * P, held
//            as log2(P) + 127 clamped to [1, 254]; code = E4M3(y / P), a product
//            with a power of two.
// amax is the largest finite magnitude: an infinity or a NaN becomes the
// E4M3 NaN (E4M3 has no infinity) and leaves the scale of its row or block to
// the finite elements.  Values beyond 448 (only where a scale was clamped or
// rounded down) saturate.
#pragma once

#include "nvfp4_device.h"

namespace nvfp4 {

// |v| as an ordered integer, 0 where v is not finite (so a maximum skips it).
__device__ __forceinline__ uint32_t finite_mag(float v) {
  const uint32_t m = __float_as_uint(v) & 0x7FFFFFFFu;
  return m < 0x7F800000u ? m : 0u;
}

// Row scale and its multiplier from the row's largest finite magnitude.
__device__ __forceinline__ float row_scale(uint32_t amax_bits, float& inv) {
  const float s = __uint_as_float(amax_bits) / kE4M3Max;
  inv = s > 0.0f ? fminf(1.0f / s, kFltMax) : 0.0f;
  return s;
}

// UE8M0 code of a block and the multiplier 2^(127 - code).  448 = 1.75 * 2^8,
// so the exponent of the smallest covering power is that of amax minus 8, plus
// one where the mantissa of amax exceeds 1.75 (0x600000).
__device__ __forceinline__ uint32_t block_scale_code(uint32_t amax_bits, float& inv) {
  int c = (int)(amax_bits >> 23) - 8 + ((amax_bits & 0x7FFFFFu) > 0x600000u ? 1 : 0);
  c = c < 1 ? 1 : c;                                  // amax is finite: c <= 247
  inv = __uint_as_float((uint32_t)(254 - c) << 23);   // 2^(127 - c), a normal float
  return (uint32_t)c;
}

__device__ __forceinline__ float e4m3_clamp(float y, float inv) {
  const float v = y * inv;
  const float c = fminf(fmaxf(v, -kE4M3Max), kE4M3Max);
  return finite_mag(y) == (__float_as_uint(y) & 0x7FFFFFFFu) ? c : __uint_as_float(0x7FC00000u);
}

// Four values -> four E4M3 codes in one word, each rounded once, to nearest
// with ties to even.
__device__ __forceinline__ uint32_t encode4_e4m3(const float* y, float inv) {
  int w = 0;
  w = __builtin_amdgcn_cvt_pk_fp8_f32(e4m3_clamp(y[0], inv), e4m3_clamp(y[1], inv), w, false);
  w = __builtin_amdgcn_cvt_pk_fp8_f32(e4m3_clamp(y[2], inv), e4m3_clamp(y[3], inv), w, true);
  return (uint32_t)w;
}

// The same for values whose products with inv are finite and at most 448.
__device__ __forceinline__ uint32_t encode4_scaled(const float* y, float inv) {
  int w = 0;
  w = __builtin_amdgcn_cvt_pk_fp8_f32(y[0] * inv, y[1] * inv, w, false);
  w = __builtin_amdgcn_cvt_pk_fp8_f32(y[2] * inv, y[3] * inv, w, true);
  return (uint32_t)w;
}

// Maximum over aligned groups of four lanes.
__device__ __forceinline__ uint32_t quad_max(uint32_t v) {
  const uint32_t a = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0xB1, 0xF, 0xF, false);
  v = a > v ? a : v;
  const uint32_t b = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x4E, 0xF, 0xF, false);
  return b > v ? b : v;
}

// fp32 -> 16-bit pairs, rounded to nearest even (bf16: one instruction a pair).
__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  typedef float f32x2_t __attribute__((ext_vector_type(2)));
  typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));
  return __builtin_bit_cast(uint32_t, __builtin_convertvector(f32x2_t{a, b}, bf16x2_t));
}
__device__ __forceinline__ uint32_t pack_f16(float a, float b) {
  return (uint32_t)__builtin_bit_cast(uint16_t, (_Float16)a) |
         ((uint32_t)__builtin_bit_cast(uint16_t, (_Float16)b) << 16);
}

}  // namespace nvfp4

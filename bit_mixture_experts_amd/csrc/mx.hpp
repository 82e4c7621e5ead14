// MXFP8 and MXFP4: e4m3 or e2m1 codes in blocks of 32 with one e8m0 scale (a power of two) per
// block.
#pragma once

#include "common.hpp"

namespace moe4 {

constexpr uint32_t kMxNanScale = 255, kMxNanCode = 0x7F;

// |v| as bits: an unsigned maximum of these orders magnitudes and lets infinities and NaNs win
__device__ __forceinline__ uint32_t abs_bits(float v) { return __float_as_uint(v) & 0x7FFFFFFFu; }

// e8m0 byte of a block whose largest magnitude has these bits: 127 + the smallest e >= -127
// with magnitude <= 1.75 * 2^(e + P); 255 (NaN) where the block holds an infinity or a NaN.
// P = 8: 448, e4m3's largest value, so no code saturates. P = 2: 7, half a step past e2m1's
// largest value 6, so that none is off by more than half a step there either.
template <int P = 8>
__device__ __forceinline__ uint32_t mx_scale_byte(uint32_t top) {
  const int e = (int)(top >> 23) - P + ((top & 0x7FFFFFu) > 0x600000u ? 1 : 0);
  return top >= 0x7F800000u ? kMxNanScale : (uint32_t)max(e, 0);
}
// 2^(127 - byte), the factor that takes a value to its code's range (bytes up to 247; exact,
// and the product is too unless it falls below e4m3's smallest step)
__device__ __forceinline__ float mx_inverse(uint32_t byte) {
  return __uint_as_float((254u - min(byte, 253u)) << 23);
}
// four codes, v_cvt_pk_fp8_f32 (round to nearest even); NaN codes in a block of scale 255
__device__ __forceinline__ uint32_t mx_codes4(float a, float b, float c, float d, uint32_t byte) {
  const float f = mx_inverse(byte);
  int w = __builtin_amdgcn_cvt_pk_fp8_f32(a * f, b * f, 0, false);
  w = __builtin_amdgcn_cvt_pk_fp8_f32(c * f, d * f, w, true);
  return byte == kMxNanScale ? kMxNanCode * 0x01010101u : (uint32_t)w;
}
// maximum over the four lanes of a quad (a block of 32 as 8 values per lane)
__device__ __forceinline__ uint32_t quad_max(uint32_t v) {
  v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0xB1, 0xF, 0xF, false));
  return max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x4E, 0xF, 0xF, false));
}
// 8 values of a block that four neighbouring lanes share (all of them in the call): their
// codes and the block's scale byte
__device__ __forceinline__ u32x2 mx_quantize8(const float* v, uint32_t& byte) {
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) top = max(top, abs_bits(v[i]));
  byte = mx_scale_byte(quad_max(top));
  u32x2 q;
  q[0] = mx_codes4(v[0], v[1], v[2], v[3], byte);
  q[1] = mx_codes4(v[4], v[5], v[6], v[7], byte);
  return q;
}

// MXFP4: 8 values of a block that four neighbouring lanes share: their codes, the first in the
// low nibble, and the block's scale byte. The conversion divides by the scale and rounds to
// nearest even, past 6 to 6; a block of scale 255 (NaN) gets zeros.
__device__ __forceinline__ uint32_t mx4_quantize8(const float* v, uint32_t& byte) {
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) top = max(top, abs_bits(v[i]));
  byte = mx_scale_byte<2>(quad_max(top));
  const float f = mx_inverse(byte);
  uint32_t w = 0;
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[0] * f, v[1] * f, 1.0f, 0);
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[2] * f, v[3] * f, 1.0f, 1);
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[4] * f, v[5] * f, 1.0f, 2);
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[6] * f, v[7] * f, 1.0f, 3);
  return byte == kMxNanScale ? 0u : w;
}
// 8 codes (a dword) of a block with scale `byte` as bf16 (exact); a NaN scale gives NaNs
__device__ __forceinline__ u32x4 mx4_bf16x8(uint32_t w, uint32_t byte) {
  const float f = __uint_as_float(byte << 23);
  u32x4 r;
  r[0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, f, 0));
  r[1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, f, 1));
  r[2] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, f, 2));
  r[3] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, f, 3));
  return r;
}

// 8 codes (two dwords) of a block with scale `byte` as bf16: exact from 2^-133 on, e4m3's four
// significant bits and the scale's power of two fit; a NaN scale gives NaNs
__device__ __forceinline__ bf16x8 mx_bf16x8(uint32_t lo, uint32_t hi, uint32_t byte) {
  const float f = __uint_as_float(byte << 23);
  u32x4 r;
  r[0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, f, false));
  r[1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, f, true));
  r[2] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, f, false));
  r[3] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, f, true));
  return __builtin_bit_cast(bf16x8, r);
}

}  // namespace moe4

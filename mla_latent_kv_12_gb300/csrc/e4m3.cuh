// The 8-bit latent: e4m3 codes (OCP 8-bit float: 1 sign, 4 exponent and 3
// mantissa bits, bias 7, largest value 448, no infinity, NaN = 0x7F / 0xFF) in
// units of a power of two 2^(e - 127) per block of buffer rows, e one byte in
// [64, 134].
//
// Powers of two make the conversions to bf16 and f32 exact: a code times
// 2^(e - 127) has 4 significant bits and an exponent between -72 and 15, so it
// is a normal number of both, and moving a code to a larger unit only loses
// what falls below e4m3's smallest step.  fp16, the tensor cores' operand, is
// exact down to unit 2^-15 (a block whose largest magnitude is above 0.0068);
// below it values round to multiples of 2^-24.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <stdint.h>

namespace mla {

constexpr int kMinExponent = 64, kMaxExponent = 134;   // 448 * 2^(134 - 127) = 57344, inside the fp16 range
constexpr int kMaxScaleBlock = 64;                     // rows per exponent

__host__ __device__ __forceinline__ int clamp_exponent(int e) {
  return e < kMinExponent ? kMinExponent : (e > kMaxExponent ? kMaxExponent : e);
}

// The smallest exponent byte whose unit holds `amax` (>= 0): amax = f * 2^k with
// 1 <= f < 2 fits 448 = 1.75 * 2^8 units when f <= 1.75 at unit 2^(k - 8), else at 2^(k - 7).
__device__ __forceinline__ int exponent_for(float amax) {
  const uint32_t bits = __float_as_uint(amax);
  return clamp_exponent((int)(bits >> 23) - 8 + ((bits & 0x7FFFFFu) > 0x600000u ? 1 : 0));
}

__device__ __forceinline__ float unit_of(int e) { return __uint_as_float((uint32_t)e << 23); }
__device__ __forceinline__ float inverse_unit_of(int e) { return __uint_as_float((uint32_t)(254 - e) << 23); }

// Nearest e4m3 (ties to even), saturating at +-448; NaN becomes the NaN code.
__device__ __forceinline__ uint16_t encode_e4m3x2(float lo, float hi) {
  return (uint16_t)__nv_cvt_float2_to_fp8x2(make_float2(lo, hi), __NV_SATFINITE, __NV_E4M3);
}
__device__ __forceinline__ uint8_t encode_e4m3(float x) {
  return (uint8_t)__nv_cvt_float_to_fp8(x, __NV_SATFINITE, __NV_E4M3);
}

// code * unit in f32, exact: the code's exponent and mantissa bits placed at an
// f32's read as the value times 2^-120 (also below the smallest normal e4m3).
__device__ __forceinline__ float decode_e4m3(uint32_t code, float unit) {
  const float mag = __uint_as_float((code & 0x7Fu) << 20) * 0x1p120f;
  const float v = (code & 0x80u) ? -mag : mag;
  return (code & 0x7Fu) == 0x7Fu ? __uint_as_float(0x7FC00000u) : v * unit;
}

// Eight codes to eight fp16 values (four packed pairs): the hardware's exact
// conversion (NaN codes become NaN) and one packed multiplication by the unit
// `mul2` = 2^(e - 127) in both halves.  Exact for e >= kMinExponentF16: a code's
// least bit is at least 2^-9.  Below, values round to multiples of 2^-24.
constexpr int kMinExponentF16 = 127 - 15;
__device__ __forceinline__ uint32_t f16_unit(int e) {
  const __half h = __float2half_rn(__uint_as_float((uint32_t)e << 23));   // subnormal below 2^-14, 0 from 2^-25 down
  return (uint32_t)__half_as_ushort(h) * 0x00010001u;
}
__device__ __forceinline__ void decode_e4m3x8_f16(const uint2 codes, uint32_t mul2, uint32_t (&out)[4]) {
  const uint32_t w[2] = {codes.x, codes.y};
  const __half2 unit = *reinterpret_cast<const __half2*>(&mul2);
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    uint32_t lo, hi;
    asm("{\n .reg .b16 a, b;\n mov.b32 {a, b}, %2;\n cvt.rn.f16x2.e4m3x2 %0, a;\n cvt.rn.f16x2.e4m3x2 %1, b;\n}"
        : "=r"(lo), "=r"(hi) : "r"(w[j]));
    const __half2 x = __hmul2(*reinterpret_cast<const __half2*>(&lo), unit), y = __hmul2(*reinterpret_cast<const __half2*>(&hi), unit);
    out[2 * j] = *reinterpret_cast<const uint32_t*>(&x);
    out[2 * j + 1] = *reinterpret_cast<const uint32_t*>(&y);
  }
}

// Two bf16 values as fp16: exact from 2^-14 to 65280 in magnitude, multiples of
// 2^-24 below, saturating above.
__device__ __forceinline__ uint32_t bf16x2_to_f16x2(uint32_t v) {
  const float lo = __uint_as_float(v << 16), hi = __uint_as_float(v & 0xFFFF0000u);
  // (written so that NaN stays NaN)
  const __half2 h = __floats2half2_rn(lo > 65504.f ? 65504.f : lo < -65504.f ? -65504.f : lo,
                                      hi > 65504.f ? 65504.f : hi < -65504.f ? -65504.f : hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// Running maximum of the magnitudes of bf16 pairs (both halves; NaN ignored),
// and whether fp16 cannot hold it.
__device__ __forceinline__ uint32_t max_abs_bf16x2(uint32_t top, uint32_t v) {
  const __nv_bfloat162 r = __hmax2(*reinterpret_cast<const __nv_bfloat162*>(&top),
                                   __habs2(*reinterpret_cast<const __nv_bfloat162*>(&v)));
  return *reinterpret_cast<const uint32_t*>(&r);
}
__device__ __forceinline__ bool beyond_f16(uint32_t top) {
  return __uint_as_float(top << 16) > 65504.f || __uint_as_float(top & 0xFFFF0000u) > 65504.f;
}

// Sixteen codes to sixteen bf16 values (eight packed pairs), exact.  A code's
// bits placed at a bf16's exponent and mantissa read as the value times
// 2^-120; one packed multiplication by `mul2` = 2^(e - 7) in both halves
// (bf16_unit) gives the value.  The high byte of a bf16 is (sign, 4 zeros, 3
// exponent bits), the low one (exponent bit, 3 mantissa bits, 4 zeros): both
// are masked shifts of the whole word, and a byte permutation pairs them.
// NaN codes would read as 480: the returned word has bit 7 of a byte set iff
// some code is NaN (the carry of magnitude 0x7F + 1), and the caller mends those.
__device__ __forceinline__ uint32_t bf16_unit(int e) { return (uint32_t)(e + 120) * 0x00800080u; }

__device__ __forceinline__ uint32_t mul_bf16x2(uint32_t a, uint32_t b) {
  const __nv_bfloat162 r = __hmul2(*reinterpret_cast<const __nv_bfloat162*>(&a), *reinterpret_cast<const __nv_bfloat162*>(&b));
  return *reinterpret_cast<const uint32_t*>(&r);
}

__device__ __forceinline__ uint32_t decode_e4m3x16(const uint4 codes, uint32_t mul2, uint32_t (&out)[8]) {
  const uint32_t w[4] = {codes.x, codes.y, codes.z, codes.w};
  uint32_t carry = 0;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    carry |= (w[j] & 0x7F7F7F7Fu) + 0x01010101u;
    const uint32_t high = ((w[j] >> 4) & 0x07070707u) | (w[j] & 0x80808080u);
    const uint32_t low = (w[j] << 4) & 0xF0F0F0F0u;
    out[2 * j] = mul_bf16x2(__byte_perm(low, high, 0x5140), mul2);
    out[2 * j + 1] = mul_bf16x2(__byte_perm(low, high, 0x7362), mul2);
  }
  return carry & 0x80808080u;
}

// Puts NaN where `codes` have it.
__device__ __forceinline__ void mend_nan_e4m3x16(const uint4 codes, uint32_t (&out)[8]) {
  const uint32_t w[4] = {codes.x, codes.y, codes.z, codes.w};
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const uint32_t two = w[j >> 1] >> (16 * (j & 1));
    if ((two & 0x7Fu) == 0x7Fu) out[j] = (out[j] & 0xFFFF0000u) | 0x7FC0u;
    if ((two & 0x7F00u) == 0x7F00u) out[j] = (out[j] & 0xFFFFu) | 0x7FC00000u;
  }
}

}  // namespace mla

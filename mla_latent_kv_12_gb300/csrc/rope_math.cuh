// One rotary pair of the partial interleaved RoPE ("glm52-mla.ts",
// partialInterleavedRopeMlx), shared by the RoPE kernel and the fused
// RoPE + absorb kernel.  The angle is f32(p * invf_j), the exact product
// rounded once (the page forms it in f64 and rounds with fround); sin/cos are
// CUDA's accurate sincosf of that f32 angle.
#pragma once

#include <stdint.h>

namespace mla {

// f32(pos * inv_freq), the exact product rounded once.  While |pos| <= 2^24
// the position is an exact f32 and the f32 product is already that rounding
// (the exact product of two f32 values fits a double, so both routes round the
// same real number); beyond, the product is formed in double.
__device__ __forceinline__ float rope_angle(int64_t pos, float inv_freq) {
  if (pos >= -(1LL << 24) && pos <= (1LL << 24)) return __fmul_rn((float)pos, inv_freq);
  return __double2float_rn((double)pos * (double)inv_freq);
}

__device__ __forceinline__ void rope_rotate_pair(float a, float b, int64_t pos, float inv_freq, float& re,
                                                 float& im) {
  const float ang = rope_angle(pos, inv_freq);
  float s, c;
  sincosf(ang, &s, &c);
  re = a * c - b * s;
  im = b * c + a * s;
}

// Sine and cosine of |x| <= kSmallAngle without branches: x less the nearest
// multiple of pi / 2, which is subtracted in three f32 parts with fused
// multiply-adds (Cody and Waite; the first is exact: x and the multiple are both
// multiples of 2^-24, their difference is below 1), then the Taylor sums, whose
// remainders on [-pi/4, pi/4] are below 2^-28.  Absolute error below 1.2 * 2^-24
// (against 64 bits over the range and next to the multiples of pi / 2).
constexpr float kSmallAngle = 65536.f;
__device__ __forceinline__ void sincos_small(float x, float& sine, float& cosine) {
  const float shifted = fmaf(x, 0.6366197723675814f, 12582912.f);   // 1.5 * 2^23: the low bits are the nearest integer
  const uint32_t quadrant = __float_as_uint(shifted);
  const float k = shifted - 12582912.f;
  float r = fmaf(-k, 0x1.921fb6p+0f, x);
  r = fmaf(-k, -0x1.777a5cp-25f, r);
  r = fmaf(-k, -0x1.ee59dap-50f, r);
  const float z = r * r;
  float s = fmaf(fmaf(fmaf(1.f / 362880, z, -1.f / 5040), z, 1.f / 120), z, -1.f / 6);
  s = fmaf(r * z, s, r);
  float c = fmaf(fmaf(fmaf(-1.f / 3628800, z, 1.f / 40320), z, -1.f / 720), z, 1.f / 24);
  c = fmaf(fmaf(c, z, -0.5f), z, 1.f);
  const bool swap = quadrant & 1u;
  sine = __uint_as_float(__float_as_uint(swap ? c : s) ^ ((quadrant & 2u) << 30));
  cosine = __uint_as_float(__float_as_uint(swap ? s : c) ^ (((quadrant + 1u) & 2u) << 30));
}

}  // namespace mla

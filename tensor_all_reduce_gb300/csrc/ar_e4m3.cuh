// E4M3 codes and the scales of their blocks.
#pragma once

#include "ar_common.cuh"
#include "ar_serve.h"

namespace ar {

__device__ __forceinline__ float clamp_scale(float s) { return fminf(fmaxf(s, kScaleLow), kScaleHigh); }

// Smallest power of two 2^e with top <= 448 * 2^e = 1.75 * 2^(e + 8), in the scales' range: the exponent of
// top, and one more where its fraction is above 1.75's.
__device__ __forceinline__ float fresh_scale(float top) {
  const int e = (int)((__float_as_uint(top) + 0x1fffffu) >> 23) - 8;
  return __uint_as_float((unsigned)min(max(e, 127 - 32), 127 + 32) << 23);
}

// Magnitude that counts for a scale.
__device__ __forceinline__ float finite_magnitude(float y) { return fabsf(y) <= 3.402823466e38f ? fabsf(y) : 0.0f; }

// y / scale before its rounding to E4M3 (inv = 1 / scale, a power of two or not far from one).
__device__ __forceinline__ float for_code(float y, float inv) { return fabsf(y) <= 3.402823466e38f ? y * inv : __uint_as_float(0x7fffffffu); }

// Two codes to floats.
__device__ __forceinline__ void from_e4m3x2(uint32_t codes, float& a, float& b) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((unsigned short)codes));
  a = to_f32<kF16>(h & 0xffffu);
  b = to_f32<kF16>(h >> 16);
}

// Of a k scale and what a row of q was divided by: finite, so that a product of 0 stays 0 under it.
__device__ __forceinline__ float finite_product(float k, float q) { return fminf(k * q, 3.402823466e38f); }

// What attention needs of a block's scales: the k scale, log2 and reciprocal of the v scale.
__device__ __forceinline__ float4 load_scales(const AttnParams& p, int64_t block, int h) {
  const float k = clamp_scale(p.k_scale.p[block * p.k_scale.bs + h * p.k_scale.hs]);
  const float v = clamp_scale(p.v_scale.p[block * p.v_scale.bs + h * p.v_scale.hs]);
  return make_float4(k, log2f(v), 1.0f / v, 0.0f);
}

}  // namespace ar

// MX8, the 8-bit form that the library's operators share (the OCP microscaling
// format MXFP8 with E4M3 elements): 32 consecutive elements of a row have one
// E8M0 scale, a byte b that stands for 2^(b - 127) (255: NaN).  A row of n
// elements has ceil(n / 32) scales; its last group may be shorter.
//
//   b = the smallest byte >= 1 with amax * 2^(127 - b) <= 448 (E4M3's largest value)
//   q = E4M3(x * 2^(127 - b)), rounded to nearest even
//
// Both follow from x alone: a power of two scales exactly, so the only rounding
// is that of the element, and nothing saturates.  b >= 1 keeps 2^(127 - b) and
// its inverse normal float32 numbers (a group of values below 2^-118 loses
// relative precision, never more than 2^-136 absolutely).  A NaN is a NaN
// element and leaves its neighbours alone; a group with an infinity, which
// E4M3 lacks, has the scale NaN: all its values read NaN.
#pragma once

#include <cstdint>

#include <cuda_fp8.h>

#include "device_common.cuh"

namespace ep {

constexpr int kMxGroup = 32;
inline int64_t mx_groups(int64_t n) { return (n + kMxGroup - 1) / kMxGroup; }

namespace dev {

// The scale's byte for a group whose largest magnitude is amax (>= 0; NaN
// values left out).  448 = 1.75 * 2^8: the exponent goes up by one where the
// fraction is above 1.75, which the addition carries into it.
__device__ __forceinline__ uint32_t mx_scale(float amax) {
  const uint32_t bits = __float_as_uint(amax);
  const int b = int((bits + 0x1FFFFFu) >> 23) - 8;
  return bits == 0x7F800000u ? 255u : uint32_t(max(b, 1));
}

// 2^(127 - b), the factor in front of the rounding (b <= 247; 2^-128 flushed to 0 for the NaN scale).
__device__ __forceinline__ float mx_factor(uint32_t b) { return __uint_as_float(b == 255u ? 0u : (254u - b) << 23); }

// 2^(b - 127); 2^-127 (b = 0, which mx_scale does not make) is subnormal.
__device__ __forceinline__ float mx_value(uint32_t b) {
  return __uint_as_float(b == 0u ? 0x00400000u : b == 255u ? 0x7FFFFFFFu : b << 23);
}

// Two float32 to two E4M3 bytes, the first in the low byte.
__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ uint32_t e4m3x4(float a, float b, float c, float d) {
  return e4m3x2(a, b) | (e4m3x2(c, d) << 16);
}

// Two E4M3 bytes (the low 16 bits) to float32, exactly.
__device__ __forceinline__ float2 e4m3_floats(uint32_t two) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(uint16_t(two)));
  return __half22float2(*reinterpret_cast<const __half2*>(&h));
}

__device__ __forceinline__ float from_float(float v, float) { return v; }
__device__ __forceinline__ __half from_float(float v, __half) { return __float2half_rn(v); }
__device__ __forceinline__ __nv_bfloat16 from_float(float v, __nv_bfloat16) { return __float2bfloat16_rn(v); }

}  // namespace dev
}  // namespace ep

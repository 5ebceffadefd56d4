// The activations of the matrix product's epilogue and their derivatives, in
// float32, for results that are rounded to 16 (or 8) bits.
//
//   silu z s(z);  quick_gelu z s(alpha z);  fast_gelu (the tanh form) z s(t(z)),
//   t(z) = 2 sqrt(2/pi) (z + 0.044715 z^3), as (1 + tanh(x)) / 2 = s(2 x);
//   gelu z Phi(z);  relu max(z, 0).  s(x) = 1 / (1 + e^-x).
//   d/dz [z s(t)] = s + z t' s (1 - s);  d/dz [z Phi(z)] = Phi(z) + z e^(-z^2/2) / sqrt(2 pi)
//
// s is taken from the hardware's 2^x and 1/x: a few float32 ulp, which the
// rounding to 11 bits or fewer hides.  Phi is 1/2 erfc(|z| / sqrt(2)), or 1 less that,
// in the form of Abramowitz and Stegun 7.1.26 (Handbook of Mathematical Functions, 1964),
// erfc(x) = (a1 t + .. + an t^n) e^(-x^2), t = 1 / (1 + p x).  Its own five coefficients
// bound the absolute error (1.5e-7), which is 5e-4 of the result at z = -4 and 4e-2 at
// -12.9; these seven, fitted here to the least relative error over 0 <= x <= 9.3, are
// within 5.1e-7 of erfc everywhere, so that the negative tail of gelu is rounded once
// too.  13 instructions without a branch (with erff the epilogue of f16 1331 x 1000 x 768
// took 6 us longer), and its e^(-z^2/2) is the density's too.  Where s has run down to 0
// the result is 0 also for z = -inf (its limit), and NaN stays NaN.
#pragma once

#include "device_common.cuh"
#include "mx8_internal.h"

namespace ep {
namespace dev {

__device__ __forceinline__ float sigmoid_fast(float x) { return rcp_approx(1.0f + ex2_approx(-kLog2e * x)); }

constexpr float kTanhScale = 1.5957691216057308f;  // 2 sqrt(2/pi)
constexpr float kTanhCubic = 0.044715f;

// z s(t), t of z's sign (or both reversed); below t = -87 s is under 2^-125.
__device__ __forceinline__ float gated(float z, float t) { return t < -87.0f ? 0.0f : z * sigmoid_fast(t); }

// Phi(z) and e^(-z^2/2), |z| <= 13.
__device__ __forceinline__ float normal_cdf(float z, float* e) {
  const float t = rcp_approx(fmaf(0.26359382f, fabsf(z), 1.0f));  // 0.37277796 / sqrt(2)
  *e = ex2_approx(-0.5f * kLog2e * z * z);
  float q = fmaf(-0.13974904f, t, 0.41349297f);
  q = fmaf(q, t, -0.16074581f);
  q = fmaf(q, t, 0.30254010f);
  q = fmaf(q, t, 0.15880841f);
  q = fmaf(q, t, 0.21565410f);
  q = fmaf(q, t, 0.20999877f);
  q *= 0.5f * t * *e;
  return z < 0.0f ? q : 1.0f - q;
}

// z held within [-lim, lim], where a slope has reached its limits; NaN stays.
__device__ __forceinline__ float held(float z, float lim) { return z < -lim ? -lim : z > lim ? lim : z; }

template <int ACT>
__device__ __forceinline__ float act_value(float z, float alpha) {
  if constexpr (ACT == kActSilu) return gated(z, z);
  if constexpr (ACT == kActRelu) return z < 0.0f ? 0.0f : z;
  if constexpr (ACT == kActQuickGelu) return gated(z, alpha * z);
  if constexpr (ACT == kActGelu) {
    float e;
    return z < -13.0f ? 0.0f : z * normal_cdf(held(z, 13.0f), &e);
  }
  if constexpr (ACT == kActFastGelu) return gated(z, z * fmaf(kTanhScale * kTanhCubic, z * z, kTanhScale));
  return z;
}

template <int ACT>
__device__ __forceinline__ float act_slope(float z, float alpha) {
  if constexpr (ACT == kActSilu || ACT == kActQuickGelu) {
    const float t = held(ACT == kActSilu ? z : alpha * z, 80.0f);
    const float s = sigmoid_fast(t);
    return fmaf(t * s, 1.0f - s, s);
  }
  if constexpr (ACT == kActRelu) return z > 0.0f ? 1.0f : 0.0f;
  if constexpr (ACT == kActGelu) {
    z = held(z, 13.0f);
    float e;
    const float cdf = normal_cdf(z, &e);
    return fmaf(z * 0.3989422804014327f, e, cdf);
  }
  if constexpr (ACT == kActFastGelu) {
    z = held(z, 13.0f);
    const float s = sigmoid_fast(z * fmaf(kTanhScale * kTanhCubic, z * z, kTanhScale));
    const float slope = fmaf(3.0f * kTanhScale * kTanhCubic, z * z, kTanhScale);
    return fmaf(z * slope * s, 1.0f - s, s);
  }
  return 1.0f;
}

// f(std::integral_constant) by the activation, outside the loops over elements.
template <int A> struct ActTag { static constexpr int value = A; };
template <typename F>
__device__ __forceinline__ void by_act(int act, F f) {
  switch (act) {
    case kActSilu: f(ActTag<kActSilu>()); break;
    case kActRelu: f(ActTag<kActRelu>()); break;
    case kActQuickGelu: f(ActTag<kActQuickGelu>()); break;
    case kActGelu: f(ActTag<kActGelu>()); break;
    case kActFastGelu: f(ActTag<kActFastGelu>()); break;
    default: f(ActTag<kActNone>()); break;
  }
}

}  // namespace dev
}  // namespace ep

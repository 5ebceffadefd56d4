// What the two forms of GroupNorm share: the activation and its derivative, and
// the interface of the fused form.
#pragma once

#include <cstdint>
#include <type_traits>

#include "device_common.cuh"
#include "training_internal.h"

namespace ep {

// sigmoid(u) = 1 / (1 + e^-u).
//  float32: e^-u = 2^p (1 + c), p = -u log2(e) rounded and c what the rounding
//  and log2(e)'s own left out, times ln 2; the reciprocal by the hardware's
//  approximation and one Newton step: within 3 float32 ulp.  u comes from -87 on
//  (from_87), and from 100 on e^-u counts as e^-100: nothing overflows.
//  16-bit results: 2^x and 1/x by the hardware approximations with p rounded,
//  errors of a few float32 ulp and |u| 2^-24, far below the results' rounding;
//  from u = -88.7 down 2^p overflows and sigmoid(u) is 0.
template <typename T>
__device__ __forceinline__ float sigmoid(float u) {
  if constexpr (std::is_same_v<T, float>) {
    constexpr float kL = 1.44269502162933349609375f;  // log2(e) rounded to float32
    constexpr float kLlo = 1.92596298909109e-08f;     // log2(e) - kL
    constexpr float kLn2 = 0.6931471805599453f;
    const float t = fmaxf(-u, -100.f);
    const float p = __fmul_rn(t, kL);
    const float c = fmaf(t, kL, -p) + t * kLlo;
    const float e = dev::ex2_approx(p);
    const float d = 1.0f + fmaf(e * c, kLn2, e);
    const float r = dev::rcp_approx(d);
    return fmaf(r, fmaf(-d, r, 1.0f), r);
  } else {
    return dev::rcp_approx(1.0f + dev::ex2_approx(u * -dev::kLog2e));
  }
}

// float32: u, or -87 below that (NaN stays NaN), where u sigmoid(u) is above -1.5e-36 and
// goes to 0: with u itself beside a sigmoid held at e^-87 it grew again, to -4.9 at -3e38.
template <typename T>
__device__ __forceinline__ float from_87(float u) {
  if constexpr (std::is_same_v<T, float>) asm("max.NaN.f32 %0, %0, %1;" : "+f"(u) : "f"(-87.f));
  return u;
}

template <typename T>
__device__ __forceinline__ float silu(float u) {
  u = from_87<T>(u);
  return u * sigmoid<T>(u);
}

// du of the definition.
template <typename T>
__device__ __forceinline__ float silu_grad(float dy, float u) {
  u = from_87<T>(u);
  const float s = sigmoid<T>(u);
  return dy * (s * fmaf(u, 1.0f - s, 1.0f));
}

// The same on VW values, two to a packed float32 instruction where there is
// one (each lane rounded as the scalar operation would).
//   activate: v <- v * sigmoid(v);  activate_grad: w <- w * derivative at u
template <typename T, int VW>
__device__ __forceinline__ void activate(float (&v)[VW]) {
  if constexpr (std::is_same_v<T, float>) {
#pragma unroll
    for (int e = 0; e < VW; ++e) v[e] = silu<T>(v[e]);
  } else {
#pragma unroll
    for (int e = 0; e < VW; e += 2) {
      const float2 u = make_float2(v[e], v[e + 1]);
      const float2 t = __fmul2_rn(u, make_float2(-dev::kLog2e, -dev::kLog2e));
      const float2 d = __fadd2_rn(make_float2(dev::ex2_approx(t.x), dev::ex2_approx(t.y)), make_float2(1.f, 1.f));
      const float2 y = __fmul2_rn(u, make_float2(dev::rcp_approx(d.x), dev::rcp_approx(d.y)));
      v[e] = y.x;
      v[e + 1] = y.y;
    }
  }
}
template <typename T, int VW>
__device__ __forceinline__ void activate_grad(float (&w)[VW], const float (&u)[VW]) {
  if constexpr (std::is_same_v<T, float>) {
#pragma unroll
    for (int e = 0; e < VW; ++e) w[e] = silu_grad<T>(w[e], u[e]);
  } else {
#pragma unroll
    for (int e = 0; e < VW; e += 2) {
      const float2 one = make_float2(1.f, 1.f);
      const float2 u2 = make_float2(u[e], u[e + 1]), w2 = make_float2(w[e], w[e + 1]);
      const float2 t = __fmul2_rn(u2, make_float2(-dev::kLog2e, -dev::kLog2e));
      const float2 d = __fadd2_rn(make_float2(dev::ex2_approx(t.x), dev::ex2_approx(t.y)), one);
      const float2 s = make_float2(dev::rcp_approx(d.x), dev::rcp_approx(d.y));
      const float2 f = __ffma2_rn(u2, __ffma2_rn(s, make_float2(-1.f, -1.f), one), one);
      const float2 y = __fmul2_rn(__fmul2_rn(w2, s), f);
      w[e] = y.x;
      w[e + 1] = y.y;
    }
  }
}

// v <- (v - m) * k + b, and v <- (v - m) * k, each product and sum rounded once
// (m, k: one value, or one for each element).
template <int VW, int EV>
__device__ __forceinline__ float2 pair_of(const float (&a)[EV], int e) {
  return EV == 1 ? make_float2(a[0], a[0]) : make_float2(a[EV == 1 ? 0 : e], a[EV == 1 ? 0 : e + 1]);
}
template <int VW, int EV>
__device__ __forceinline__ void centre_scale_add(float (&v)[VW], const float (&m)[EV], const float (&k)[VW],
                                                 const float (&b)[VW]) {
#pragma unroll
  for (int e = 0; e < VW; e += 2) {
    const float2 m2 = pair_of<VW>(m, e);
    const float2 t = __fadd2_rn(make_float2(v[e], v[e + 1]), make_float2(-m2.x, -m2.y));
    const float2 r = __ffma2_rn(t, make_float2(k[e], k[e + 1]), make_float2(b[e], b[e + 1]));
    v[e] = r.x;
    v[e + 1] = r.y;
  }
}
template <int VW, int EV>
__device__ __forceinline__ void centre_scale(float (&v)[VW], const float (&m)[EV], const float (&k)[EV]) {
#pragma unroll
  for (int e = 0; e < VW; e += 2) {
    const float2 m2 = pair_of<VW>(m, e);
    const float2 t = __fadd2_rn(make_float2(v[e], v[e + 1]), make_float2(-m2.x, -m2.y));
    const float2 r = __fmul2_rn(t, pair_of<VW>(k, e));
    v[e] = r.x;
    v[e + 1] = r.y;
  }
}
// c <- a * b + c and c <- a * b, element by element.
template <int VW>
__device__ __forceinline__ void fma_pairs(const float (&a)[VW], const float (&b)[VW], float (&c)[VW]) {
#pragma unroll
  for (int e = 0; e < VW; e += 2) {
    const float2 r = __ffma2_rn(make_float2(a[e], a[e + 1]), make_float2(b[e], b[e + 1]), make_float2(c[e], c[e + 1]));
    c[e] = r.x;
    c[e + 1] = r.y;
  }
}

// f(e, c, g) for the channels c (and their groups g) of the VW elements from c on, modulo C.
template <int VW, typename F>
__device__ __forceinline__ void for_channels(int c, int C, int D, F f) {
  int g = c / D, in = c - g * D;
#pragma unroll
  for (int e = 0; e < VW; ++e) {
    f(e, c, g);
    if (++in == D) {
      in = 0;
      ++g;
    }
    if (++c == C) c = g = in = 0;
  }
}

// For each i < n: val(i, k, a, b) over k < terms, added up in a and b, then
// out(i, a, b) by one thread.  `lanes` neighbouring lanes (a power of two) share
// the terms of one i, as many as `threads` (whole warps, all calling) allow.
template <typename VAL, typename OUT>
__device__ __forceinline__ void sum_sets(int threads, int n, int terms, VAL val, OUT out) {
  int log = 0;
  while (log < 5 && (2 << log) * n <= threads && (2 << log) <= terms) ++log;
  const int lanes = 1 << log, l = threadIdx.x & (lanes - 1);
  for (int i0 = 0; i0 < n; i0 += threads >> log) {
    const int i = i0 + (threadIdx.x >> log);
    float a = 0.f, b = 0.f;
    if (i < n) {
#pragma unroll 4
      for (int k = l; k < terms; k += lanes) val(i, k, a, b);
    }
    for (int o = lanes >> 1; o > 0; o >>= 1) {
      a += __shfl_xor_sync(0xffffffffu, a, o);
      b += __shfl_xor_sync(0xffffffffu, b, o);
    }
    if (i < n && l == 0) out(i, a, b);
  }
}

// The median of three values: no single outlier moves it.
__device__ __forceinline__ float median3(float a, float b, float c) {
  return fmaxf(fminf(a, b), fminf(fmaxf(a, b), c));
}

// A centre for sums: the median, or 0 where that is no farther from it than the three
// spread (half of it): the mean may then be much smaller than the values, and a sum
// about 0 keeps the digits that it has, where centre + distance would round at the
// centre's size (means of 8 to 20000 values of spread 1 around 0: 3e-8 off, 1.5e-8 so).
__device__ __forceinline__ float centre3(float a, float b, float c) {
  const float m = median3(a, b, c);
  return fabsf(m) <= 0.5f * (fmaxf(a, fmaxf(b, c)) - fminf(a, fminf(b, c))) ? 0.f : m;
}

// Whether sums were taken about a centre more than 4 standard deviations off the mean:
// `cut` = n (mean - centre)^2 against m2, what is left of the squares.  Up to there the
// rounding of the squares reaches the variance 17 times at most; beyond (two of three
// values outlying, 6e-9 of normal ones) it is worth summing again about the mean.
// False for infinities and NaN, where nothing is to be gained.
__device__ __forceinline__ bool far_off(float cut, float m2) { return cut > 16.f * m2 && cut < INFINITY; }

// A sum of squares that rounding took below zero is 0 (and NaN stays NaN).
__device__ __forceinline__ float not_negative(float q) { return q < 0.f ? 0.f : q; }

// The fused form (group_norm_fused.cu): small samples, and few tokens, in one
// launch.  *done says whether the shape and the alignment allow it; if not,
// nothing has been launched.
cudaError_t launch_group_norm_fused(const GroupNormArgs& a, cudaStream_t stream, int* launches, bool* done);
cudaError_t launch_group_norm_grad_fused(const GroupNormGradArgs& a, cudaStream_t stream, int* launches, bool* done);
// Whether the fused form takes a shape whose x and y are 16-byte aligned.
bool group_norm_fused_applies(DType t, int64_t N, int64_t S, int64_t C, int64_t G);
// Workspace bytes of the fused gradient: for 16-byte-aligned operands, or the most for any.
// *applies: whether it takes the aligned shape.
size_t group_norm_grad_fused_bytes(DType t, int64_t N, int64_t S, int64_t C, int64_t G, bool aligned, bool* applies);

}  // namespace ep

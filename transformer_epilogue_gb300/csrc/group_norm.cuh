// What the two forms of GroupNorm share: the activation and its derivative, and
// the interface of the fused form.
#pragma once

#include <cstdint>
#include <type_traits>

#include "device_common.cuh"
#include "ep_internal.h"

namespace ep {

// sigmoid(u) = 1 / (1 + e^-u).
//  float32: e^-u = 2^p (1 + c), p = -u log2(e) rounded and c what the rounding
//  and log2(e)'s own left out, times ln 2; the reciprocal by the hardware's
//  approximation and one Newton step: within 3 float32 ulp.  u is held in
//  [-87, 100], where nothing overflows: below, sigmoid is e^-87 = 1.6e-38.
//  16-bit results: 2^x and 1/x by the hardware approximations with p rounded,
//  errors of a few float32 ulp and |u| 2^-24, far below the results' rounding;
//  from u = -88.7 down 2^p overflows and sigmoid(u) is 0.
template <typename T>
__device__ __forceinline__ float sigmoid(float u) {
  if constexpr (std::is_same_v<T, float>) {
    constexpr float kL = 1.44269502162933349609375f;  // log2(e) rounded to float32
    constexpr float kLlo = 1.92596298909109e-08f;     // log2(e) - kL
    constexpr float kLn2 = 0.6931471805599453f;
    const float t = fmaxf(fminf(-u, 87.f), -100.f);
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

template <typename T>
__device__ __forceinline__ float silu(float u) {
  return u * sigmoid<T>(u);
}

// du of the definition.
template <typename T>
__device__ __forceinline__ float silu_grad(float dy, float u) {
  const float s = sigmoid<T>(u);
  return dy * (s * fmaf(u, 1.0f - s, 1.0f));
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

// A sum of squares that rounding took below zero is 0 (and NaN stays NaN).
__device__ __forceinline__ float not_negative(float q) { return q < 0.f ? 0.f : q; }

// The fused form (group_norm_fused.cu): a sample's slab of channels stays on
// chip between the statistics and the result.  *done says whether the shape and
// the alignment allow it; if not, nothing has been launched.
cudaError_t launch_group_norm_fused(const GroupNormArgs& a, int sm_count, cudaStream_t stream, int* launches,
                                    bool* done);
cudaError_t launch_group_norm_grad_fused(const GroupNormGradArgs& a, int sm_count, cudaStream_t stream,
                                         int* launches, bool* done);
// Workspace bytes of the fused gradient (0 where it does not apply).
size_t group_norm_grad_fused_bytes(DType t, int64_t N, int64_t S, int64_t C, int64_t G);

}  // namespace ep

// What the two forms of GroupNorm share: the activation and its derivative, and
// the interface of the fused form.
#pragma once

#include <cstdint>
#include <type_traits>

#include "device_common.cuh"
#include "ep_internal.h"

namespace ep {

// u * sigmoid(u).  float32: the library exponential and a rounded division.
// 16-bit results: 2^x and 1/x by the hardware approximations, whose errors (a
// few float32 ulp) are far below the result's rounding; below u = -88.7 the
// exponential overflows and the result, above -1e-36, is -0.
template <typename T>
__device__ __forceinline__ float silu(float u) {
  if constexpr (std::is_same_v<T, float>) return __fdiv_rn(u, 1.0f + expf(-u));
  else return u * dev::rcp_approx(1.0f + dev::ex2_approx(u * -dev::kLog2e));
}

template <typename T>
__device__ __forceinline__ float sigmoid(float u) {
  if constexpr (std::is_same_v<T, float>) return __fdiv_rn(1.0f, 1.0f + expf(-u));
  else return dev::rcp_approx(1.0f + dev::ex2_approx(u * -dev::kLog2e));
}

// du of the definition.
template <typename T, bool SILU>
__device__ __forceinline__ float act_grad(float dy, float u) {
  if constexpr (!SILU) return dy;
  const float s = sigmoid<T>(u);
  return dy * (s * fmaf(u, 1.0f - s, 1.0f));
}

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

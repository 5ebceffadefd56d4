// Internal interface of GroupNorm and BiasDropout, as ep_internal.h is that of the
// other ops (a header of its own: the kernels compiled from ep_internal.h do not
// depend on it).
#pragma once

#include "ep_internal.h"

namespace ep {

constexpr int64_t kMaxGroupNormChannels = int64_t(1) << 24;

struct GroupNormArgs {
  DType t;
  const void* x;
  const void* gamma;
  const void* beta;     // nullable
  void* y;
  float* mean;          // nullable: N * G float32 means
  float* inv;           // nullable: N * G float32 1/sqrt(var + eps)
  int64_t N, S, C, G;   // > 0, G divides C
  float eps;
  bool silu;
  void* workspace;      // group_norm_workspace_bytes (nullable where 0)
};

struct GroupNormGradArgs {
  DType t;
  const void* dy;
  const void* x;
  const void* gamma;
  const void* beta;     // nullable
  const float* mean;
  const float* inv;
  void* dx;
  void* dgamma;         // nullable
  void* dbeta;          // nullable
  int64_t N, S, C, G;   // > 0, G divides C
  bool silu;
  void* workspace;      // group_norm_grad_workspace_bytes
};

struct BiasDropoutArgs {
  DType t;
  const void* x;        // X, or dY for the gradient
  const void* bias;     // nullable
  const void* residual; // nullable
  void* y;              // Y, or dX for the gradient
  void* dbias;          // gradient only, nullable
  int64_t n;            // numel > 0
  int64_t C;            // last dimension > 0, divides n
  uint64_t seed;
  uint64_t offset;
  const uint64_t* offset_dev;  // nullable: added to offset when the kernel runs
  uint32_t last_kept;   // the largest word that keeps an element
  float scale;          // 1 / (1 - ratio)
  void* workspace;      // bias_dropout_grad_workspace_bytes, with dbias only
};

// As the launchers of ep_internal.h.
cudaError_t launch_group_norm(const GroupNormArgs& a, cudaStream_t stream, int* launches);
cudaError_t launch_group_norm_grad(const GroupNormGradArgs& a, cudaStream_t stream, int* launches);
cudaError_t launch_bias_dropout(const BiasDropoutArgs& a, int sm_count, cudaStream_t stream, int* launches);
cudaError_t launch_bias_dropout_grad(const BiasDropoutArgs& a, int sm_count, cudaStream_t stream, int* launches);

// Workspace bytes of those launches, by shape and type.  `aligned`: of the forms that
// take x, y (dy, x, dx) which start on 16-byte boundaries; else of any.
size_t group_norm_workspace_bytes(DType t, int64_t N, int64_t S, int64_t C, int64_t G, bool aligned);
size_t group_norm_grad_workspace_bytes(DType t, int64_t N, int64_t S, int64_t C, int64_t G, bool aligned);
size_t bias_dropout_grad_workspace_bytes(DType t, int64_t n, int64_t C);

cudaError_t group_norm_pipe_timeouts(unsigned int* count, bool clear);

}  // namespace ep

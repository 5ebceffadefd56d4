// Internal interface of the MX8 operators and the matrix product, as ep_internal.h
// is that of the other ops.
#pragma once

#include "ep_internal.h"

namespace ep {

struct QuantizeArgs {
  DType t;
  const void* x;        // x, or y of the other direction
  uint8_t* q;
  uint8_t* scales;
  int64_t rows, H;      // > 0
};

struct RmsNormArgs {
  DType t;
  const void* x;
  const void* skip;     // nullable
  const void* bias;     // nullable
  const void* gamma;
  uint8_t* q;
  uint8_t* scales;
  void* sum_out;        // nullable
  float* inv_out;       // nullable
  int64_t rows, H;      // > 0
  float eps;
};

struct RmsNormGradArgs {
  DType t;
  const void* dy;
  const void* s;        // the forward pass's sum
  const void* gamma;
  const float* inv;
  const void* dsum;     // nullable: the gradient that reaches the sum by other ways
  void* dx;
  void* dgamma;         // nullable
  void* dbias;          // nullable
  int64_t rows, H;      // > 0
  void* workspace;      // rms_norm_grad_workspace_bytes
};

// Activations; the codes of ep_activation.
enum Act : int { kActNone = 0, kActSilu = 1, kActRelu = 2, kActQuickGelu = 3, kActGelu = 4, kActFastGelu = 5 };

// out = act(A W^T + bias) + residual, A (M, K), W (N, K).
struct MatmulArgs {
  DType t;              // outputs, bias, residual; the operands too unless mx8
  bool mx8;             // A and W are E4M3 bytes with scales
  const void* a;
  const uint8_t* a_scales;
  const void* w;
  const uint8_t* w_scales;
  const void* bias;     // nullable
  const void* residual; // nullable
  void* y;
  void* z;              // nullable: the pre-activation, T or (z_scales) E4M3 bytes
  uint8_t* z_scales;
  int64_t M, N, K;      // M, N > 0, K >= 0
  int act;
  float alpha;
  void* workspace;      // matmul_workspace_bytes
};

struct MatmulGradArgs {
  DType t;
  const void* dy;
  const void* a;        // T, or (a_scales) E4M3 bytes
  const uint8_t* a_scales;
  const void* w;
  const void* z;        // T, or (z_scales) E4M3 bytes; nullable without an activation
  const uint8_t* z_scales;
  void* da;             // nullable
  void* dw;             // nullable
  void* dbias;          // nullable
  int64_t M, N, K;      // M, N, K >= 0
  int act;
  float alpha;
  void* workspace;      // matmul_grad_workspace_bytes
};

cudaError_t launch_quantize_mx8(const QuantizeArgs& a, int sm_count, cudaStream_t stream, int* launches);
cudaError_t launch_dequantize_mx8(const QuantizeArgs& a, int sm_count, cudaStream_t stream, int* launches);
cudaError_t launch_rms_norm_mx8(const RmsNormArgs& a, int sm_count, cudaStream_t stream, int* launches);
cudaError_t launch_rms_norm_grad(const RmsNormGradArgs& a, int sm_count, cudaStream_t stream, int* launches);
cudaError_t launch_matmul(const MatmulArgs& a, int sm_count, cudaStream_t stream, int* launches);
cudaError_t launch_matmul_grad(const MatmulGradArgs& a, int sm_count, cudaStream_t stream, int* launches);

size_t rms_norm_grad_workspace_bytes(DType t, int64_t rows, int64_t H);
// Workspace of launches whose operands start on 16-byte boundaries (`aligned`) or anywhere.
size_t matmul_workspace_bytes(bool mx8, int64_t M, int64_t N, int64_t K, bool aligned);
size_t matmul_grad_workspace_bytes(int64_t M, int64_t N, int64_t K, bool act, bool a_mx8, bool aligned);

// E4M3 rows with scales to T, rows `ld` elements apart (the tail behind a row's n elements set to 0).
cudaError_t launch_dequantize_pitched(DType t, const uint8_t* q, const uint8_t* scales, void* y, int64_t rows,
                                      int64_t n, int64_t ld, int sm_count, cudaStream_t stream, int* launches);

cudaError_t matmul_pipe_timeouts(unsigned int* count, bool clear);

}  // namespace ep

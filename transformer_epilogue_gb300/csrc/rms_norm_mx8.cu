// RMS norm with the residual's addition and an 8-bit output (MX8, mx8.cuh), its
// gradient, and rows of any values to and from MX8.
//
//   s = (x + skip) + bias, inv = 1 / sqrt(mean(s^2) + eps), y = s inv gamma, (q, scales) = MX8(y)
//   u = dY gamma, x^ = s inv:  ds = inv (u - x^ mean(u x^)) + dsum,  dgamma = sum dY x^,  dbias = sum ds
//
// All of it is bound by memory: a row is read once, held in registers across its
// reduction and written once.  A row belongs to TPR threads (whole warps), each
// with NF fragments of VW consecutive elements, TPR fragments apart: 8 elements
// where rows start on 16-byte boundaries, so that a group of 32 is four
// neighbouring lanes and its maximum two shuffles; else one element, so that a
// group is a warp.  Blocks keep gamma (and the bias, and the gradient's column
// sums) in registers and walk over rows, with the next row's loads issued
// before the present row's reduction: at 2 x 256 threads and 48 bytes each an SM
// has the 45 KB in flight that the memory's latency takes.  Rows too long for
// that are read twice by a block of 512 threads.
#include <algorithm>
#include <cstdint>

#include <cuda_runtime.h>

#include "column_walk.cuh"
#include "device_common.cuh"
#include "launch_util.h"
#include "mx8.cuh"
#include "mx8_internal.h"

namespace ep {
namespace {

using namespace dev;

constexpr int kRowThreads = 256;   // threads of a block of short rows
constexpr int kLongThreads = 512;  // threads of a block of one long row

// VW elements as they lie in memory.
template <typename T, int VW> struct Raw;
template <typename T> struct Raw<T, 1> {
  T v;
  __device__ __forceinline__ void zero() { v = from_float(0.f, T()); }
  __device__ __forceinline__ void stream(const T* p) { v = __ldcs(p); }
  __device__ __forceinline__ void keep(const T* p) { v = __ldg(p); }
  __device__ __forceinline__ void floats(float (&f)[1]) const { f[0] = to_float(v); }
};
template <typename T> struct Raw<T, 8> {
  static constexpr int W = sizeof(T) / 2;  // 16-byte words
  uint4 v[W];
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int i = 0; i < W; ++i) v[i] = make_uint4(0, 0, 0, 0);
  }
  __device__ __forceinline__ void stream(const T* p) {
#pragma unroll
    for (int i = 0; i < W; ++i) v[i] = ld16_stream(reinterpret_cast<const uint4*>(p) + i);
  }
  __device__ __forceinline__ void keep(const T* p) {
#pragma unroll
    for (int i = 0; i < W; ++i) v[i] = ld16_keep(reinterpret_cast<const uint4*>(p) + i);
  }
  __device__ __forceinline__ void floats(float (&f)[8]) const {
    if constexpr (W == 1) {
      Conv<T>::unpack(v[0], f);
    } else {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        float g[4];
        Conv<T>::unpack(v[i], g);
#pragma unroll
        for (int e = 0; e < 4; ++e) f[4 * i + e] = g[e];
      }
    }
  }
};

template <typename T, int VW>
__device__ __forceinline__ void store_row(T* p, const float (&f)[VW]) {
  if constexpr (VW == 1) {
    st1_stream(p, f[0]);
  } else if constexpr (sizeof(T) == 2) {
    st16_stream(p, Conv<T>::pack(f));
  } else {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const float g[4] = {f[4 * i], f[4 * i + 1], f[4 * i + 2], f[4 * i + 3]};
      st16_stream(p + 4 * i, Conv<T>::pack(g));
    }
  }
}

// MX8 of a fragment whose group is held by 32 / VW neighbouring lanes (all of
// them here; `in`: the fragment lies in the row).
template <int VW>
__device__ __forceinline__ void store_mx8(const float (&y)[VW], bool in, bool first, uint8_t* q, uint8_t* scale) {
  float amax = 0.f;
#pragma unroll
  for (int e = 0; e < VW; ++e) amax = fmaxf(amax, fabsf(y[e]));
#pragma unroll
  for (int o = 16 / VW; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
  const uint32_t b = mx_scale(amax);
  const float k = mx_factor(b);
  if (!in) return;
  if constexpr (VW == 8) {
    const uint2 w = make_uint2(e4m3x4(y[0] * k, y[1] * k, y[2] * k, y[3] * k),
                               e4m3x4(y[4] * k, y[5] * k, y[6] * k, y[7] * k));
    __stcs(reinterpret_cast<uint2*>(q), w);
  } else {
    *q = uint8_t(e4m3x2(y[0] * k, 0.f));
  }
  if (first) *scale = uint8_t(b);
}

// Sum over the TPR threads of a row.  `red`: 2 x the row's warps, taken in turn
// (`turn`), so that one barrier a row is enough.
__device__ __forceinline__ float row_sum(float v, float* red, int turn, int tpr, int slot) {
  v = warp_sum(v);
  if (tpr == 32) return v;
  const int warps = tpr >> 5;
  float* r = red + turn * warps;
  if ((threadIdx.x & 31) == 0) r[threadIdx.x >> 5] = v;
  asm volatile("bar.sync %0, %1;" ::"r"(1 + slot), "r"(tpr) : "memory");
  float t = 0.f;
  for (int i = 0; i < warps; ++i) t += r[i];
  return t;
}

// ---------------------------------------------------------------------------
// to MX8 and back
// ---------------------------------------------------------------------------

// i = row * d + col; 64-bit divisions only where 32 bits do not do.
__device__ __forceinline__ void split_index(uint64_t i, uint32_t d, uint64_t* row, uint32_t* col) {
  if ((i >> 32) == 0) {
    const uint32_t r = uint32_t(i) / d;
    *row = r;
    *col = uint32_t(i) - r * d;
  } else {
    *row = i / d;
    *col = uint32_t(i - *row * d);
  }
}

// A group of 32 to 32 / VW lanes, U groups each before the first is used.
template <typename T, int VW, int U>
__global__ void __launch_bounds__(kRowThreads)
k_quantize(const T* __restrict__ x, uint8_t* __restrict__ q, uint8_t* __restrict__ scales, int64_t items, uint32_t H,
           uint32_t G) {
  pdl_wait();
  pdl_trigger();
  constexpr int L = kMxGroup / VW;
  const int lane = threadIdx.x & (L - 1);
  const int64_t i0 = int64_t(blockIdx.x) * (kRowThreads / L * U) + threadIdx.x / L;
  Raw<T, VW> raw[U];
  int64_t off[U];
  bool in[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int64_t i = i0 + u * (kRowThreads / L);
    in[u] = false;
    off[u] = 0;
    if (i < items) {
      if (H % kMxGroup == 0) {
        off[u] = i * kMxGroup + lane * VW;
        in[u] = true;
      } else {
        uint64_t row;
        uint32_t g;
        split_index(uint64_t(i), G, &row, &g);
        const uint32_t col = g * kMxGroup + lane * VW;
        off[u] = int64_t(row) * H + col;
        in[u] = col < H;
      }
    }
    if (in[u]) raw[u].stream(x + off[u]);
    else raw[u].zero();
  }
#pragma unroll
  for (int u = 0; u < U; ++u) {
    float f[VW];
    raw[u].floats(f);
    store_mx8<VW>(f, in[u], lane == 0, q + off[u], scales + i0 + u * (kRowThreads / L));
  }
}

// Fragments of VW elements of rows `ld` apart (a multiple of VW); what lies behind a row's H elements is set to 0.
template <typename T, int VW, int U>
__global__ void __launch_bounds__(kRowThreads)
k_dequantize(const uint8_t* __restrict__ q, const uint8_t* __restrict__ scales, T* __restrict__ y, int64_t items,
             uint32_t H, uint32_t G, uint32_t ld) {
  pdl_wait();
  pdl_trigger();
  const uint32_t frags = ld / VW;
  const int64_t i0 = int64_t(blockIdx.x) * (kRowThreads * U) + threadIdx.x;
  uint2 raw[U];
  uint32_t b[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int64_t i = i0 + u * kRowThreads;
    raw[u] = make_uint2(0, 0);
    b[u] = 127;
    if (i >= items) continue;
    uint64_t row;
    uint32_t col;
    split_index(uint64_t(i), frags, &row, &col);
    col *= VW;
    if (col >= H) continue;
    const uint8_t* p = q + row * H + col;
    if constexpr (VW == 8) raw[u] = __ldcs(reinterpret_cast<const uint2*>(p));
    else raw[u].x = *p;
    b[u] = scales[row * G + col / kMxGroup];
  }
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int64_t i = i0 + u * kRowThreads;
    if (i >= items) continue;
    const float k = mx_value(b[u]);
    float f[VW];
    if constexpr (VW == 8) {
      const uint32_t w[4] = {raw[u].x, raw[u].x >> 16, raw[u].y, raw[u].y >> 16};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float2 t = e4m3_floats(w[e]);
        f[2 * e] = t.x * k;
        f[2 * e + 1] = t.y * k;
      }
    } else {
      f[0] = e4m3_floats(raw[u].x).x * k;
    }
    store_row<T, VW>(y + i * VW, f);
  }
}

// ---------------------------------------------------------------------------
// RMS norm to MX8
// ---------------------------------------------------------------------------

// Block (TPR, R): R rows at a time, rows blockIdx.x * R + y, then gridDim.x * R further on.
template <typename T, int VW, int NF>
__global__ void __launch_bounds__(kLongThreads)
k_norm(RmsNormArgs a) {
  __shared__ float red[2 * kLongThreads / 32];
  pdl_wait();
  pdl_trigger();
  const T* x = static_cast<const T*>(a.x);
  const T* skip = static_cast<const T*>(a.skip);
  const T* gamma = static_cast<const T*>(a.gamma);
  const T* bias = static_cast<const T*>(a.bias);
  T* sum_out = static_cast<T*>(a.sum_out);
  const int tpr = blockDim.x, slot = threadIdx.y;
  const int64_t step = int64_t(gridDim.x) * blockDim.y, groups = (a.H + kMxGroup - 1) / kMxGroup;
  constexpr bool kAhead = NF * VW <= 16;  // registers for a second row
  int64_t row = int64_t(blockIdx.x) * blockDim.y + slot;
  float* rred = red + slot * (2 * tpr / 32);
  const float inv_h = 1.0f / float(a.H);

  Raw<T, VW> gm[NF], bs[NF], rx[NF], rs[NF];
  int col[NF];
#pragma unroll
  for (int j = 0; j < NF; ++j) {
    col[j] = (j * tpr + int(threadIdx.x)) * VW;
    gm[j].zero();
    bs[j].zero();
    rx[j].zero();
    rs[j].zero();
    if (col[j] < a.H) {
      gm[j].keep(gamma + col[j]);
      if (bias != nullptr) bs[j].keep(bias + col[j]);
      if (kAhead && row < a.rows) {
        rx[j].stream(x + row * a.H + col[j]);
        if (skip != nullptr) rs[j].stream(skip + row * a.H + col[j]);
      }
    }
  }
  for (int turn = 0; row < a.rows; row += step, turn ^= 1) {
    if constexpr (!kAhead) {
#pragma unroll
      for (int j = 0; j < NF; ++j)
        if (col[j] < a.H) {
          rx[j].stream(x + row * a.H + col[j]);
          if (skip != nullptr) rs[j].stream(skip + row * a.H + col[j]);
        }
    }
    float s[NF][VW];
    float sq = 0.f;
#pragma unroll
    for (int j = 0; j < NF; ++j) {
      float t[VW];
      rx[j].floats(s[j]);
      rs[j].floats(t);
#pragma unroll
      for (int e = 0; e < VW; ++e) s[j][e] += t[e];
      if (bias != nullptr) {
        bs[j].floats(t);
#pragma unroll
        for (int e = 0; e < VW; ++e) s[j][e] += t[e];
      }
#pragma unroll
      for (int e = 0; e < VW; ++e) sq += s[j][e] * s[j][e];
    }
    const int64_t next = row + step;
    if (kAhead && next < a.rows) {
#pragma unroll
      for (int j = 0; j < NF; ++j)
        if (col[j] < a.H) {
          rx[j].stream(x + next * a.H + col[j]);
          if (skip != nullptr) rs[j].stream(skip + next * a.H + col[j]);
        }
    }
    if (sum_out != nullptr) {
#pragma unroll
      for (int j = 0; j < NF; ++j)
        if (col[j] < a.H) store_row<T, VW>(sum_out + row * a.H + col[j], s[j]);
    }
    const float inv = 1.0f / sqrtf(row_sum(sq, rred, turn, tpr, slot) * inv_h + a.eps);
    if (a.inv_out != nullptr && threadIdx.x == 0) a.inv_out[row] = inv;
#pragma unroll
    for (int j = 0; j < NF; ++j) {
      float g[VW];
      gm[j].floats(g);
#pragma unroll
      for (int e = 0; e < VW; ++e) s[j][e] *= inv * g[e];
      store_mx8<VW>(s[j], col[j] < a.H, col[j] % kMxGroup == 0, a.q + row * a.H + col[j],
                    a.scales + row * groups + col[j] / kMxGroup);
    }
  }
}

// One row a block, read twice (the second time out of L2), one element a lane.
template <typename T>
__device__ __forceinline__ float sum_at(const T* x, const T* skip, const T* bias, int64_t row, int64_t H, int64_t c) {
  float s = to_float(x[row * H + c]);
  if (skip != nullptr) s += to_float(skip[row * H + c]);
  if (bias != nullptr) s += to_float(bias[c]);
  return s;
}

template <typename T>
__global__ void __launch_bounds__(kLongThreads)
k_norm_long(RmsNormArgs a) {
  __shared__ float red[2 * kLongThreads / 32];
  pdl_wait();
  pdl_trigger();
  const T* x = static_cast<const T*>(a.x);
  const T* skip = static_cast<const T*>(a.skip);
  const T* gamma = static_cast<const T*>(a.gamma);
  const T* bias = static_cast<const T*>(a.bias);
  T* sum_out = static_cast<T*>(a.sum_out);
  const int64_t groups = (a.H + kMxGroup - 1) / kMxGroup;
  int turn = 0;
  for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x, turn ^= 1) {
    float sq = 0.f;
#pragma unroll 4
    for (int64_t c = threadIdx.x; c < a.H; c += kLongThreads) {
      const float s = sum_at(x, skip, bias, row, a.H, c);
      sq += s * s;
    }
    const float inv = 1.0f / sqrtf(row_sum(sq, red, turn, kLongThreads, 0) / float(a.H) + a.eps);
    if (a.inv_out != nullptr && threadIdx.x == 0) a.inv_out[row] = inv;
    // whole warps: a group's lanes stay together.  (sum_out may be x or skip: an element is read by the thread
    // that writes it, before it does.)
#pragma unroll 2
    for (int64_t c = threadIdx.x; c < groups * kMxGroup; c += kLongThreads) {
      float y[1] = {0.f};
      if (c < a.H) {
        const float s = sum_at(x, skip, bias, row, a.H, c);
        if (sum_out != nullptr) st1_stream(sum_out + row * a.H + c, s);
        y[0] = s * (inv * to_float(gamma[c]));
      }
      store_mx8<1>(y, c < a.H, c % kMxGroup == 0, a.q + row * a.H + c, a.scales + row * groups + c / kMxGroup);
    }
  }
}

// ---------------------------------------------------------------------------
// its gradient
// ---------------------------------------------------------------------------

// As k_norm; each thread also adds up its columns over the block's rows, and the
// block's sums go to `partial` (gridDim.x, H), dbias's behind dgamma's.
template <typename T, int VW, int NF, bool DB>
__global__ void __launch_bounds__(kLongThreads)
k_norm_grad(RmsNormGradArgs a) {
  extern __shared__ float cols[];  // R > 1: threads x NF x VW
  __shared__ float red[2 * kLongThreads / 32];
  pdl_wait();
  pdl_trigger();
  const T* dy = static_cast<const T*>(a.dy);
  const T* sp = static_cast<const T*>(a.s);
  const T* gamma = static_cast<const T*>(a.gamma);
  const T* dsum = static_cast<const T*>(a.dsum);
  T* dx = static_cast<T*>(a.dx);
  const int tpr = blockDim.x, slot = threadIdx.y, slots = blockDim.y;
  const int64_t step = int64_t(gridDim.x) * slots;
  constexpr bool kAhead = NF * VW <= 16;  // registers for a second row
  int64_t row = int64_t(blockIdx.x) * slots + slot;
  float* rred = red + slot * (2 * tpr / 32);
  const float inv_h = 1.0f / float(a.H);

  Raw<T, VW> gm[NF], ry[NF], rs[NF], rd[NF];
  float dg[NF][VW], db[NF][DB ? VW : 1];
  float inv = 0.f;
  int col[NF];
#pragma unroll
  for (int j = 0; j < NF; ++j) {
    col[j] = (j * tpr + int(threadIdx.x)) * VW;
    gm[j].zero();
    ry[j].zero();
    rs[j].zero();
    rd[j].zero();
#pragma unroll
    for (int e = 0; e < VW; ++e) {
      dg[j][e] = 0.f;
      if constexpr (DB) db[j][e] = 0.f;
    }
    if (col[j] < a.H) {
      gm[j].keep(gamma + col[j]);
      if (kAhead && row < a.rows) {
        ry[j].stream(dy + row * a.H + col[j]);
        rs[j].stream(sp + row * a.H + col[j]);
        if (dsum != nullptr) rd[j].stream(dsum + row * a.H + col[j]);
      }
    }
  }
  if (row < a.rows) inv = a.inv[row];
  for (int turn = 0; row < a.rows; row += step, turn ^= 1) {
    if constexpr (!kAhead) {
#pragma unroll
      for (int j = 0; j < NF; ++j)
        if (col[j] < a.H) {
          ry[j].stream(dy + row * a.H + col[j]);
          rs[j].stream(sp + row * a.H + col[j]);
          if (dsum != nullptr) rd[j].stream(dsum + row * a.H + col[j]);
        }
    }
    float u[NF][VW], xh[NF][VW];
    float dot = 0.f;
#pragma unroll
    for (int j = 0; j < NF; ++j) {
      float g[VW];
      ry[j].floats(u[j]);
      rs[j].floats(xh[j]);
      gm[j].floats(g);
#pragma unroll
      for (int e = 0; e < VW; ++e) {
        xh[j][e] *= inv;
        dg[j][e] += u[j][e] * xh[j][e];
        u[j][e] *= g[e];
        dot += u[j][e] * xh[j][e];
      }
    }
    Raw<T, VW> rc[NF];
#pragma unroll
    for (int j = 0; j < NF; ++j) rc[j] = rd[j];
    const float here = inv;
    const int64_t next = row + step;
    if (!kAhead && next < a.rows) inv = a.inv[next];
    if (kAhead && next < a.rows) {
#pragma unroll
      for (int j = 0; j < NF; ++j)
        if (col[j] < a.H) {
          ry[j].stream(dy + next * a.H + col[j]);
          rs[j].stream(sp + next * a.H + col[j]);
          if (dsum != nullptr) rd[j].stream(dsum + next * a.H + col[j]);
        }
      inv = a.inv[next];
    }
    const float c = row_sum(dot, rred, turn, tpr, slot) * inv_h;
#pragma unroll
    for (int j = 0; j < NF; ++j) {
      float d[VW];
      rc[j].floats(d);
      if constexpr (!kAhead) {  // made again from what was loaded, in place of registers that hold it
        float g[VW];
        ry[j].floats(u[j]);
        rs[j].floats(xh[j]);
        gm[j].floats(g);
#pragma unroll
        for (int e = 0; e < VW; ++e) {
          xh[j][e] *= here;
          u[j][e] *= g[e];
        }
      }
#pragma unroll
      for (int e = 0; e < VW; ++e) {
        d[e] += here * (u[j][e] - xh[j][e] * c);
        if constexpr (DB) db[j][e] += d[e];
      }
      if (col[j] < a.H) store_row<T, VW>(dx + row * a.H + col[j], d);
    }
  }
  float* partial = static_cast<float*>(a.workspace);
#pragma unroll
  for (int b = 0; b < (DB ? 2 : 1); ++b) {
    if (slots > 1) {  // the block's rows, added in the order of their slots
      __syncthreads();
#pragma unroll
      for (int j = 0; j < NF; ++j)
#pragma unroll
        for (int e = 0; e < VW; ++e) {
          float v = dg[j][e];
          if constexpr (DB) v = b == 0 ? v : db[j][e];
          cols[((slot * NF + j) * tpr + threadIdx.x) * VW + e] = v;
        }
      __syncthreads();
    }
    if (slot != 0) continue;
#pragma unroll
    for (int j = 0; j < NF; ++j) {
      if (col[j] >= a.H) continue;
      float* out = partial + (int64_t(b) * gridDim.x + blockIdx.x) * a.H + col[j];
#pragma unroll
      for (int e = 0; e < VW; ++e) {
        float v = dg[j][e];
        if constexpr (DB) v = b == 0 ? v : db[j][e];
        for (int r = 1; r < slots; ++r) v += cols[((r * NF + j) * tpr + threadIdx.x) * VW + e];
        out[e] = v;
      }
    }
  }
}

// Long rows: dX and the row's mean(u x^), which the column sums read.
template <typename T>
__global__ void __launch_bounds__(kLongThreads)
k_norm_grad_long(RmsNormGradArgs a, float* means) {
  __shared__ float red[2 * kLongThreads / 32];
  pdl_wait();
  pdl_trigger();
  const T* dy = static_cast<const T*>(a.dy);
  const T* sp = static_cast<const T*>(a.s);
  const T* gamma = static_cast<const T*>(a.gamma);
  int turn = 0;
  for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x, turn ^= 1) {
    const float inv = a.inv[row];
    float dot = 0.f;
#pragma unroll 4
    for (int64_t c = threadIdx.x; c < a.H; c += kLongThreads)
      dot += to_float(dy[row * a.H + c]) * to_float(gamma[c]) * (to_float(sp[row * a.H + c]) * inv);
    const float m = row_sum(dot, red, turn, kLongThreads, 0) / float(a.H);
    if (threadIdx.x == 0) means[row] = m;
  }
}

// Column sums of long rows, and dX beside them: lane = column, 8 warps share a
// chunk of rows.  (dX may be dY, the sum or dsum: an element is read by the
// thread that writes it, before it does.)
template <typename T>
__global__ void __launch_bounds__(256)
k_norm_grad_columns(RmsNormGradArgs a, const float* means, int64_t rows_per_chunk, float* partial) {
  __shared__ float part[2][8][32];
  pdl_wait();
  pdl_trigger();
  const T* dy = static_cast<const T*>(a.dy);
  const T* sp = static_cast<const T*>(a.s);
  const T* gamma = static_cast<const T*>(a.gamma);
  const T* dsum = static_cast<const T*>(a.dsum);
  T* dx = static_cast<T*>(a.dx);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t c = int64_t(blockIdx.x) * 32 + lane;
  const int64_t r0 = int64_t(blockIdx.y) * rows_per_chunk, r1 = min(r0 + rows_per_chunk, a.rows);
  float dg = 0.f, db = 0.f;
  if (c < a.H) {
    const float g = to_float(gamma[c]);
#pragma unroll 4
    for (int64_t r = r0 + warp; r < r1; r += 8) {
      const float inv = a.inv[r], y = to_float(dy[r * a.H + c]), xh = to_float(sp[r * a.H + c]) * inv;
      float d = inv * (y * g - xh * means[r]);
      if (dsum != nullptr) d += to_float(dsum[r * a.H + c]);
      dg += y * xh;
      db += d;
      st1_stream(dx + r * a.H + c, d);
    }
  }
  part[0][warp][lane] = dg;
  part[1][warp][lane] = db;
  __syncthreads();
  if (warp < 2 && c < a.H) {
    float v = 0.f;
    for (int w = 0; w < 8; ++w) v += part[warp][w][lane];
    partial[(int64_t(warp) * gridDim.y + blockIdx.y) * a.H + c] = v;
  }
}

// ---------------------------------------------------------------------------
// launches
// ---------------------------------------------------------------------------

bool on(const void* p, unsigned bytes) { return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) == 0; }

struct RowPlan {
  int vw, nf, tpr, slots;  // nf 0: the long form
};

// Fragments to threads: whole warps, of which as few lanes idle as the fragments a
// thread (1, 2, 4 .. most_nf) allow; among those within an eighth of the best, the
// most fragments, which leaves the fewest warps to join.
RowPlan plan_rows(int64_t H, bool vec, int most_nf) {
  RowPlan p{vec ? 8 : 1, 0, 0, 1};
  const int64_t frags = (H + p.vw - 1) / p.vw;
  int64_t best = INT64_MAX;
  for (int pass = 0; pass < 2; ++pass)
    for (int nf = 1; nf <= most_nf; nf *= 2) {
      const int64_t tpr = (frags + 32 * nf - 1) / (32 * nf) * 32;
      if (tpr > kLongThreads) continue;
      if (pass == 0) best = std::min(best, tpr * nf);
      else if (tpr * nf * 8 <= best * 9) p.nf = nf, p.tpr = int(tpr);
    }
  if (p.nf != 0) p.slots = std::max(1, kRowThreads / p.tpr);
  return p;
}

// 8 elements a fragment: two fragments a thread leave registers for the next row; four (rows of 8193 to 16384
// elements) are taken where two do not hold the row.
RowPlan plan_rows(int64_t H, bool vec) {
  if (!vec) return plan_rows(H, false, 8);
  const RowPlan p = plan_rows(H, true, 2);
  return p.nf != 0 ? p : plan_rows(H, true, 4);
}

template <typename F>
cudaError_t by_type(DType t, F f) {
  switch (t) {
    case DType::F32: return f(float());
    case DType::F16: return f(__half());
    default: return f(__nv_bfloat16());
  }
}

// How many blocks of a kernel that walks over rows: what fits on the device, no more than there are rows.
template <typename K>
cudaError_t walk_grid(K kernel, int threads, size_t smem, int sm_count, int64_t blocks, unsigned* grid) {
  int per_sm = 1;
  const cudaError_t e = resident_ctas(reinterpret_cast<const void*>(kernel), threads, smem, &per_sm);
  *grid = unsigned(std::max<int64_t>(1, std::min<int64_t>(blocks, int64_t(sm_count) * per_sm)));
  return e;
}

template <typename T, int VW, int NF>
cudaError_t norm_form(const RmsNormArgs& a, const RowPlan& p, int sm_count, cudaStream_t stream) {
  unsigned grid;
  cudaError_t e = walk_grid(k_norm<T, VW, NF>, p.tpr * p.slots, 0, sm_count, (a.rows + p.slots - 1) / p.slots, &grid);
  if (e != cudaSuccess) return e;
  return launch(k_norm<T, VW, NF>, dim3(grid), dim3(p.tpr, p.slots), 0, stream, a);
}

// The gradient's blocks: two to an SM (the sums that they leave are read again),
// a number that follows from the shape alone, as the workspace does.
int64_t grad_blocks(int64_t rows, int slots) { return std::min<int64_t>((rows + slots - 1) / slots, 2 * kPlanSms); }
int64_t grad_chunks(int64_t rows, int64_t H) {
  const int64_t want = std::max<int64_t>(1, 8 * kPlanSms / ((H + 31) / 32));
  return std::max<int64_t>(1, std::min({want, (rows + 31) / 32, int64_t(65535)}));
}

template <typename T, int VW, int NF, bool DB>
cudaError_t grad_form(const RmsNormGradArgs& a, const RowPlan& p, cudaStream_t stream) {
  const size_t smem = p.slots > 1 ? size_t(p.tpr) * p.slots * NF * VW * sizeof(float) : 0;
  return launch(k_norm_grad<T, VW, NF, DB>, dim3(unsigned(grad_blocks(a.rows, p.slots))), dim3(p.tpr, p.slots), smem,
                stream, a);
}

template <typename T, int VW, int NF>
cudaError_t grad_form(const RmsNormGradArgs& a, const RowPlan& p, cudaStream_t stream) {
  return a.dbias != nullptr ? grad_form<T, VW, NF, true>(a, p, stream) : grad_form<T, VW, NF, false>(a, p, stream);
}

}  // namespace

cudaError_t launch_quantize_mx8(const QuantizeArgs& a, int, cudaStream_t stream, int* launches) {
  const int64_t G = mx_groups(a.H), items = a.rows * G;
  const bool vec = a.H % 8 == 0 && on(a.x, 16) && on(a.q, 8);
  ++*launches;
  return by_type(a.t, [&](auto tag) {
    using T = decltype(tag);
    const T* x = static_cast<const T*>(a.x);
    auto run = [&](auto kernel, int per_block) {
      return launch(kernel, dim3(unsigned((items + per_block - 1) / per_block)), dim3(kRowThreads), 0, stream, x, a.q,
                    a.scales, items, uint32_t(a.H), uint32_t(G));
    };
    return vec ? run(k_quantize<T, 8, 4>, kRowThreads / 4 * 4) : run(k_quantize<T, 1, 8>, kRowThreads / 32 * 8);
  });
}

cudaError_t launch_dequantize_pitched(DType t, const uint8_t* q, const uint8_t* scales, void* y, int64_t rows,
                                      int64_t n, int64_t ld, int, cudaStream_t stream, int* launches) {
  const bool vec = n % 8 == 0 && ld % 8 == 0 && on(q, 8) && on(y, 16);
  const int64_t items = rows * (vec ? ld / 8 : ld);
  const int per_block = kRowThreads * 4;
  ++*launches;
  return by_type(t, [&](auto tag) {
    using T = decltype(tag);
    auto run = [&](auto kernel) {
      return launch(kernel, dim3(unsigned((items + per_block - 1) / per_block)), dim3(kRowThreads), 0, stream, q,
                    scales, static_cast<T*>(y), items, uint32_t(n), uint32_t(mx_groups(n)), uint32_t(ld));
    };
    return vec ? run(k_dequantize<T, 8, 4>) : run(k_dequantize<T, 1, 4>);
  });
}

cudaError_t launch_dequantize_mx8(const QuantizeArgs& a, int sm_count, cudaStream_t stream, int* launches) {
  return launch_dequantize_pitched(a.t, a.q, a.scales, const_cast<void*>(a.x), a.rows, a.H, a.H, sm_count, stream,
                                   launches);
}

cudaError_t launch_rms_norm_mx8(const RmsNormArgs& a, int sm_count, cudaStream_t stream, int* launches) {
  const bool vec = a.H % 8 == 0 && on(a.x, 16) && on(a.skip, 16) && on(a.gamma, 16) && on(a.bias, 16) && on(a.q, 8) &&
                   on(a.sum_out, 16);
  const RowPlan p = plan_rows(a.H, vec);
  ++*launches;
  return by_type(a.t, [&](auto tag) {
    using T = decltype(tag);
    if (p.nf == 0) {
      unsigned grid;
      cudaError_t e = walk_grid(k_norm_long<T>, kLongThreads, 0, sm_count, a.rows, &grid);
      if (e != cudaSuccess) return e;
      return launch(k_norm_long<T>, dim3(grid), dim3(kLongThreads), 0, stream, a);
    }
    if (vec) {
      if (p.nf == 1) return norm_form<T, 8, 1>(a, p, sm_count, stream);
      if (p.nf == 2) return norm_form<T, 8, 2>(a, p, sm_count, stream);
      return norm_form<T, 8, 4>(a, p, sm_count, stream);
    }
    if (p.nf == 1) return norm_form<T, 1, 1>(a, p, sm_count, stream);
    if (p.nf == 2) return norm_form<T, 1, 2>(a, p, sm_count, stream);
    if (p.nf == 4) return norm_form<T, 1, 4>(a, p, sm_count, stream);
    return norm_form<T, 1, 8>(a, p, sm_count, stream);
  });
}

size_t rms_norm_grad_workspace_bytes(DType, int64_t rows, int64_t H) {
  size_t most = 0;
  for (const bool vec : {false, true}) {
    if (vec && H % 8 != 0) continue;
    const RowPlan p = plan_rows(H, vec);
    const size_t sums = p.nf == 0 ? size_t(grad_chunks(rows, H)) : size_t(grad_blocks(rows, p.slots));
    most = std::max(most, 2 * sums * size_t(H) * 4 + (p.nf == 0 ? (size_t(rows) * 4 + 15) / 16 * 16 : 0));
  }
  return most;
}

cudaError_t launch_rms_norm_grad(const RmsNormGradArgs& a, int sm_count, cudaStream_t stream, int* launches) {
  const bool vec = a.H % 8 == 0 && on(a.dy, 16) && on(a.s, 16) && on(a.gamma, 16) && on(a.dsum, 16) && on(a.dx, 16);
  const RowPlan p = plan_rows(a.H, vec);
  return by_type(a.t, [&](auto tag) {
    using T = decltype(tag);
    float* partial = static_cast<float*>(a.workspace);
    int64_t terms;
    cudaError_t e;
    if (p.nf == 0) {
      const int64_t chunks = grad_chunks(a.rows, a.H), per = (a.rows + chunks - 1) / chunks;
      terms = (a.rows + per - 1) / per;
      float* means = partial + 2 * chunks * a.H;
      unsigned grid;
      e = walk_grid(k_norm_grad_long<T>, kLongThreads, 0, sm_count, a.rows, &grid);
      if (e != cudaSuccess) return e;
      e = launch(k_norm_grad_long<T>, dim3(grid), dim3(kLongThreads), 0, stream, a, means);
      if (e != cudaSuccess) return e;
      ++*launches;
      e = launch(k_norm_grad_columns<T>, dim3(unsigned((a.H + 31) / 32), unsigned(terms)), dim3(256), 0, stream, a,
                 static_cast<const float*>(means), per, partial);
    } else {
      terms = grad_blocks(a.rows, p.slots);
      if (vec) {
        e = p.nf == 1 ? grad_form<T, 8, 1>(a, p, stream)
                      : p.nf == 2 ? grad_form<T, 8, 2>(a, p, stream) : grad_form<T, 8, 4>(a, p, stream);
      } else {
        e = p.nf == 1   ? grad_form<T, 1, 1>(a, p, stream)
            : p.nf == 2 ? grad_form<T, 1, 2>(a, p, stream)
            : p.nf == 4 ? grad_form<T, 1, 4>(a, p, stream)
                        : grad_form<T, 1, 8>(a, p, stream);
      }
    }
    if (e != cudaSuccess) return e;
    ++*launches;
    if (a.dgamma == nullptr && a.dbias == nullptr) return cudaSuccess;
    const int buffers = a.dbias != nullptr ? 2 : 1;
    const unsigned blocks = unsigned(std::min<int64_t>((a.H + 31) / 32 * buffers, 65535));
    e = launch(k_channel_sums<T>, dim3(blocks), dim3(kSumsThreads), 0, stream, static_cast<const float*>(partial),
               terms, int64_t(1), a.H, buffers, static_cast<T*>(a.dgamma), static_cast<T*>(a.dbias));
    if (e == cudaSuccess) ++*launches;
    return e;
  });
}

}  // namespace ep

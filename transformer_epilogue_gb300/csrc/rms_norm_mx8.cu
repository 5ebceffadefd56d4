// RMS norm with the residual's addition and an 8-bit output (MX8, mx8.cuh), its
// gradient, and rows of any values to and from MX8.
//
//   s = (x + skip) + bias, inv = 1 / sqrt(mean(s^2) + eps), y = s inv gamma, (q, scales) = MX8(y)
//   u = dY gamma, x^ = s inv:  ds = inv (u - x^ mean(u x^)) + dsum,  dgamma = sum dY x^,  dbias = sum ds
//
// All of it is bound by memory: a row is read once, held in registers across its
// reduction and written once.  A row belongs to TPR threads, each with NF fragments of
// VW consecutive elements, TPR fragments apart: 8 elements where rows start on 16-byte
// boundaries, so that a group of 32 is four neighbouring lanes and its maximum two
// shuffles; else one element, so that a group is a warp.  Blocks walk over rows, with
// the next row's loads issued before the present row's reduction; what hides a row's
// latency (loads, reduction, stores: some 3000 cycles) is also the other rows of the
// SM's blocks.  Beside the memory it is the instructions that bind (38 an element at
// first, 70 % of the issue slots: bf16 16384 x 4096 in 88 us): products and sums go two
// to an instruction, indexes are 32-bit within a row (29 an element, 72 us, 96 % of the copy rate).
// Rows that came through a ring of bulk copies took 104 us, blocks of one row each 91.
// Rows too long for the registers are read twice by a block of 512 threads.
#include <algorithm>
#include <cstdint>
#include <cstring>
#include <type_traits>

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
  __device__ __forceinline__ void add_to(float (&f)[1]) const { f[0] += to_float(v); }
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
  // Elements lo <= e < hi, one by one.
  __device__ __forceinline__ void part(const T* p, int lo, int hi) {
    T t[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) t[e] = e >= lo && e < hi ? p[e] : from_float(0.f, T());
    memcpy(v, t, sizeof(v));
  }
  __device__ __forceinline__ void add_to(float (&f)[8]) const {
    if constexpr (W == 1) {
      add_raw<T, 8>(v[0], f);
    } else {
      float g[8];
      floats(g);
      add_pairs(f, g);
    }
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

// f *= k, f *= g, two to an instruction where there are two.
template <int VW>
__device__ __forceinline__ void scale_all(float (&f)[VW], float k) {
  if constexpr (VW == 1) f[0] *= k;
  else scale_pairs(f, k);
}
template <int VW>
__device__ __forceinline__ void mul_all(float (&f)[VW], const float (&g)[VW]) {
  if constexpr (VW == 1) {
    f[0] *= g[0];
  } else {
#pragma unroll
    for (int e = 0; e < VW; e += 2) {
      const float2 t = __fmul2_rn(make_float2(f[e], f[e + 1]), make_float2(g[e], g[e + 1]));
      f[e] = t.x;
      f[e + 1] = t.y;
    }
  }
}
// a + b c
template <int VW>
__device__ __forceinline__ void fma_all(float (&a)[VW], const float (&b)[VW], const float (&c)[VW]) {
  if constexpr (VW == 1) {
    a[0] = fmaf(b[0], c[0], a[0]);
  } else {
#pragma unroll
    for (int e = 0; e < VW; e += 2) {
      const float2 t =
          __ffma2_rn(make_float2(b[e], b[e + 1]), make_float2(c[e], c[e + 1]), make_float2(a[e], a[e + 1]));
      a[e] = t.x;
      a[e + 1] = t.y;
    }
  }
}
template <int VW>
__device__ __forceinline__ float sum_all(const float (&f)[VW]) {
  float t = f[0];
#pragma unroll
  for (int e = 1; e < VW; ++e) t += f[e];
  return t;
}

// MX8 of a fragment m whose group is held by 32 / VW neighbouring lanes (all of them
// here; `in`: the fragment lies in the row).  Returns the scale's byte.
template <int VW>
__device__ __forceinline__ uint32_t store_elements(float (&m)[VW], bool in, uint8_t* q) {
  float amax;
  if constexpr (VW == 1) {  // magnitudes compare as their bits do; NaN is left out
    const float f = fabsf(m[0]);
    amax = __uint_as_float(__reduce_max_sync(0xffffffffu, f == f ? __float_as_uint(f) : 0u));
  } else {
    amax = max3(fabsf(m[0]), fabsf(m[1]), fabsf(m[2]));
    amax = max3(amax, fabsf(m[3]), fabsf(m[4]));
    amax = max3(amax, fabsf(m[5]), fabsf(m[6]));
    amax = fmaxf(amax, fabsf(m[7]));
    amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
    amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
    amax = fmaxf(amax, 0.f);  // (eight NaN leave a NaN)
  }
  const uint32_t b = mx_scale(amax);
  scale_all(m, mx_factor(b));
  if (in) {
    if constexpr (VW == 8)
      __stcs(reinterpret_cast<uint2*>(q), make_uint2(e4m3x4(m[0], m[1], m[2], m[3]), e4m3x4(m[4], m[5], m[6], m[7])));
    else
      __stcs(q, uint8_t(e4m3x2(m[0], 0.f)));
  }
  return b;
}
template <int VW>
__device__ __forceinline__ void store_mx8(float (&m)[VW], bool in, bool first, uint8_t* q, uint8_t* scale) {
  const uint32_t b = store_elements<VW>(m, in, q);
  if (in && first) *scale = uint8_t(b);
}

// Sum over the blockDim.x threads of a row (a power of two below 32, or whole warps);
// the block's rows (blockDim.y) do it together.  `red`: 2 x the block's warps, taken
// in turn (`turn`), so that one barrier is enough.
__device__ __forceinline__ float row_sum(float v, float* red, int turn) {
  const int tpr = int(blockDim.x);
  for (int o = min(tpr, 32) / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  if (tpr <= 32) return v;
  const int warps = tpr >> 5;
  float* r = red + (turn * int(blockDim.y) + int(threadIdx.y)) * warps;
  if ((threadIdx.x & 31) == 0) r[threadIdx.x >> 5] = v;
  __syncthreads();
  float t = r[0];
  for (int i = 1; i < warps; ++i) t += r[i];
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

// A group of 32 to 32 / VW lanes, U groups each before the first is used.  VW 1: rows of
// a few groups, which would leave most of k_quantize_ragged's 256 elements empty (f16
// 60710 x 3: 7 us for 18).
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

// Rows that start on no 16-byte boundary: a warp takes 256 elements of a row, a group
// at a time, one lane an element (one division for all of them).
template <typename T>
__global__ void __launch_bounds__(kRowThreads)
k_quantize_ragged(const T* __restrict__ x, uint8_t* __restrict__ q, uint8_t* __restrict__ scales, int64_t items,
                  uint32_t H, uint32_t G) {
  pdl_wait();
  pdl_trigger();
  const uint32_t segs = (G + 7) / 8;
  const int lane = threadIdx.x & 31;
  const int64_t i = int64_t(blockIdx.x) * (kRowThreads / 32) + (threadIdx.x >> 5);
  if (i >= items) return;
  uint64_t row;
  uint32_t seg;
  split_index(uint64_t(i), segs, &row, &seg);
  const uint32_t left = H - seg * 256;  // elements from here on
  const T* xs = x + row * H + seg * 256 + lane;
  uint8_t* qs = q + row * H + seg * 256 + lane;
  Raw<T, 1> raw[8];
#pragma unroll
  for (int u = 0; u < 8; ++u) {
    if (32u * u + lane < left) raw[u].stream(xs + 32 * u);
    else raw[u].zero();
  }
  uint32_t mine = 0;
#pragma unroll
  for (int u = 0; u < 8; ++u) {
    float f[1];
    raw[u].floats(f);
    const uint32_t b = store_elements<1>(f, 32u * u + lane < left, qs + 32 * u);
    mine = lane == u ? b : mine;
  }
  if (lane < 8 && 32u * lane < left) scales[row * G + seg * 8 + lane] = uint8_t(mine);
}

template <typename T>
__global__ void __launch_bounds__(kRowThreads)
k_dequantize_ragged(const uint8_t* __restrict__ q, const uint8_t* __restrict__ scales, T* __restrict__ y, int64_t items,
                    uint32_t H, uint32_t G, uint32_t ld) {
  pdl_wait();
  pdl_trigger();
  const uint32_t segs = (ld + 255) / 256;
  const int lane = threadIdx.x & 31;
  const int64_t i = int64_t(blockIdx.x) * (kRowThreads / 32) + (threadIdx.x >> 5);
  if (i >= items) return;
  uint64_t row;
  uint32_t seg;
  split_index(uint64_t(i), segs, &row, &seg);
  const uint32_t c0 = seg * 256 + lane, g0 = seg * 8;
  const uint8_t* qs = q + row * H + c0;
  T* ys = y + row * ld + c0;
  const uint32_t mine = lane < 8 && g0 + lane < G ? __ldg(scales + row * G + g0 + lane) : 127u;
  uint32_t e[8];
#pragma unroll
  for (int u = 0; u < 8; ++u) e[u] = c0 + 32 * u < H ? __ldcs(qs + 32 * u) : 0u;
#pragma unroll
  for (int u = 0; u < 8; ++u) {
    const float k = mx_value(__shfl_sync(0xffffffffu, mine, u));
    if (c0 + 32 * u < ld) st1_stream(ys + 32 * u, e4m3_floats(e[u]).x * k);
  }
}

// Fragments of 8 elements of rows `ld` apart (a multiple of 8); what lies behind a row's H elements is set to 0.
template <typename T, int U>
__global__ void __launch_bounds__(kRowThreads)
k_dequantize(const uint8_t* __restrict__ q, const uint8_t* __restrict__ scales, T* __restrict__ y, int64_t items,
             uint32_t H, uint32_t G, uint32_t ld) {
  pdl_wait();
  pdl_trigger();
  constexpr int VW = 8;
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
    raw[u] = __ldcs(reinterpret_cast<const uint2*>(p));
    b[u] = scales[row * G + col / kMxGroup];
  }
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int64_t i = i0 + u * kRowThreads;
    if (i >= items) continue;
    const float k = mx_value(b[u]);
    float f[VW];
    const uint32_t w[4] = {raw[u].x, raw[u].x >> 16, raw[u].y, raw[u].y >> 16};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float2 v = e4m3_floats(w[e]);
      f[2 * e] = v.x * k;
      f[2 * e + 1] = v.y * k;
    }
    store_row<T, VW>(y + i * VW, f);
  }
}

// ---------------------------------------------------------------------------
// RMS norm to MX8
// ---------------------------------------------------------------------------

// Blocks that an SM holds at once, by the registers of a thread's elements (the
// present row's in float32, the next row's as loaded).
constexpr int norm_blocks(int elements, bool wide) { return wide ? 1 : elements <= 16 ? 4 : elements <= 24 ? 3 : 2; }

// Block (TPR, R): R rows at a time, the next R rows' loads issued before the present
// rows' reduction.
template <typename T, int VW, int NF, bool LONG>
__global__ void __launch_bounds__(LONG ? kLongThreads : kRowThreads, norm_blocks(NF * VW, LONG))
k_norm(const __grid_constant__ RmsNormArgs a, float inv_h) {
  __shared__ float red[2 * kLongThreads / 32];
  pdl_wait();
  pdl_trigger();
  const T* x = static_cast<const T*>(a.x);
  const T* skip = static_cast<const T*>(a.skip);
  const T* gamma = static_cast<const T*>(a.gamma);
  const T* bias = static_cast<const T*>(a.bias);
  T* sum_out = static_cast<T*>(a.sum_out);
  const int H = int(a.H), groups = (H + kMxGroup - 1) / kMxGroup, step = int(blockDim.x) * VW;
  const int c0 = int(threadIdx.x) * VW;
  const int64_t rows_step = int64_t(gridDim.x) * blockDim.y;
  Raw<T, VW> rx[NF], rs[NF];
  auto load = [&](int64_t row) {
    const int cols = row < a.rows ? H : 0;
    const int64_t at = row * H;
#pragma unroll
    for (int j = 0; j < NF; ++j) {
      const int c = c0 + j * step;
      if (c < cols) {
        rx[j].stream(x + at + c);
        if (skip != nullptr) rs[j].stream(skip + at + c);
      }
    }
  };
#pragma unroll
  for (int j = 0; j < NF; ++j) {
    rx[j].zero();
    rs[j].zero();
  }
  int64_t r0 = int64_t(blockIdx.x) * blockDim.y;
  load(r0 + threadIdx.y);
  for (int turn = 0; r0 < a.rows; r0 += rows_step, turn ^= 1) {
    const int64_t row = r0 + threadIdx.y, at = row * H;
    const int cols = row < a.rows ? H : 0;  // (rows behind the last take part in the barriers)
    float s[NF][VW], sq[VW] = {};
#pragma unroll
    for (int j = 0; j < NF; ++j) {
      const int c = c0 + j * step;
      rx[j].floats(s[j]);
      rs[j].add_to(s[j]);
      if (bias != nullptr && c < cols) {
        Raw<T, VW> b;
        b.keep(bias + c);
        b.add_to(s[j]);
      }
      fma_all(sq, s[j], s[j]);
    }
    if (r0 + rows_step < a.rows) load(row + rows_step);
    if (sum_out != nullptr) {
#pragma unroll
      for (int j = 0; j < NF; ++j)
        if (c0 + j * step < cols) store_row<T, VW>(sum_out + at + c0 + j * step, s[j]);
    }
    const float inv = rsqrtf(row_sum(sum_all(sq), red, turn) * inv_h + a.eps);
    if (a.inv_out != nullptr && cols != 0 && threadIdx.x == 0) a.inv_out[row] = inv;
    uint8_t* qr = a.q + at;
    uint8_t* scale = a.scales + row * groups;
    uint32_t mine = 0;  // one element a fragment: lane j stores the warp's j-th group's scale
#pragma unroll
    for (int j = 0; j < NF; ++j) {
      const int c = c0 + j * step;
      Raw<T, VW> gm;
      float g[VW];
      gm.zero();
      if (c < H) gm.keep(gamma + c);
      gm.floats(g);
      // (s inv) gamma in this order: s inv is at most sqrt(H), whatever s.  (inv taken into the scale's power of two
      // saved a multiplication in two elements and no time, and was infinite beside groups of 0.)
      scale_all(s[j], inv);
      mul_all(s[j], g);
      if constexpr (VW == 8) {
        store_mx8<VW>(s[j], c < cols, c % kMxGroup == 0, qr + c, scale + c / kMxGroup);
      } else {
        const uint32_t b = store_elements<VW>(s[j], c < cols, qr + c);
        mine = (c0 & 31) == j ? b : mine;
      }
    }
    if constexpr (VW == 1) {
      const int lane = c0 & 31, c = (c0 & ~31) + lane * step;
      if (lane < NF && c < cols) scale[c / kMxGroup] = uint8_t(mine);
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
    const float inv = rsqrtf(row_sum(sq, red, turn) / float(a.H) + a.eps);
    if (a.inv_out != nullptr && threadIdx.x == 0) a.inv_out[row] = inv;
    // whole warps: a group's lanes stay together.  (sum_out may be x or skip: an element is read by the thread
    // that writes it, before it does.)
#pragma unroll 2
    for (int64_t c = threadIdx.x; c < groups * kMxGroup; c += kLongThreads) {
      float y[1] = {0.f};
      if (c < a.H) {
        const float s = sum_at(x, skip, bias, row, a.H, c);
        if (sum_out != nullptr) st1_stream(sum_out + row * a.H + c, s);
        y[0] = s * inv * to_float(gamma[c]);
      }
      store_mx8<1>(y, c < a.H, c % kMxGroup == 0, a.q + row * a.H + c, a.scales + row * groups + c / kMxGroup);
    }
  }
}

// ---------------------------------------------------------------------------
// its gradient
// ---------------------------------------------------------------------------

// As k_norm; each thread adds up its columns, and the block's sums go to `partial`
// (gridDim.x, H), dbias's behind dgamma's.  AHEAD: the next rows' loads are issued
// before the present rows' reduction (where registers allow).
// ODD: rows that start on no 16-byte boundary, in a tensor that does.  A row's fragments
// begin at the boundary in front of it, and rows 8 apart lie alike, so with steps of
// 8 rows a thread keeps its columns; those of a fragment that are not in the row, at either
// end, are left out one by one.  (f16 13331 x 5034: 186 us for 488 element by element, bf16
// 26577 x 2525 with dbias 154 for 207.)
template <typename T, int VW, int NF, bool LONG, bool DB, bool ODD>
__global__ void __launch_bounds__(LONG ? kLongThreads : kRowThreads, LONG ? 1 : NF * VW <= 4 ? 4 : 2)
k_norm_grad(const __grid_constant__ RmsNormGradArgs a, float inv_h) {
  extern __shared__ float cols_sum[];  // blockDim.y > 1: threads x NF x VW
  __shared__ float red[2 * kLongThreads / 32];
  pdl_wait();
  pdl_trigger();
  constexpr bool AHEAD = NF * VW <= 16;
  const T* dy = static_cast<const T*>(a.dy);
  const T* sp = static_cast<const T*>(a.s);
  const T* gamma = static_cast<const T*>(a.gamma);
  const T* dsum = static_cast<const T*>(a.dsum);
  T* dx = static_cast<T*>(a.dx);
  const int64_t rows_step = int64_t(gridDim.x) * blockDim.y;
  const int H = int(a.H), step = int(blockDim.x) * VW;
  const int before = ODD ? int((int64_t(blockIdx.x) * blockDim.y + threadIdx.y) * H % (16 / int(sizeof(T)))) : 0;
  const int c0 = int(threadIdx.x) * VW - before;
  // (a fragment with columns below 0 or from the row's end on)
  auto ragged = [&](int c) { return ODD && (c < 0 || c + VW > H); };

  Raw<T, VW> gm[NF], ry[NF], rs[NF], rd[NF];
  float dg[NF][VW], db[DB ? NF : 1][VW];
  float inv = 0.f;
  auto load = [&](int64_t row) {
    const int cols = row < a.rows ? H : 0;
    inv = cols != 0 ? __ldg(a.inv + row) : 0.f;
#pragma unroll
    for (int j = 0; j < NF; ++j) {
      const int c = c0 + j * step;
      ry[j].zero();
      rs[j].zero();
      rd[j].zero();
      if (c >= cols || (ODD && cols == 0)) continue;
      if constexpr (ODD)
        if (ragged(c)) {
          ry[j].part(dy + row * H + c, -c, H - c);
          rs[j].part(sp + row * H + c, -c, H - c);
          if (dsum != nullptr) rd[j].part(dsum + row * H + c, -c, H - c);
          continue;
        }
      ry[j].stream(dy + row * H + c);
      rs[j].stream(sp + row * H + c);
      if (dsum != nullptr) rd[j].stream(dsum + row * H + c);
    }
  };
#pragma unroll
  for (int j = 0; j < NF; ++j) {
    gm[j].zero();
#pragma unroll
    for (int e = 0; e < VW; ++e) {
      dg[j][e] = 0.f;
      if constexpr (DB) db[j][e] = 0.f;
    }
    const int c = c0 + j * step;
    if constexpr (ODD) gm[j].part(gamma + c, -c, H - c);
    else if (c < H) gm[j].keep(gamma + c);
  }
  int turn = 0;
  int64_t r0 = int64_t(blockIdx.x) * blockDim.y;
  if (AHEAD) load(r0 + threadIdx.y);
  for (; r0 < a.rows; r0 += rows_step, turn ^= 1) {
    const int64_t row = r0 + threadIdx.y;
    const int cols = row < a.rows ? H : 0;
    if (!AHEAD) load(row);
    const float now = inv;
    float u[NF][VW], xh[NF][VW], dot[VW] = {};
    auto terms = [&](int j) {  // u = dY gamma, x^ = s inv; returns dY in u first
      ry[j].floats(u[j]);
      rs[j].floats(xh[j]);
      scale_all(xh[j], now);
    };
#pragma unroll
    for (int j = 0; j < NF; ++j) {
      float g[VW];
      terms(j);
      fma_all(dg[j], u[j], xh[j]);
      gm[j].floats(g);
      mul_all(u[j], g);
      fma_all(dot, u[j], xh[j]);
    }
    Raw<T, VW> rc[NF];
#pragma unroll
    for (int j = 0; j < NF; ++j) rc[j] = rd[j];
    if (AHEAD && r0 + rows_step < a.rows) load(row + rows_step);
    const float c = -row_sum(sum_all(dot), red, turn) * inv_h;
#pragma unroll
    for (int j = 0; j < NF; ++j) {
      if constexpr (!AHEAD) {  // made again from what was loaded, in place of registers that hold it
        float g[VW];
        terms(j);
        gm[j].floats(g);
        mul_all(u[j], g);
      }
      float d[VW], k[VW];
      rc[j].floats(d);
#pragma unroll
      for (int e = 0; e < VW; ++e) k[e] = c;
      fma_all(u[j], xh[j], k);  // u - x^ mean
#pragma unroll
      for (int e = 0; e < VW; ++e) k[e] = now;
      fma_all(d, u[j], k);
      if constexpr (DB) {
        if constexpr (VW == 1) db[j][0] += d[0];
        else add_pairs(db[j], d);
      }
      const int at = c0 + j * step;
      if (at >= cols || (ODD && cols == 0)) continue;
      if constexpr (ODD)
        if (ragged(at)) {
#pragma unroll
          for (int e = 0; e < VW; ++e)
            if (at + e >= 0 && at + e < H) st1_stream(dx + row * H + at + e, d[e]);
          continue;
        }
      store_row<T, VW>(dx + row * H + at, d);
    }
  }
  if (a.dgamma == nullptr && !DB) return;
  float* partial = static_cast<float*>(a.workspace);
  const int tpr = int(blockDim.x), slots = int(blockDim.y), lane = int(threadIdx.x);
#pragma unroll
  for (int b = 0; b < (DB ? 2 : 1); ++b) {
    if constexpr (ODD) {  // the block's rows do not lie alike: by column
      if (slots > 1) __syncthreads();
      float* mine = partial + (int64_t(b) * gridDim.x + blockIdx.x) * H;
      const int width = tpr * NF * VW;
#pragma unroll
      for (int j = 0; j < NF; ++j)
#pragma unroll
        for (int e = 0; e < VW; ++e) {
          float v = dg[j][e];
          if constexpr (DB) v = b == 0 ? v : db[j][e];
          const int c = c0 + j * step + e;
          if (c < 0 || c >= H) continue;
          if (slots > 1) cols_sum[int(threadIdx.y) * width + c] = v;
          else mine[c] = v;
        }
      if (slots == 1) continue;
      __syncthreads();
      for (int c = int(threadIdx.y) * tpr + lane; c < H; c += tpr * slots) {
        float v = cols_sum[c];
        for (int r = 1; r < slots; ++r) v += cols_sum[r * width + c];
        mine[c] = v;
      }
      continue;
    }
    if (slots > 1) {  // the block's rows, added in their order
      __syncthreads();
#pragma unroll
      for (int j = 0; j < NF; ++j)
#pragma unroll
        for (int e = 0; e < VW; ++e) {
          float v = dg[j][e];
          if constexpr (DB) v = b == 0 ? v : db[j][e];
          cols_sum[((int(threadIdx.y) * NF + j) * VW + e) * tpr + lane] = v;
        }
      __syncthreads();
    }
    if (threadIdx.y != 0) continue;
#pragma unroll
    for (int j = 0; j < NF; ++j) {
      const int c = c0 + j * step;
      if (c >= H) continue;
      float* out = partial + (int64_t(b) * gridDim.x + blockIdx.x) * H + c;
#pragma unroll
      for (int e = 0; e < VW; ++e) {
        float v = dg[j][e];
        if constexpr (DB) v = b == 0 ? v : db[j][e];
        for (int r = 1; r < slots; ++r) v += cols_sum[((r * NF + j) * VW + e) * tpr + lane];
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
    const float m = row_sum(dot, red, turn) / float(a.H);
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
  bool wide;               // more than kRowThreads threads
  bool odd;                // fragments of 8 in rows that start on no 16-byte boundary
};

// Fragments to threads: whole warps, of which as few lanes idle as the fragments a
// thread (1 to most_nf) allow; among those within an eighth of the best, `best_nf`
// fragments a thread, or else the most (which leaves the fewest warps to join).  Over
// 256 threads only with the most fragments.
void plan_threads(RowPlan* p, int64_t frags, int most_nf, int best_nf) {
  int64_t best = INT64_MAX;
  for (int pass = 0; pass < 2; ++pass)
    for (int nf = 1; nf <= most_nf; nf += nf < 4 ? 1 : 4) {
      const int64_t tpr = (frags + 32 * nf - 1) / (32 * nf) * 32;
      if (tpr > (nf == most_nf ? kLongThreads : kRowThreads)) continue;
      if (pass == 0) best = std::min(best, tpr * nf);
      else if (tpr * nf * 8 <= best * 9 && p->nf != best_nf) p->nf = nf, p->tpr = int(tpr);
    }
}

// 8 elements a fragment: rows of up to 128 elements share a warp (4, 8 or 16 threads
// each); else two fragments a thread and four blocks an SM where that wastes no lanes
// (bf16 16384 x 4096: 72 us, as four fragments and two blocks), up to four where it
// does or does not hold the row (f16 65536 x 768: 55 us with three, 86 with two; bf16
// 8192 x 8192: 73 with four).  The gradient has its column sums in
// registers too: two, and four where two do not hold the row.
RowPlan plan_rows(int64_t H, bool vec, bool grad) {
  RowPlan p{vec ? 8 : 1, 0, 0, 1, false, false};
  const int64_t frags = (H + p.vw - 1) / p.vw;
  if (vec && frags <= 16) {
    p.nf = 1;
    for (p.tpr = 4; p.tpr < frags; p.tpr *= 2) {}
  } else if (!vec) {
    plan_threads(&p, frags, 8, grad ? 4 : 8);
  } else {
    plan_threads(&p, frags, grad ? 2 : 4, 2);
    if (p.nf == 0) plan_threads(&p, frags, 4, 4);
  }
  if (p.nf == 0) return p;
  p.slots = std::max(1, kRowThreads / p.tpr);
  p.wide = p.tpr > kRowThreads;
  return p;
}

// The gradient's rows where the tensors (but not the rows) start on 16-byte boundaries: with up
// to 7 elements in front, in fragments of 8, from 96 elements a row and 8 million in all on
// (bf16 65536 x 129: 49 us for 78, f16 20000 x 1001 46 for 62, f32 40775 x 325 50 for 50; where the
// elements left out one by one and fewer warps are felt it loses: f32 2053 x 1001 with dbias 18 for 15, bf16
// 65536 x 101 28.7 for 27.5, and among those it takes f16 90000 x 97 37 for 35).
RowPlan plan_grad_rows(int64_t rows, int64_t H, bool aligned) {
  RowPlan p = plan_rows(H, aligned && H % 8 == 0, true);
  if (!aligned || H % 8 == 0 || H < 96 || rows * H < int64_t(8) << 20) return p;
  const RowPlan odd = plan_rows(H + 7, true, true);
  if (odd.nf == 0) return p;
  p = odd;
  p.odd = true;
  return p;
}

template <typename F>
cudaError_t by_type(DType t, F f) {
  switch (t) {
    case DType::F32: return f(float());
    case DType::F16: return f(__half());
    default: return f(__nv_bfloat16());
  }
}

// Blocks of a kernel that walks over rows: `per_sm` that its registers let an SM hold, no more than there are.
unsigned walk_grid(int64_t blocks, int sm_count, int per_sm) {
  return unsigned(std::max<int64_t>(1, std::min<int64_t>(blocks, int64_t(sm_count) * per_sm)));
}

template <typename T, int VW, int NF, bool LONG>
cudaError_t norm_form(const RmsNormArgs& a, const RowPlan& p, int sm_count, cudaStream_t stream) {
  const unsigned grid = walk_grid((a.rows + p.slots - 1) / p.slots, sm_count, norm_blocks(NF * VW, LONG));
  return launch(k_norm<T, VW, NF, LONG>, dim3(grid), dim3(p.tpr, p.slots), 0, stream, a, 1.0f / float(a.H));
}

// The gradient's blocks: as many as an SM's registers hold (up to 64, 112 and 128 a
// thread), but no more than leave sums of a fourth of what is read (their sums are
// written and read again); a number that follows from the shape alone, as the
// workspace does.  (f16 65536 x 768: 82 us with three blocks of 192 threads an SM, 103 with two.)
int64_t grad_blocks(int64_t rows, const RowPlan& p, int es) {
  const int elements = p.nf * p.vw, regs = elements <= 4 ? 64 : elements <= 8 ? 112 : 128;
  const int64_t per_sm = p.wide ? 1 : std::max(1, 65536 / (regs * p.tpr * p.slots));
  const int64_t most = std::max<int64_t>(kPlanSms / 2, rows * es / 16);
  const int64_t blocks = std::min({(rows + p.slots - 1) / p.slots, per_sm * kPlanSms, most});
  return p.odd ? (blocks + 7) / 8 * 8 : blocks;  // (steps of a multiple of 8 rows)
}
int64_t grad_chunks(int64_t rows, int64_t H) {
  const int64_t want = std::max<int64_t>(1, 8 * kPlanSms / ((H + 31) / 32));
  return std::max<int64_t>(1, std::min({want, (rows + 31) / 32, int64_t(65535)}));
}

template <typename T, int VW, int NF, bool LONG, bool DB, bool ODD>
cudaError_t grad_form(const RmsNormGradArgs& a, const RowPlan& p, cudaStream_t stream) {
  const size_t smem = p.slots > 1 ? size_t(p.tpr) * p.slots * NF * VW * sizeof(float) : 0;
  return launch(k_norm_grad<T, VW, NF, LONG, DB, ODD>, dim3(unsigned(grad_blocks(a.rows, p, dtype_size(a.t)))),
                dim3(p.tpr, p.slots), smem, stream, a, 1.0f / float(a.H));
}

template <typename T, int VW, int NF, bool LONG>
cudaError_t grad_form(const RmsNormGradArgs& a, const RowPlan& p, cudaStream_t stream) {
  if constexpr (VW == 8)
    if (p.odd)
      return a.dbias != nullptr ? grad_form<T, VW, NF, LONG, true, true>(a, p, stream)
                                : grad_form<T, VW, NF, LONG, false, true>(a, p, stream);
  return a.dbias != nullptr ? grad_form<T, VW, NF, LONG, true, false>(a, p, stream)
                            : grad_form<T, VW, NF, LONG, false, false>(a, p, stream);
}

// f(VW, NF, LONG) of the plan, as constants.
template <int V> using Int = std::integral_constant<int, V>;
template <bool GRAD, typename F>
cudaError_t by_plan(const RowPlan& p, F f) {
  using std::false_type;
  using std::true_type;
  if (p.vw == 8) {
    if (p.nf == 1) return f(Int<8>(), Int<1>(), false_type());
    if constexpr (GRAD) {
      if (p.nf == 2) return p.wide ? f(Int<8>(), Int<2>(), true_type()) : f(Int<8>(), Int<2>(), false_type());
      return f(Int<8>(), Int<4>(), true_type());
    } else {
      if (p.nf == 2) return f(Int<8>(), Int<2>(), false_type());
      if (p.nf == 3) return f(Int<8>(), Int<3>(), false_type());
      return p.wide ? f(Int<8>(), Int<4>(), true_type()) : f(Int<8>(), Int<4>(), false_type());
    }
  }
  if (p.nf == 1) return f(Int<1>(), Int<1>(), false_type());
  if (p.nf == 2) return f(Int<1>(), Int<2>(), false_type());
  if (p.nf == 3) return f(Int<1>(), Int<3>(), false_type());
  if (p.nf == 4) return f(Int<1>(), Int<4>(), false_type());
  return p.wide ? f(Int<1>(), Int<8>(), true_type()) : f(Int<1>(), Int<8>(), false_type());
}

}  // namespace

cudaError_t launch_quantize_mx8(const QuantizeArgs& a, int, cudaStream_t stream, int* launches) {
  const int64_t G = mx_groups(a.H);
  const bool vec = a.H % 8 == 0 && on(a.x, 16) && on(a.q, 8);
  ++*launches;
  return by_type(a.t, [&](auto tag) {
    using T = decltype(tag);
    auto run = [&](auto kernel, int64_t items, int per_block) {
      return launch(kernel, dim3(unsigned((items + per_block - 1) / per_block)), dim3(kRowThreads), 0, stream,
                    static_cast<const T*>(a.x), a.q, a.scales, items, uint32_t(a.H), uint32_t(G));
    };
    if (!vec && G < 4) return run(k_quantize<T, 1, 8>, a.rows * G, kRowThreads / 4);
    return vec ? run(k_quantize<T, 8, 4>, a.rows * G, kRowThreads)
               : run(k_quantize_ragged<T>, a.rows * ((G + 7) / 8), kRowThreads / 32);
  });
}

cudaError_t launch_dequantize_pitched(DType t, const uint8_t* q, const uint8_t* scales, void* y, int64_t rows,
                                      int64_t n, int64_t ld, int, cudaStream_t stream, int* launches) {
  const bool vec = n % 8 == 0 && ld % 8 == 0 && on(q, 8) && on(y, 16);
  ++*launches;
  return by_type(t, [&](auto tag) {
    using T = decltype(tag);
    auto run = [&](auto kernel, int64_t items, int per_block) {
      return launch(kernel, dim3(unsigned((items + per_block - 1) / per_block)), dim3(kRowThreads), 0, stream, q,
                    scales, static_cast<T*>(y), items, uint32_t(n), uint32_t(mx_groups(n)), uint32_t(ld));
    };
    return vec ? run(k_dequantize<T, 4>, rows * (ld / 8), kRowThreads * 4)
               : run(k_dequantize_ragged<T>, rows * ((ld + 255) / 256), kRowThreads / 32);
  });
}

cudaError_t launch_dequantize_mx8(const QuantizeArgs& a, int sm_count, cudaStream_t stream, int* launches) {
  return launch_dequantize_pitched(a.t, a.q, a.scales, const_cast<void*>(a.x), a.rows, a.H, a.H, sm_count, stream,
                                   launches);
}

cudaError_t launch_rms_norm_mx8(const RmsNormArgs& a, int sm_count, cudaStream_t stream, int* launches) {
  const bool vec = a.H % 8 == 0 && on(a.x, 16) && on(a.skip, 16) && on(a.gamma, 16) && on(a.bias, 16) && on(a.q, 8) &&
                   on(a.sum_out, 16);
  const RowPlan p = plan_rows(a.H, vec, false);
  ++*launches;
  return by_type(a.t, [&](auto tag) {
    using T = decltype(tag);
    if (p.nf == 0) {
      return launch(k_norm_long<T>, dim3(walk_grid(a.rows, sm_count, 3)), dim3(kLongThreads), 0, stream, a);
    }
    return by_plan<false>(p, [&](auto vw, auto nf, auto wide) {
      return norm_form<T, vw.value, nf.value, wide.value>(a, p, sm_count, stream);
    });
  });
}

size_t rms_norm_grad_workspace_bytes(DType t, int64_t rows, int64_t H) {
  size_t most = 0;
  for (const bool aligned : {false, true}) {
    const RowPlan p = plan_grad_rows(rows, H, aligned);
    const size_t sums = p.nf == 0 ? size_t(grad_chunks(rows, H)) : size_t(grad_blocks(rows, p, dtype_size(t)));
    most = std::max(most, 2 * sums * size_t(H) * 4 + (p.nf == 0 ? (size_t(rows) * 4 + 15) / 16 * 16 : 0));
  }
  return most;
}

cudaError_t launch_rms_norm_grad(const RmsNormGradArgs& a, int sm_count, cudaStream_t stream, int* launches) {
  const bool aligned = on(a.dy, 16) && on(a.s, 16) && on(a.gamma, 16) && on(a.dsum, 16) && on(a.dx, 16);
  const RowPlan p = plan_grad_rows(a.rows, a.H, aligned);
  return by_type(a.t, [&](auto tag) {
    using T = decltype(tag);
    float* partial = static_cast<float*>(a.workspace);
    int64_t terms;
    cudaError_t e;
    if (p.nf == 0) {
      const int64_t chunks = grad_chunks(a.rows, a.H), per = (a.rows + chunks - 1) / chunks;
      terms = (a.rows + per - 1) / per;
      float* means = partial + 2 * chunks * a.H;
      e = launch(k_norm_grad_long<T>, dim3(walk_grid(a.rows, sm_count, 4)), dim3(kLongThreads), 0, stream, a, means);
      if (e != cudaSuccess) return e;
      ++*launches;
      e = launch(k_norm_grad_columns<T>, dim3(unsigned((a.H + 31) / 32), unsigned(terms)), dim3(256), 0, stream, a,
                 static_cast<const float*>(means), per, partial);
    } else {
      terms = grad_blocks(a.rows, p, dtype_size(a.t));
      e = by_plan<true>(p, [&](auto vw, auto nf, auto wide) {
        return grad_form<T, vw.value, nf.value, wide.value>(a, p, stream);
      });
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

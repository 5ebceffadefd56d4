// Walking a dense (rows, C) block by 16-byte fragments so that a thread always
// meets the same channels, for the kernels that need per-channel values (group
// norm's parameters) or per-channel sums (its gradients, the bias gradient of
// dropout), for every C and alignment.
//
// A fragment has VW elements.  Fragment columns repeat every
// lcm(C, VW) / VW = C / gcd(C, VW) fragments: a "walk row" of that many
// fragments (or a multiple of it, to fill a block) starts at the same channel
// every time, so the thread at fragment column j of every walk row sees the
// channels (j * VW + e) mod C.  A walk row is cut into tiles of at most
// kWalkThreads fragments, one thread each, and the walk rows into chunks.
//
// Where a block starts off a 16-byte boundary, by `off` elements, the walk
// starts at the boundary before it: element e of fragment f is the block's
// element f * VW + e - off, its channel is that modulo C, and the elements
// before 0 and from L on are left alone.  Only the first and the last fragment
// of a block can be partial.
#pragma once

#include <algorithm>
#include <cstdint>
#include <numeric>

#include "device_common.cuh"

namespace ep {

constexpr int kWalkThreads = 256;
constexpr int kPlanSms = 152;  // plans (and workspace sizes) depend on the shape alone

struct WalkPlan {
  int64_t row_frags;       // fragments in a walk row
  int64_t rows;            // walk rows of one block of L elements
  int64_t rows_per_chunk;
  int chunks;              // chunks of walk rows, >= 1
  int tiles;               // tiles of a walk row
  int tile_frags;          // fragments (threads) of a tile, the last may have fewer
  int threads;             // tile_frags rounded up to whole warps
  int64_t reps;            // times each channel occurs in a walk row
};

// `blocks` blocks of L elements each; chunks are made until about `ctas` CTAs
// have work, each of at least `min_rows` walk rows.
inline WalkPlan make_walk(int64_t L, int64_t C, int vw, int64_t blocks, int64_t ctas, int64_t min_rows) {
  WalkPlan p;
  const int64_t period = C / std::gcd(C, int64_t(vw));
  const int64_t total = (L + (vw - 1) + vw - 1) / vw;  // fragments, wherever the block starts
  // several periods side by side fill a block of threads (no more than there are)
  const int64_t fill = std::max<int64_t>(1, std::min(kWalkThreads / period, (total + period - 1) / period));
  p.row_frags = period * fill;
  p.reps = p.row_frags * vw / C;
  p.tiles = static_cast<int>((p.row_frags + kWalkThreads - 1) / kWalkThreads);
  p.tile_frags = static_cast<int>((p.row_frags + p.tiles - 1) / p.tiles);
  p.threads = (p.tile_frags + 31) / 32 * 32;
  p.rows = (total + p.row_frags - 1) / p.row_frags;
  const int64_t want = std::max<int64_t>(1, ctas / std::max<int64_t>(1, blocks * p.tiles));
  const int64_t most = std::max<int64_t>(1, p.rows / std::max<int64_t>(1, min_rows));
  const int64_t chunks = std::min(want, most);
  p.rows_per_chunk = (p.rows + chunks - 1) / chunks;
  p.chunks = static_cast<int>((p.rows + p.rows_per_chunk - 1) / p.rows_per_chunk);
  return p;
}

namespace dev {

// Elements [0, VW) of a fragment starting at element e0 of a block of L
// elements of T, as float32.  VEC: whole fragments are 16-byte aligned.
// Elements outside [0, L) give 0.
template <typename T, bool VEC>
__device__ __forceinline__ void load_frag(const T* block, int64_t e0, int64_t L, float (&v)[Vec16<T>::N]) {
  constexpr int VW = Vec16<T>::N;
  if (VEC && e0 >= 0 && e0 + VW <= L) {
    Conv<T>::unpack(ld16_stream(block + e0), v);
  } else {
#pragma unroll
    for (int e = 0; e < VW; ++e) v[e] = (e0 + e >= 0 && e0 + e < L) ? ld1_stream(block + e0 + e) : 0.f;
  }
}

template <typename T, bool VEC>
__device__ __forceinline__ void store_frag(T* block, int64_t e0, int64_t L, const float (&v)[Vec16<T>::N]) {
  constexpr int VW = Vec16<T>::N;
  if (VEC && e0 >= 0 && e0 + VW <= L) {
    st16_stream(block + e0, Conv<T>::pack(v));
  } else {
#pragma unroll
    for (int e = 0; e < VW; ++e)
      if (e0 + e >= 0 && e0 + e < L) st1_stream(block + e0 + e, v[e]);
  }
}

// Elements between the 16-byte boundary at or before p and p.
template <typename T>
__device__ __forceinline__ int misalignment(const T* p) {
  return static_cast<int>((reinterpret_cast<uintptr_t>(p) & 15u) / sizeof(T));
}

__device__ __forceinline__ float to_float(float v) { return v; }
__device__ __forceinline__ float to_float(__half v) { return __half2float(v); }
__device__ __forceinline__ float to_float(__nv_bfloat16 v) { return __bfloat162float(v); }

__device__ __forceinline__ float warp_sum(float x) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}

}  // namespace dev

namespace {

// Per-channel sums from per-CTA partial sums: partial[b][r][w] (b of `buffers`
// arrays, r < terms, w < reps * C) -> out_b[c] = sum over r and over the w = c
// mod C, in a fixed order, rounded once.  A block takes 32 channels; its warps
// share the terms.  Bound by the latency of its reads: partials are a few per
// cent of what the kernel before read.  Block `block` of `blocks`.
constexpr int kSumsThreads = 1024;

template <typename T>
__device__ __forceinline__ void channel_sums(const float* partial, int64_t terms, int64_t reps, int64_t C, int buffers,
                                             T* out0, T* out1, unsigned block, unsigned blocks) {
  __shared__ float part[kSumsThreads / 32][33];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const unsigned cblocks = unsigned((C + 31) / 32);
  for (unsigned job = block; job < cblocks * buffers; job += blocks) {
    const unsigned b = job / cblocks;
    const int64_t c = int64_t(job - b * cblocks) * 32 + lane;
    T* out = b == 0 ? out0 : out1;
    const int64_t n = terms * reps;  // (r, k) with w = c + k * C: a row of C values each
    const float* src = partial + int64_t(b) * n * C + c;
    float acc = 0.f;
    if (c < C && out != nullptr) {
#pragma unroll 10
      for (int64_t q = warp; q < n; q += kSumsThreads / 32) acc += __ldcg(src + q * C);
    }
    part[warp][lane] = acc;
    __syncthreads();
    // warp w adds up the columns of channel w
    const float s = dev::warp_sum(part[lane][warp]);
    const int64_t cw = int64_t(job - b * cblocks) * 32 + warp;
    if (lane == 0 && cw < C && out != nullptr) dev::st1_stream(out + cw, s);
    __syncthreads();
  }
}

template <typename T>
__global__ void __launch_bounds__(kSumsThreads)
k_channel_sums(const float* partial, int64_t terms, int64_t reps, int64_t C, int buffers, T* out0, T* out1) {
  dev::pdl_wait();
  dev::pdl_trigger();
  channel_sums<T>(partial, terms, reps, C, buffers, out0, out1, blockIdx.x, gridDim.x);
}

}  // namespace
}  // namespace ep

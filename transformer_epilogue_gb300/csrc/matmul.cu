// Matrix product with bias, activation and residual in its epilogue, on the
// tcgen05 tensor cores, and what its gradient needs beside the products.
//
//   forward   z = A W^T + bias, y = act(z) + residual          A (M, K), W (N, K)
//   gradient  dz = dY act'(z), dA = dz W, dW = dz^T A, dbias = sum of dz's rows
//
// All three products are C(i, j) = sum_k R(i, k) Q(j, k), i the rows and j the
// columns of a row-major result, with R and Q either K-major (k contiguous:
// A, W, and dz in dA) or MN-major (i or j contiguous: W in dA, dz and A in dW);
// the tensor core reads both (umma.cuh), so nothing is transposed in memory.
// Sums are float32 in tensor memory; E4M3 operands bring a scale for each 32 of
// K, which the tensor core applies (kind::mxf8f6f4), so an 8-bit product has no
// rounding but its sums'.
//
// Two kernels:
//   k_mm_pair   large results: pairs of CTAs on tiles of 256 x 256 (8-bit: 256 x 192,
//     the scales need the tensor memory of the rest; 256 x 128 where those leave SMs
//     idle), one pair to two SMs, walking over the tiles.  A pair reads each operand byte once for two SMs, which halves what
//     shared memory and L2 deliver per product.  Two accumulators: a tile is written
//     while the next is computed.
//   k_mm_split  few rows, or few tiles: 128 columns of the result (the weights' rows,
//     on the tensor core's 128 lanes) x 16 to 128 rows, K cut among the CTAs of a
//     cluster, whose partial sums meet in distributed shared memory in the order of
//     their ranks: one launch, no scratch, the same result every time.
#include <algorithm>
#include <cstdint>
#include <mutex>

#include <cuda.h>
#include <cuda_runtime.h>

#include "activation.cuh"
#include "cluster_launch.h"
#include "column_walk.cuh"
#include "device_common.cuh"
#include "launch_util.h"
#include "mx8.cuh"
#include "mx8_internal.h"
#include "ring_tail.h"
#include "umma.cuh"

namespace ep {
namespace {

using namespace dev;

// ---------------------------------------------------------------------------
// epilogue
// ---------------------------------------------------------------------------

struct Epilogue {
  const void* bias;      // nullable
  const void* residual;  // nullable
  void* y;
  void* z;               // nullable: T, or (z_scales) E4M3
  uint8_t* z_scales;
  int64_t rows, cols;
  int act;
  float alpha;
  bool vec;              // rows of y, z and residual start on 16-byte boundaries (E4M3: of cols % 16 == 0 too)
  bool pairs;            // on 4-byte boundaries (E4M3: on 2-byte boundaries)
  bool vec_bias;
};

// ---------------------------------------------------------------------------
// the scales of 8-bit operands
//
// A K tile of 128 has 4 scales a row.  The tensor core wants the scales of rows
// l, l + 32, l + 64, l + 96 (4 bytes each) in lane l of tensor memory, so the
// shared-memory block that is copied there has 16 bytes for each l: one lane
// brings them together.  In global memory they are rows of `groups` bytes, of
// which a lane takes 16 (4 K tiles) at a time, two such quads ahead of the one
// in use: a quad's products take 0.8 us, a load that misses L2 as long.
// ---------------------------------------------------------------------------

struct ScaleRows {
  const uint8_t* p;
  int64_t rows, groups;
  int unit;  // bytes that can be loaded together: p and groups are multiples of it (16, 4, 2 or 1)
};

// The quads have a ring of their own in shared memory, with barriers of their own:
// one proxy fence and one arrival for 4 K tiles (a fence for each K tile held the
// products back to 0.46 us a tile, of 0.2).
constexpr int kScaleQuads = 3;
struct QuadRing : Ring {
  uint32_t buf = 0;  // which of two sets of tensor-memory columns
  __device__ __forceinline__ QuadRing() : Ring(kScaleQuads) {}
};

// 16 bytes from group g on of a row; 127 (the scale 1) outside, where the values are 0.
__device__ __forceinline__ void scale_quad(const ScaleRows& s, int64_t row, int64_t g, uint32_t (&w)[4]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) w[i] = 0x7F7F7F7Fu;
  if (row >= s.rows || g >= s.groups) return;
  const uint8_t* p = s.p + row * s.groups + g;
  if (s.unit == 16) {
    const uint4 v = __ldg(reinterpret_cast<const uint4*>(p));
    w[0] = v.x, w[1] = v.y, w[2] = v.z, w[3] = v.w;
  } else if (s.unit == 4) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (g + 4 * i < s.groups) w[i] = __ldg(reinterpret_cast<const uint32_t*>(p) + i);
  } else if (s.unit == 2) {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (g + 2 * i < s.groups)
        w[i / 2] = (w[i / 2] & ~(65535u << (16 * (i % 2)))) |
                   uint32_t(__ldg(reinterpret_cast<const uint16_t*>(p) + i)) << (16 * (i % 2));
  } else {
#pragma unroll
    for (int i = 0; i < 16; ++i)
      if (g + i < s.groups) w[i / 4] = (w[i / 4] & ~(255u << (8 * (i % 4)))) | uint32_t(__ldg(p + i)) << (8 * (i % 4));
  }
}

// A lane's quads of N rows 32 apart: the one in use and the next two.
template <int N>
struct ScaleAhead {
  uint32_t w[3][N][4];
  __device__ __forceinline__ void fetch(int at, const ScaleRows& s, int64_t row, int64_t g) {
#pragma unroll
    for (int j = 0; j < N; ++j) scale_quad(s, row + 32 * j, g, w[at][j]);
  }
  __device__ __forceinline__ void shift() {
#pragma unroll
    for (int j = 0; j < N; ++j)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        w[0][j][i] = w[1][j][i];
        w[1][j][i] = w[2][j][i];
      }
  }
  // K tile i of the quad in use, to the blocks of 512 bytes at `sf`.
  __device__ __forceinline__ void store(int i, uint4* sf, int lane) const {
#pragma unroll
    for (int b = 0; b < (N + 3) / 4; ++b) {
      uint32_t v[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) v[j] = 4 * b + j < N ? w[0][4 * b + j < N ? 4 * b + j : 0][i] : 0x7F7F7F7Fu;
      sf[32 * b + lane] = make_uint4(v[0], v[1], v[2], v[3]);
    }
  }
};

// ---------------------------------------------------------------------------
// large results: a pair of CTAs
// ---------------------------------------------------------------------------

constexpr int kLine = 128;                 // bytes of K (or of MN) in an operand line
constexpr int kTileM = 256;                // rows of a pair's tile
constexpr int kHalfM = kTileM / 2;
constexpr int kOperandM = kHalfM * kLine;  // bytes of a CTA's half of R
constexpr int kEpiWarps = 8;
constexpr int kPairThreads = (4 + kEpiWarps) * 32;
constexpr int kStaging = 4096;             // bytes an epilogue warp has to turn rows around
constexpr int kRaster = 8;                 // tiles of rows that are walked together

constexpr int kScaleColumns = 12;          // of tensor memory, for a K tile's scales
constexpr int kScaleSets = 8;              // K tiles whose scales are there

template <bool MX, int TN> struct PairShape {
  static constexpr int kTileN = TN;
  static constexpr int kHalfN = kTileN / 2;
  static constexpr int kOperandN = kHalfN * kLine;
  static constexpr int kStageBytes = kOperandM + kOperandN;
  static constexpr int kQBlocks = (TN + 127) / 128;
  static constexpr int kScaleBytes = MX ? 512 * (1 + kQBlocks) : 0;  // R's 128 rows and Q's
  static constexpr int kStages = TN == 128 ? 7 : MX ? 6 : 5;
  static constexpr int kChunk = TN == 192 ? 32 : 64;              // columns that a warp turns around at once
  static constexpr int kBarriers = 2 * kStages + 5;
  static constexpr int kSmem = 1024 + kStages * (kStageBytes + kScaleBytes) + kEpiWarps * (kStaging + 64 * 4) +
                               kBarriers * 8 + 16;
};

struct PairProduct {
  CUtensorMap r, q;
  CUtensorMap rs, qs;    // 8-bit: blocks of scales as k_arrange left them, by tile and K tile
  Epilogue epi;
  int64_t tiles_m, tiles_n;
  int k_tiles;
  int k_tile;            // elements
  bool r_mn, q_mn;
  uint32_t idesc;
};

// One product, or (TWO) two of the same kind whose tiles are walked one after the other:
// the two of a gradient, whose last tiles then leave SMs idle once, not twice (bf16
// 4096 x 1024 x 4096: 42 us for 49).  A kernel of its own: the choice of a tile's
// product costs one product alone a little (mx8 8192 x 4096 x 8192 165.5 us for 164.7).
struct PairArgs {
  PairProduct p[2];
  int64_t first, tiles;  // tiles of p[0], and of both
};

// Row-major scales to the blocks of 512 bytes that tensor memory takes, for the pair
// kernel's loads: block (tile, K tile) of `blocks` x 128 rows each, tiles `rows`
// rows apart.  A thread takes a quad of four rows.  (Warps of the pair kernel that did
// this held its products back to 0.41 us a K tile, where 0.2 is their time.)
struct ArrangeArgs {
  ScaleRows s[2];
  uint4* out[2];
  int64_t tiles[2];
  int rows[2], blocks[2];
  int k_tiles;
};
__global__ void __launch_bounds__(256) k_arrange(const __grid_constant__ ArrangeArgs a) {
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31;
  const int64_t quads = (a.k_tiles + 3) / 4, step = int64_t(gridDim.x) * 8;
#pragma unroll
  for (int o = 0; o < 2; ++o) {
    const int64_t work = a.tiles[o] * a.blocks[o] * quads;
    for (int64_t i = int64_t(blockIdx.x) * 8 + (threadIdx.x >> 5); i < work; i += step) {
      const int64_t q = i % quads, tb = i / quads, t = tb / a.blocks[o];
      const int b = int(tb - t * a.blocks[o]);
      uint32_t w[4][4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int in = 128 * b + 32 * j + lane;  // behind the tile's rows: never read by a product
        scale_quad(a.s[o], in < a.rows[o] ? t * a.rows[o] + in : a.s[o].rows, q * 16, w[j]);
      }
#pragma unroll
      for (int k = 0; k < 4; ++k)
        if (4 * q + k < a.k_tiles)
          a.out[o][((t * a.k_tiles + 4 * q + k) * a.blocks[o] + b) * 32 + lane] =
              make_uint4(w[0][k], w[1][k], w[2][k], w[3][k]);
    }
  }
}

// A staging row of NC 16-byte words; words are exchanged within a row so that
// neither one word of 32 rows nor NC words of 32 / NC rows meet in a bank.
template <int NC>
__device__ __forceinline__ uint8_t* staged(uint8_t* buf, int r, int c) {
  return buf + (r * NC + (c ^ ((r / (8 / NC)) & (NC - 1)))) * 16;
}

// A warp's 32 rows x NC words of 16 bytes, a row's words in neighbouring lanes, from
// global to shared memory and back.
template <int NC, typename E>
__device__ __forceinline__ void read_words(uint8_t* buf, const E* g, int64_t row0, int64_t col0, int64_t rows,
                                           int64_t cols, int lane) {
  constexpr int PER = 16 / sizeof(E);
  uint4 w[NC];
#pragma unroll
  for (int i = 0; i < NC; ++i) {
    const int64_t row = row0 + (i * 32 + lane) / NC, col = col0 + (i * 32 + lane) % NC * PER;
    w[i] = make_uint4(0, 0, 0, 0);
    if (row < rows && col < cols) w[i] = __ldcs(reinterpret_cast<const uint4*>(g + row * cols + col));
  }
#pragma unroll
  for (int i = 0; i < NC; ++i)
    *reinterpret_cast<uint4*>(staged<NC>(buf, (i * 32 + lane) / NC, (i * 32 + lane) % NC)) = w[i];
}
template <int NC, typename E>
__device__ __forceinline__ void write_words(uint8_t* buf, E* g, int64_t row0, int64_t col0, int64_t rows, int64_t cols,
                                            int lane) {
  constexpr int PER = 16 / sizeof(E);
#pragma unroll
  for (int i = 0; i < NC; ++i) {
    const int r = (i * 32 + lane) / NC, c = (i * 32 + lane) % NC;
    const int64_t row = row0 + r, col = col0 + c * PER;
    if (row < rows && col < cols)
      __stcs(reinterpret_cast<uint4*>(g + row * cols + col), *reinterpret_cast<const uint4*>(staged<NC>(buf, r, c)));
  }
}

// The same by smaller units U (an element, or two neighbours), a row's units to
// neighbouring lanes, for rows that start on no 16-byte boundary.  16 rows' loads
// are in flight together (with 8 in a loop that stored each, f16 1331 x 1001 x 771
// with a residual took 10 us longer).
template <int NC, typename U, bool LOAD>
__device__ __forceinline__ void turn_units(uint8_t* buf, U* g, int64_t row0, int64_t col0, int64_t rows, int64_t cols,
                                           int lane) {
  constexpr int PER = 16 / sizeof(U), N = NC * PER;
  const int high = int(min(rows - row0, int64_t(32)));
#pragma unroll 1
  for (int l0 = 0; l0 < N; l0 += 32) {
    const int l = l0 + lane;
    const bool in = l < N && col0 + l < cols;
    U* p = g + row0 * cols + col0 + l;
    auto at = [&](int r) { return reinterpret_cast<U*>(staged<NC>(buf, r, l / PER)) + l % PER; };
#pragma unroll 1
    for (int r0 = 0; r0 < high; r0 += 16) {
      if constexpr (LOAD) {
        U v[16];
#pragma unroll
        for (int r = 0; r < 16; ++r) v[r] = in && r0 + r < high ? p[(r0 + r) * cols] : U(0);
#pragma unroll
        for (int r = 0; r < 16; ++r)
          if (l < N) *at(r0 + r) = v[r];
      } else {
#pragma unroll 8
        for (int r = r0; r < min(r0 + 16, high); ++r)
          if (in) p[r * cols] = *at(r);
      }
    }
  }
}

template <int NC, typename E, typename E2>
__device__ __forceinline__ void write_rows(uint8_t* buf, void* g, int64_t row0, int64_t col0, int64_t rows, int64_t cols,
                                           bool vec, bool pairs, int lane) {
  if (vec) write_words<NC, E>(buf, static_cast<E*>(g), row0, col0, rows, cols, lane);
  else if (pairs) turn_units<NC, E2, false>(buf, static_cast<E2*>(g), row0, col0 / 2, rows, cols / 2, lane);
  else turn_units<NC, E, false>(buf, static_cast<E*>(g), row0, col0, rows, cols, lane);
}

// CW columns of a warp's 32 rows, from tensor memory to the outputs.  (A residual
// fetched a chunk ahead, into 32 more registers, took longer: bf16 8192 x 8192 x 256 in
// 100 us for 89.)
template <typename T, int CW>
__device__ __forceinline__ void pair_chunk(const Epilogue& e, uint8_t* buf, float* bs, uint32_t tmem, int64_t row0,
                                           int64_t col0, int lane) {
  if (row0 >= e.rows || col0 >= e.cols) return;
  const T* bias = static_cast<const T*>(e.bias);
#pragma unroll
  for (int i = 0; i < CW / 32; ++i) {
    const int64_t c = col0 + lane + 32 * i;
    bs[lane + 32 * i] = bias != nullptr && c < e.cols ? to_float(__ldg(bias + c)) : 0.f;
  }
  __syncwarp();
  auto load = [&](int h, float (&z)[32]) {
    uint32_t r[32];
    tmem_ld32(tmem + 32 * h, r);
    tmem_wait_ld(r);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float4 b = *reinterpret_cast<const float4*>(bs + 32 * h + 4 * i);
      z[4 * i] = __uint_as_float(r[4 * i]) + b.x;
      z[4 * i + 1] = __uint_as_float(r[4 * i + 1]) + b.y;
      z[4 * i + 2] = __uint_as_float(r[4 * i + 2]) + b.z;
      z[4 * i + 3] = __uint_as_float(r[4 * i + 3]) + b.w;
    }
  };
  constexpr int NC = CW / 8, NC8 = CW / 16;
  auto put = [&](int h, const float (&z)[32]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float f[8] = {z[8 * i], z[8 * i + 1], z[8 * i + 2], z[8 * i + 3],
                          z[8 * i + 4], z[8 * i + 5], z[8 * i + 6], z[8 * i + 7]};
      *reinterpret_cast<uint4*>(staged<NC>(buf, lane, 4 * h + i)) = Conv<T>::pack(f);
    }
  };
  if (e.z != nullptr) {
    const int64_t groups = (e.cols + kMxGroup - 1) / kMxGroup;
#pragma unroll
    for (int h = 0; h < CW / 32; ++h) {
      float z[32];
      load(h, z);
      if (e.z_scales == nullptr) {
        put(h, z);
      } else {  // a lane has the whole group (columns behind the last are 0)
        float amax = 0.f;
#pragma unroll
        for (int i = 0; i < 32; ++i) amax = fmaxf(amax, fabsf(z[i]));
        const uint32_t b = mx_scale(amax);
        const float k = mx_factor(b);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          uint32_t w[4];
#pragma unroll
          for (int j = 0; j < 4; ++j)
            w[j] = e4m3x4(z[16 * i + 4 * j] * k, z[16 * i + 4 * j + 1] * k, z[16 * i + 4 * j + 2] * k,
                          z[16 * i + 4 * j + 3] * k);
          *reinterpret_cast<uint4*>(staged<NC8>(buf, lane, 2 * h + i)) = make_uint4(w[0], w[1], w[2], w[3]);
        }
        if (row0 + lane < e.rows && col0 + 32 * h < e.cols)
          e.z_scales[(row0 + lane) * groups + (col0 / 32 + h)] = uint8_t(b);
      }
    }
    __syncwarp();
    if (e.z_scales == nullptr)
      write_rows<NC, uint16_t, uint32_t>(buf, e.z, row0, col0, e.rows, e.cols, e.vec, e.pairs, lane);
    else
      write_rows<NC8, uint8_t, uint16_t>(buf, e.z, row0, col0, e.rows, e.cols, e.vec && e.cols % 16 == 0, e.pairs, lane);
    __syncwarp();
  }
  if (e.residual != nullptr) {
    void* r = const_cast<void*>(e.residual);
    if (e.vec) read_words<NC>(buf, static_cast<const T*>(e.residual), row0, col0, e.rows, e.cols, lane);
    else if (e.pairs) turn_units<NC, uint32_t, true>(buf, static_cast<uint32_t*>(r), row0, col0 / 2, e.rows, e.cols / 2, lane);
    else turn_units<NC, uint16_t, true>(buf, static_cast<uint16_t*>(r), row0, col0, e.rows, e.cols, lane);
    __syncwarp();
  }
#pragma unroll
  for (int h = 0; h < CW / 32; ++h) {
    float z[32];
    load(h, z);
    if (e.act != kActNone) by_act(e.act, [&](auto tag) {
#pragma unroll
      for (int i = 0; i < 32; ++i) z[i] = act_value<decltype(tag)::value>(z[i], e.alpha);
    });
    if (e.residual != nullptr) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        float f[8];
        Conv<T>::unpack(*reinterpret_cast<const uint4*>(staged<NC>(buf, lane, 4 * h + i)), f);
#pragma unroll
        for (int j = 0; j < 8; ++j) z[8 * i + j] += f[j];
      }
    }
    put(h, z);
  }
  __syncwarp();
  write_rows<NC, uint16_t, uint32_t>(buf, e.y, row0, col0, e.rows, e.cols, e.vec, e.pairs, lane);
  __syncwarp();
}

// Where tile `t` of the walk lies: kRaster tiles of rows together, column by column.
__device__ __forceinline__ void tile_place(int64_t t, int64_t tiles_m, int64_t tiles_n, int64_t* m, int64_t* n) {
  const int64_t band = t / (kRaster * tiles_n), first = band * kRaster;
  const int64_t high = min(tiles_m - first, int64_t(kRaster)), in = t - band * kRaster * tiles_n;
  *n = in / high;
  *m = first + in - *n * high;
}

// Warps: 0 loads, 1 issues the products (of the pair's first CTA alone), 3 has the
// tensor memory, 4.. write.  Barriers of a stage: `full`
// (the first CTA's: both CTAs' bytes), `empty` (each CTA's: the products that read
// it are done); of an accumulator: `ready` (each
// CTA's), `taken` (the first CTA's: all epilogue warps of both).  A wait that
// runs out ends its role; the others run out in turn, copies in flight are waited
// for, and the CTAs leave together.
template <typename T, bool MX, int TN, bool TWO>
__global__ void __launch_bounds__(kPairThreads, 1)
k_mm_pair(const __grid_constant__ PairArgs a) {
  using S = PairShape<MX, TN>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* scales = smem + S::kStages * S::kStageBytes;
  uint8_t* staging = scales + S::kStages * S::kScaleBytes;
  float* bias = reinterpret_cast<float*>(staging + kEpiWarps * kStaging);
  uint64_t* full = reinterpret_cast<uint64_t*>(bias + kEpiWarps * 64);
  uint64_t* empty = full + S::kStages;
  uint64_t* ready = empty + S::kStages;
  uint64_t* taken = ready + 2;
  uint64_t* drained = taken + 2;
  uint32_t* tmem_at = reinterpret_cast<uint32_t*>(drained + 1);

  const int warp = warp_number(), lane = threadIdx.x & 31;
  const uint32_t rank = cluster_rank();
  if (threadIdx.x == 0) {
    for (int s = 0; s < S::kStages; ++s) {
      mbar_init(full + s, 1);
      mbar_init(empty + s, 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(ready + i, 1);
      mbar_init(taken + i, 2 * kEpiWarps);
    }
    mbar_init(drained, 1);
    mbar_init_fence();
    prefetch_map(&a.p[0].r);
    prefetch_map(&a.p[0].q);
  }
  if (warp == 3) tmem_alloc<true>(tmem_at, 512);
  __syncwarp();
  tmem_fence_before();
  cluster_sync();
  tmem_fence_after();
  const uint32_t tmem = *tmem_at;
  pdl_wait();
  pdl_trigger();

  const int64_t tiles = a.tiles, pairs = gridDim.x >> 1, pair = blockIdx.x >> 1;
  if (warp == 0) {
    Ring ring(S::kStages);
    int issued = 0;
    bool ok = true;
    for (int64_t t = pair; t < tiles && ok; t += pairs) {
      const PairProduct& p = a.p[TWO && t >= a.first ? 1 : 0];
      const bool r_mn = !MX && p.r_mn, q_mn = !MX && p.q_mn;
      int64_t tm, tn;
      tile_place(TWO && t >= a.first ? t - a.first : t, p.tiles_m, p.tiles_n, &tm, &tn);
      const int m = int(tm * kTileM) + int(rank) * kHalfM, n = int(tn * S::kTileN) + int(rank) * S::kHalfN;
      const int rs = int((tm * 2 + rank) * p.k_tiles), qs = int(tn * p.k_tiles);
      for (int k = 0; k < p.k_tiles; ++k, ring.next()) {
        if (issued >= S::kStages && !warp_wait(empty + ring.st, ring.phase ^ 1)) {
          ok = false;
          break;
        }
        const uint32_t bar = cluster_addr(smem_addr(full + ring.st), 0);
        const uint32_t dst = smem_addr(smem + ring.st * S::kStageBytes);
        const uint32_t sf = smem_addr(scales + ring.st * S::kScaleBytes);
        const int kk = k * p.k_tile;
        if (elect_one()) {
          if (rank == 0) mbar_arrive_expect_tx(full + ring.st, 2 * (S::kStageBytes + S::kScaleBytes));
          // an MN-major operand comes 64 rows at a time, a K-major one in as many boxes of 64 rows
#pragma unroll
          for (int c = 0; c < kHalfM / 64; ++c)
            tma_load<true>(dst + c * 8192, &p.r, bar, r_mn ? m + 64 * c : kk, r_mn ? kk : m + 64 * c);
          if constexpr (S::kHalfN % 64 == 0) {
#pragma unroll
            for (int c = 0; c < S::kHalfN / 64; ++c)
              tma_load<true>(dst + kOperandM + c * 8192, &p.q, bar, q_mn ? n + 64 * c : kk, q_mn ? kk : n + 64 * c);
          } else {
            tma_load<true>(dst + kOperandM, &p.q, bar, kk, n);
          }
          if constexpr (MX) {
            tma_load<true>(sf, &p.rs, bar, 0, rs + k);
            tma_load<true>(sf + 512, &p.qs, bar, 0, qs + k);
          }
        }
        __syncwarp();
        issued = min(issued + 1, S::kStages);
      }
    }
    // the last loads (of both CTAs) have landed before anyone leaves, and so have the arrivals that the
    // last products send to both CTAs' barriers (a load is waited for also behind one that did not land)
    if (rank == 0) last_uses(ring, issued, [&](int st, uint32_t parity) { return warp_wait(full + st, parity) || true; });
    last_uses(ring, issued, [&](int st, uint32_t parity) { return warp_wait(empty + st, parity); });
  } else if (warp == 1) {
    if (rank == 0) {
      Ring ring(S::kStages);
      uint32_t set = 0;
      bool ok = true;
      int64_t i = 0;
      for (int64_t t = pair; t < tiles && ok; t += pairs, ++i) {
        const PairProduct& p = a.p[TWO && t >= a.first ? 1 : 0];
        const bool r_mn = !MX && p.r_mn, q_mn = !MX && p.q_mn;
        const uint64_t rstep = operand_step(r_mn), qstep = operand_step(q_mn);
        const uint32_t idesc = p.idesc;
        const int k_tiles = p.k_tiles;
        const int acc = int(i & 1);
        if (i >= 2 && !warp_wait(taken + acc, uint32_t((i >> 1) - 1) & 1)) {
          ok = false;
          break;
        }
        tmem_fence_after();
        const uint32_t d = tmem + acc * S::kTileN;
        for (int k = 0; k < k_tiles; ++k, ring.next()) {
          if (!warp_wait(full + ring.st, ring.phase)) {
            ok = false;
            break;
          }
          tmem_fence_after();
          const uint32_t at = smem_addr(smem + ring.st * S::kStageBytes);
          uint64_t rd = operand_desc(at, r_mn), qd = operand_desc(at + kOperandM, q_mn);
          if (elect_one()) {
            if constexpr (MX) {
              // in turn to the columns of kScaleSets sets, so that the copies need not wait for products in flight
              const uint32_t sf = smem_addr(scales + ring.st * S::kScaleBytes);
              const uint32_t sfr = tmem + 2 * S::kTileN + set * kScaleColumns, sfq = sfr + 4;
              copy_scales<true>(sfr, scales_desc(sf));
              copy_scales<true>(sfq, scales_desc(sf + 512));
              if constexpr (S::kQBlocks == 2) copy_scales<true>(sfq + 4, scales_desc(sf + 1024));
#pragma unroll
              for (int j = 0; j < 4; ++j, rd += rstep, qd += qstep)
                mma_mx8<true>(d, rd, qd, idesc | mma_scale_byte(j), sfr, sfq, (k | j) != 0);
            } else {
#pragma unroll
              for (int j = 0; j < 4; ++j, rd += rstep, qd += qstep) mma_f16<true>(d, rd, qd, idesc, (k | j) != 0);
            }
            mma_commit<true>(empty + ring.st);
            if (k + 1 == k_tiles) mma_commit<true>(ready + acc);
          }
          __syncwarp();
          set = (set + 1) % kScaleSets;
        }
      }
      if (!ok) {  // products in flight end before the tensor memory is given back
        if (elect_one()) mma_commit<true>(drained, 1);
        __syncwarp();
        warp_wait(drained, 0);
      }
    }
  } else if (warp >= 4) {
    const int w = warp - 4;
    uint8_t* buf = staging + w * kStaging;
    int64_t i = 0;
    for (int64_t t = pair; t < tiles; t += pairs, ++i) {
      const int acc = int(i & 1);
      if (!warp_wait(ready + acc, uint32_t(i >> 1) & 1)) break;
      tmem_fence_after();
      const PairProduct& p = a.p[TWO && t >= a.first ? 1 : 0];
      int64_t tm, tn;
      tile_place(TWO && t >= a.first ? t - a.first : t, p.tiles_m, p.tiles_n, &tm, &tn);
      const int64_t row0 = tm * kTileM + rank * kHalfM + 32 * (w & 3);
      const uint32_t at = tmem + acc * S::kTileN + (uint32_t(32 * (w & 3)) << 16);
      for (int c = (w >> 2) * S::kHalfN; c < ((w >> 2) + 1) * S::kHalfN; c += S::kChunk)
        pair_chunk<T, S::kChunk>(p.epi, buf, bias + w * 64, at + c, row0, tn * S::kTileN + c, lane);
      tmem_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_cluster(cluster_addr(smem_addr(taken + acc), 0));
    }
  }
  __syncwarp();
  tmem_fence_before();
  cluster_sync();
  tmem_fence_after();
  if (warp == 3) tmem_free<true>(tmem, 512);
}

// ---------------------------------------------------------------------------
// few rows or few tiles: K cut among the CTAs of a cluster
// ---------------------------------------------------------------------------

constexpr int kSplitThreads = 256;
constexpr int kSplitN = 128;                  // columns of the result
constexpr int kOperandQ = kSplitN * kLine;
constexpr int kSplitMostRows = 128;
constexpr int kSplitBudget = 110 * 1024;      // two CTAs an SM
constexpr int kSplitMostStages = 6;
constexpr int kSplitQuadBytes = 4 * 1024;     // scales of 4 K tiles: Q's 128 rows and R's, 512 bytes each

struct SplitArgs {
  CUtensorMap r, q;
  ScaleRows rs, qs;
  Epilogue epi;
  int64_t tiles_m;
  int tile_m;            // rows: 16, 32, 64 or 128
  int k_tiles, k_tile;
  int stages;
  bool sums_apart;
  bool r_mn, q_mn;
  uint32_t idesc;
};

// VW neighbouring elements of T as float32: one 16-byte access, or one element.
template <typename T, int VW>
__device__ __forceinline__ void put_out(T* p, const float (&z)[VW]) {
  if constexpr (VW == 8) st16_stream(p, Conv<T>::pack(z));
  else st1_stream(p, z[0]);
}

// The sums of a CTA's share of the rows, over the cluster's ranks in their order, and
// its outputs.  A thread has VW columns (8 where rows start on 16-byte boundaries,
// else 1: then a warp writes 32 neighbours) of U rows at a time, with the next U rows'
// residuals in flight; the columns of a group of 32 belong to 32 / VW neighbouring
// lanes.  A small loop on purpose: run once and unrolled (16 rows a turn), the
// instructions' own way from memory took 20 to 30 us.
template <typename T, int VW, int U>
__device__ __forceinline__ void finish_rows(const Epilogue& e, const float* sums, int splits, int share, int64_t first,
                                            int64_t n0, bool bad) {
  constexpr int PER_ROW = kSplitN / VW, ROWS = kSplitThreads / PER_ROW;
  const int c = int(threadIdx.x) % PER_ROW * VW;
  const int64_t col = n0 + c, groups = (e.cols + kMxGroup - 1) / kMxGroup;
  const int left = int(min(int64_t(share), e.rows - first));  // rows that are there
  const int high = col < e.cols && !bad ? left : 0;           // .. of this thread's columns
  const T* residual = e.residual != nullptr ? static_cast<const T*>(e.residual) + first * e.cols + col : nullptr;
  T* y = static_cast<T*>(e.y) + first * e.cols + col;
  float bias[VW] = {};
  if (e.bias != nullptr && col < e.cols) {
    const T* b = static_cast<const T*>(e.bias) + col;
    if (VW == 8 && e.vec_bias) {
      Frag<T, VW> f;
      f.load_keep(b);
#pragma unroll
      for (int i = 0; i < VW; ++i) bias[i] = f.v[i];
    } else {
#pragma unroll
      for (int i = 0; i < VW; ++i) bias[i] = to_float(__ldg(b + i));
    }
  }
  Frag<T, VW> next[U];
  auto fetch = [&](int r0) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
#pragma unroll
      for (int i = 0; i < VW; ++i) next[u].v[i] = 0.f;
      if (residual != nullptr && r0 + u * ROWS < high) next[u].load_stream(residual + int64_t(r0 + u * ROWS) * e.cols);
    }
  };
  // (all lanes of a warp go through the same number of turns: a shuffle takes them all)
  const int mine = int(threadIdx.x) / PER_ROW;
  fetch(mine);
#pragma unroll 1
  for (int t = 0; t < left; t += ROWS * U) {
    float z[U][VW], res[U][VW];
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int i = 0; i < VW; ++i) res[u][i] = next[u].v[i];
    fetch(t + mine + ROWS * U);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int r = t + mine + u * ROWS;
      const float* at = sums + r * kSplitN + c;
#pragma unroll
      for (int i = 0; i < VW; ++i) z[u][i] = bias[i];
      if (r >= share) continue;
      float f[VW] = {};
#pragma unroll 1
      for (int s = 0; s < splits; ++s, at += share * kSplitN) {
        if constexpr (VW == 8) {
          const float4 lo = *reinterpret_cast<const float4*>(at), hi = *reinterpret_cast<const float4*>(at + 4);
          const float g[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
          add_pairs(f, g);
        } else {
          f[0] += *at;
        }
      }
#pragma unroll
      for (int i = 0; i < VW; ++i) z[u][i] += f[i];
    }
    if (e.z != nullptr) {
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int r = t + mine + u * ROWS;
        const bool in = r < high;
        const int64_t row = first + r, at = row * e.cols + col;
        if (e.z_scales == nullptr) {
          if (in) put_out<T, VW>(static_cast<T*>(e.z) + at, z[u]);
        } else {
          float amax = 0.f;
          if (in) {
#pragma unroll
            for (int i = 0; i < VW; ++i) amax = fmaxf(amax, fabsf(z[u][i]));
          }
#pragma unroll
          for (int o = 16 / VW; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
          const uint32_t b = mx_scale(amax);
          const float k = mx_factor(b);
          if (in) {
            uint8_t* p = static_cast<uint8_t*>(e.z) + at;
            if constexpr (VW == 8)
              *reinterpret_cast<uint2*>(p) = make_uint2(e4m3x4(z[u][0] * k, z[u][1] * k, z[u][2] * k, z[u][3] * k),
                                                        e4m3x4(z[u][4] * k, z[u][5] * k, z[u][6] * k, z[u][7] * k));
            else
              *p = uint8_t(e4m3x2(z[u][0] * k, 0.f));
            if (c % kMxGroup == 0) e.z_scales[row * groups + col / kMxGroup] = uint8_t(b);
          }
        }
      }
    }
    if (e.act != kActNone)
      by_act(e.act, [&](auto tag) {
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
          for (int i = 0; i < VW; ++i) z[u][i] = act_value<decltype(tag)::value>(z[u][i], e.alpha);
      });
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int r = t + mine + u * ROWS;
#pragma unroll
      for (int i = 0; i < VW; ++i) z[u][i] += res[u][i];
      if (r < high) put_out<T, VW>(y + int64_t(r) * e.cols, z[u]);
    }
  }
}

// Warps: 0 loads, 1 issues the products, 2 and 3 bring the scales (3 has the tensor
// memory too); then all of them write.
template <typename T, bool MX>
__global__ void __launch_bounds__(kSplitThreads, 2)
k_mm_split(const __grid_constant__ SplitArgs a) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  __shared__ uint64_t full[kSplitMostStages], empty[kSplitMostStages], sfull[kScaleQuads], sempty[kScaleQuads], done;
  __shared__ uint32_t tmem_at;
  __shared__ uint32_t failed[8], failed_here;  // by rank; this CTA's
  const int stage_bytes = kOperandQ + a.tile_m * kLine;
  uint8_t* scales = smem + a.stages * stage_bytes;  // kScaleQuads x kSplitQuadBytes
  // (rank, row, column) sums in float32, of the rows that this CTA finishes: in memory of their own, so that the
  // others need not wait for this CTA's products before they send theirs; of 128 rows where the stages were
  float* sums = reinterpret_cast<float*>(a.sums_apart ? scales + (MX ? kScaleQuads * kSplitQuadBytes : 0) : smem);

  const int warp = warp_number(), lane = threadIdx.x & 31;
  uint32_t splits;
  asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(splits));
  const uint32_t rank = cluster_rank();
  const int64_t tile = blockIdx.x / splits;
  const int64_t m0 = tile % a.tiles_m * a.tile_m, n0 = tile / a.tiles_m * kSplitN;
  // K tiles of this CTA: whole quads of them, as the scales come
  const int unit = MX ? 4 : 1, units = (a.k_tiles + unit - 1) / unit;
  const int k0 = int(int64_t(units) * rank / splits) * unit,
            k1 = min(int(int64_t(units) * (rank + 1) / splits) * unit, a.k_tiles);
  const uint32_t columns = MX ? 256 : a.tile_m < 32 ? 32 : a.tile_m;
  const bool r_mn = !MX && a.r_mn, q_mn = !MX && a.q_mn;
  if (threadIdx.x == 0) {
    for (int s = 0; s < 8; ++s) failed[s] = 0;
    failed_here = 0;
    for (int s = 0; s < a.stages; ++s) {
      mbar_init(full + s, 1);
      mbar_init(empty + s, 1);
    }
    for (int i = 0; i < kScaleQuads; ++i) {
      mbar_init(sfull + i, 2);
      mbar_init(sempty + i, 1);
    }
    mbar_init(&done, 1);
    mbar_init_fence();
    if (k0 < k1) {
      prefetch_map(&a.r);
      prefetch_map(&a.q);
    }
  }
  if (warp == 3) tmem_alloc<false>(&tmem_at, columns);
  __syncwarp();
  tmem_fence_before();
  __syncthreads();
  if (splits > 1) cluster_arrive();  // waited for in front of the first store to another CTA: it is there
  tmem_fence_after();
  const uint32_t tmem = tmem_at;
  pdl_wait();
  pdl_trigger();

  if (warp == 0) {
    Ring ring(a.stages);
    int issued = 0;
    const int m = int(m0), n = int(n0);
    for (int k = k0; k < k1; ++k, ring.next()) {
      if (issued >= a.stages && !warp_wait(empty + ring.st, ring.phase ^ 1)) break;
      const uint32_t bar = smem_addr(full + ring.st), dst = smem_addr(smem + ring.st * stage_bytes);
      const int kk = k * a.k_tile;
      if (elect_one()) {
        mbar_arrive_expect_tx(full + ring.st, stage_bytes);
#pragma unroll
        for (int c = 0; c < kSplitN / 64; ++c)
          tma_load<false>(dst + c * 8192, &a.q, bar, q_mn ? n + 64 * c : kk, q_mn ? kk : n + 64 * c);
        tma_load<false>(dst + kOperandQ, &a.r, bar, r_mn ? m : kk, r_mn ? kk : m);
        if (a.tile_m > 64) tma_load<false>(dst + kOperandQ + 8192, &a.r, bar, r_mn ? m + 64 : kk, r_mn ? kk : m + 64);
      }
      __syncwarp();
      issued = min(issued + 1, a.stages);
    }
    // the last loads have landed before the stages serve for anything else, the last products' arrivals before
    // the barriers' memory may
    last_uses(ring, issued, [&](int st, uint32_t parity) { return warp_wait(full + st, parity) || true; });
    last_uses(ring, issued, [&](int st, uint32_t parity) { return warp_wait(empty + st, parity); });
  } else if (warp == 1) {
    Ring ring(a.stages);
    QuadRing quad;
    const uint64_t rstep = operand_step(r_mn), qstep = operand_step(q_mn);
    bool ok = true;
    for (int k = k0; k < k1; ++k, ring.next()) {
      if ((MX && k % 4 == 0 && !warp_wait(sfull + quad.st, quad.phase)) || !warp_wait(full + ring.st, ring.phase)) {
        ok = false;
        break;
      }
      tmem_fence_after();
      const uint32_t at = smem_addr(smem + ring.st * stage_bytes);
      uint64_t qd = operand_desc(at, q_mn), rd = operand_desc(at + kOperandQ, r_mn);
      if (elect_one()) {
        if constexpr (MX) {  // a quad's scales at once, 8 columns a K tile behind the 128 of the sums, two sets in turn
          const uint32_t sft = tmem + kSplitMostRows + quad.buf * 32;
          if (k % 4 == 0) {
            for (int i = 0; i < 4 && k + i < k1; ++i) {
              const uint32_t sf = smem_addr(scales + quad.st * kSplitQuadBytes + i * 1024);
              copy_scales<false>(sft + i * 8, scales_desc(sf));
              copy_scales<false>(sft + i * 8 + 4, scales_desc(sf + 512));
            }
            mma_commit<false>(sempty + quad.st);
          }
          const uint32_t sfq = sft + k % 4 * 8, sfr = sfq + 4;
#pragma unroll
          for (int j = 0; j < 4; ++j, rd += rstep, qd += qstep)
            mma_mx8<false>(tmem, qd, rd, a.idesc | mma_scale_byte(j), sfq, sfr, k > k0 || j > 0);
        } else {
#pragma unroll
          for (int j = 0; j < 4; ++j, rd += rstep, qd += qstep) mma_f16<false>(tmem, qd, rd, a.idesc, k > k0 || j > 0);
        }
        mma_commit<false>(empty + ring.st);
      }
      __syncwarp();
      if (MX && k % 4 == 3) {
        quad.next();
        quad.buf ^= 1;
      }
    }
    if (elect_one()) mma_commit<false>(&done);
    __syncwarp();
    ok = warp_wait(&done, 0) && ok;
    if (!ok && lane == 0) failed_here = 1;
  } else if (MX && (warp == 2 || warp == 3)) {  // Q's scales and R's
    const ScaleRows& sr = warp == 2 ? a.qs : a.rs;
    const int64_t row = (warp == 2 ? n0 : m0) + lane;
    ScaleAhead<4> ahead;
#pragma unroll
    for (int i = 0; i < 3; ++i)
      if (k0 + 4 * i < k1) ahead.fetch(i, sr, row, int64_t(k0 / 4 + i) * 16);
    Ring ring(kScaleQuads);
    int issued = 0;
    for (int k = k0; k < k1; k += 4, ring.next()) {
      if (k - k0 >= 4 * kScaleQuads && !warp_wait(sempty + ring.st, ring.phase ^ 1)) break;
#pragma unroll
      for (int i = 0; i < 4; ++i)
        ahead.store(i, reinterpret_cast<uint4*>(scales + ring.st * kSplitQuadBytes + 1024 * i + (warp == 2 ? 0 : 512)),
                    lane);
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(sfull + ring.st);
      ahead.shift();
      if (k + 12 < k1) ahead.fetch(2, sr, row, int64_t(k / 4 + 3) * 16);
      issued = min(issued + 1, kScaleQuads);
    }
    last_uses(ring, issued, [&](int st, uint32_t parity) { return warp_wait(sempty + st, parity); });
  }
  __syncwarp();
  __syncthreads();  // the products are done, the stages free
  tmem_fence_after();

  // each row's sums to the CTA that finishes it
  const int half = a.tile_m / 2, share = a.tile_m / int(splits);
  if (splits > 1) {
    cluster_wait();
    if (!a.sums_apart) cluster_sync();  // everyone's products are done
    if (failed_here != 0 && threadIdx.x < splits) st_cluster(cluster_addr(smem_addr(&failed[rank]), threadIdx.x), 1u);
  }
  for (int c = (warp >> 2) * half; c < ((warp >> 2) + 1) * half; c += 8) {
    uint32_t v[8];
    tmem_ld8(tmem + c + (uint32_t(32 * (warp & 3)) << 16), v);
    tmem_wait_ld(v);
    const int col = 32 * (warp & 3) + lane;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint32_t f = k0 < k1 ? v[i] : 0u;
      if (splits == 1) {
        sums[(c + i) * kSplitN + col] = __uint_as_float(f);
      } else {
        const int to = (c + i) / share, r = (c + i) - to * share;
        st_cluster(cluster_addr(smem_addr(sums + (int(rank) * share + r) * kSplitN + col), to), f);
      }
    }
  }
  tmem_fence_before();
  if (splits > 1) cluster_sync();
  else __syncthreads();
  tmem_fence_after();
  if (warp == 3) tmem_free<false>(tmem, columns);
  bool bad = false;
  for (uint32_t s = 0; s < splits; ++s) bad |= (splits > 1 ? failed[s] : failed_here) != 0;
  const int64_t first = m0 + int64_t(rank) * share;
  if (a.epi.vec) finish_rows<T, 8, 1>(a.epi, sums, int(splits), share, first, n0, bad);
  else finish_rows<T, 1, 4>(a.epi, sums, int(splits), share, first, n0, bad);
}

// ---------------------------------------------------------------------------
// beside the products
// ---------------------------------------------------------------------------

// Rows of n elements to rows `ld` apart (the tail set to 0): operands whose rows do
// not start on 16-byte boundaries, up to two in one launch.  A warp copies 256
// elements of a row, neighbours to neighbouring lanes.
struct PitchArgs {
  const void* x[2];
  void* y[2];
  int64_t rows[2];
  uint32_t n[2], ld[2];
};
template <typename E>
__global__ void __launch_bounds__(256) k_pitch(const __grid_constant__ PitchArgs a) {
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31;
  const int64_t warps = int64_t(gridDim.x) * 8;
#pragma unroll
  for (int o = 0; o < 2; ++o) {
    const E* x = static_cast<const E*>(a.x[o]);
    E* y = static_cast<E*>(a.y[o]);
    const uint32_t n = a.n[o], ld = a.ld[o];
    const int64_t segs = (ld + 255) / 256;
    for (int64_t i = int64_t(blockIdx.x) * 8 + (threadIdx.x >> 5); i < a.rows[o] * segs; i += warps) {
      const int64_t r = i / segs;
      const uint32_t c0 = uint32_t(i - r * segs) * 256 + lane;
      E v[8];
#pragma unroll
      for (int u = 0; u < 8; ++u) v[u] = c0 + 32 * u < n ? __ldcs(x + r * n + c0 + 32 * u) : E(0);
#pragma unroll
      for (int u = 0; u < 8; ++u)
        if (c0 + 32 * u < ld) y[r * ld + c0 + 32 * u] = v[u];
    }
  }
}

// dz = dY act'(z) (rounded to T for the tensor cores, as dY itself was: a
// relative 2^-9 of bf16 that averages out over the sums), rows `ld` apart, and
// the column sums of dz before that rounding.  A lane has VW columns, the 8 warps
// share a chunk of rows, U rows at a time with the next U rows' loads in flight;
// bound by memory, and nearly by the slopes' 25 instructions an element.  ZM: z is
// absent, T, or MX8.
constexpr int kSlopeThreads = 256;
template <typename T, int VW, int ZM>
__global__ void __launch_bounds__(kSlopeThreads, 3)
k_act_slope(const T* __restrict__ dy, const void* __restrict__ zp, const uint8_t* __restrict__ z_scales,
            T* __restrict__ dz, int64_t rows, int64_t cols, int64_t ld, int64_t rows_per_chunk, int act, float alpha,
            float* __restrict__ partial, T* __restrict__ dbias) {
  constexpr int U = 2;
  __shared__ float part[8][32][VW + 1];
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t c = (int64_t(blockIdx.x) * 32 + lane) * VW, groups = (cols + kMxGroup - 1) / kMxGroup;
  const int64_t r0 = int64_t(blockIdx.y) * rows_per_chunk, r1 = min(r0 + rows_per_chunk, rows);
  struct Row {  // as loaded
    uint4 d, z;
    uint32_t scale;
  };
  Row next[U];
  auto load = [&](int64_t r) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t row = r + 8 * u;
      next[u].d = next[u].z = make_uint4(0, 0, 0, 0);
      next[u].scale = 127;
      if (row >= r1 || c >= cols) continue;
      const int64_t at = row * cols + c;
      if constexpr (VW == 8) {
        next[u].d = ld16_stream(dy + at);
        if constexpr (ZM == 1) next[u].z = ld16_stream(static_cast<const T*>(zp) + at);
        if constexpr (ZM == 2) {
          const uint2 q = __ldcs(reinterpret_cast<const uint2*>(static_cast<const uint8_t*>(zp) + at));
          next[u].z.x = q.x;
          next[u].z.y = q.y;
        }
      } else {
        next[u].d.x = __ldcs(reinterpret_cast<const uint16_t*>(dy) + at);
        if constexpr (ZM == 1) next[u].z.x = __ldcs(static_cast<const uint16_t*>(zp) + at);
        if constexpr (ZM == 2) next[u].z.x = __ldcs(static_cast<const uint8_t*>(zp) + at);
      }
      if constexpr (ZM == 2) next[u].scale = __ldg(z_scales + row * groups + c / kMxGroup);
    }
  };
  auto floats = [](uint4 v, float (&f)[VW]) {
    if constexpr (VW == 8) {
      Conv<T>::unpack(v, f);
    } else {
      const uint16_t h = uint16_t(v.x);
      f[0] = to_float(*reinterpret_cast<const T*>(&h));
    }
  };
  float sum[VW];
#pragma unroll
  for (int e = 0; e < VW; ++e) sum[e] = 0.f;
  by_act(act, [&](auto tag) {
    if (c >= ld) return;
    load(r0 + warp);
    for (int64_t r = r0 + warp; r < r1; r += 8 * U) {
      Row now[U];
#pragma unroll
      for (int u = 0; u < U; ++u) now[u] = next[u];
      if (r + 8 * U < r1) load(r + 8 * U);
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int64_t row = r + 8 * u;
        if (row >= r1) continue;
        float d[VW];
        floats(now[u].d, d);
        if constexpr (ZM != 0) {
          float z[VW];
          if constexpr (ZM == 1) {
            floats(now[u].z, z);
          } else {
            const float k = mx_value(now[u].scale);
            const uint32_t w[4] = {now[u].z.x, now[u].z.x >> 16, now[u].z.y, now[u].z.y >> 16};
#pragma unroll
            for (int e = 0; e < VW; e += 2) {
              const float2 t = e4m3_floats(w[e / 2]);
              z[e] = t.x * k;
              if constexpr (VW == 8) z[e + 1] = t.y * k;
            }
          }
#pragma unroll
          for (int e = 0; e < VW; ++e) d[e] *= act_slope<decltype(tag)::value>(z[e], alpha);
        }
#pragma unroll
        for (int e = 0; e < VW; ++e) sum[e] += d[e];
        if (dz != nullptr) {
          if constexpr (VW == 8) *reinterpret_cast<uint4*>(dz + row * ld + c) = Conv<T>::pack(d);
          else dz[row * ld + c] = from_float(d[0], T());
        }
      }
    }
  });
  if (partial == nullptr && dbias == nullptr) return;
#pragma unroll
  for (int e = 0; e < VW; ++e) part[warp][lane][e] = sum[e];
  __syncthreads();
  for (int i = threadIdx.x; i < 32 * VW; i += kSlopeThreads) {
    const int64_t col = int64_t(blockIdx.x) * 32 * VW + i;
    if (col >= cols) continue;
    float v = 0.f;
#pragma unroll
    for (int w = 0; w < 8; ++w) v += part[w][i / VW][i % VW];
    if (dbias != nullptr) st1_stream(dbias + col, v);  // one chunk: these are the sums
    else partial[int64_t(blockIdx.y) * cols + col] = v;
  }
}

// ---------------------------------------------------------------------------
// launches
// ---------------------------------------------------------------------------

bool on(const void* p, unsigned bytes) { return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) == 0; }
int64_t round_up(int64_t v, int64_t m) { return (v + m - 1) / m * m; }

using EncodeFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                              const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                              CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

// The driver's encoder, found once (the library does not link the driver).
cudaError_t encoder(EncodeFn* fn) {
  static std::mutex mu;
  static EncodeFn found = nullptr;
  std::lock_guard<std::mutex> lk(mu);
  if (found == nullptr) {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult how;
    const cudaError_t e = cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &how);
    if (e != cudaSuccess) return e;
    if (how != cudaDriverEntryPointSuccess || p == nullptr) return cudaErrorNotSupported;
    found = reinterpret_cast<EncodeFn>(p);
  }
  *fn = found;
  return cudaSuccess;
}

// One operand of a product: `rows` rows (or columns of the result) by `depth`,
// rows (mn: depths) `ld` elements apart.
struct Operand {
  const void* p;
  const uint8_t* scales;
  int64_t rows, depth, ld;
  bool mn;
};

cudaError_t make_map(CUtensorMap* map, DType t, bool mx8, const Operand& o, int box_rows) {
  EncodeFn encode = nullptr;
  const cudaError_t e = encoder(&encode);
  if (e != cudaSuccess) return e;
  const int es = mx8 ? 1 : 2;
  const cuuint64_t dims[2] = {cuuint64_t(o.mn ? o.rows : o.depth), cuuint64_t(o.mn ? o.depth : o.rows)};
  const cuuint64_t pitch[1] = {cuuint64_t(o.ld) * es};
  const cuuint32_t box[2] = {cuuint32_t(kLine / es), cuuint32_t(o.mn ? 64 : box_rows)};
  const cuuint32_t ones[2] = {1, 1};
  const CUresult r = encode(map, mx8 ? CU_TENSOR_MAP_DATA_TYPE_UINT8
                                     : t == DType::F16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16
                                                       : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16,
                            2, const_cast<void*>(o.p), dims, pitch, box, ones, CU_TENSOR_MAP_INTERLEAVE_NONE,
                            CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

ScaleRows scale_rows(const Operand& o) {
  const int64_t g = mx_groups(o.depth);
  return ScaleRows{o.scales, o.rows, g,
                   g % 16 == 0 && on(o.scales, 16) ? 16
                   : g % 4 == 0 && on(o.scales, 4) ? 4 : g % 2 == 0 && on(o.scales, 2) ? 2 : 1};
}

// Blocks of `words` 32-bit words of scales, one after the other.
cudaError_t make_scale_map(CUtensorMap* map, const void* p, int64_t blocks, int words) {
  EncodeFn encode = nullptr;
  const cudaError_t e = encoder(&encode);
  if (e != cudaSuccess) return e;
  const cuuint64_t dims[2] = {cuuint64_t(words), cuuint64_t(blocks)}, pitch[1] = {cuuint64_t(words) * 4};
  const cuuint32_t box[2] = {cuuint32_t(words), 1}, ones[2] = {1, 1};
  const CUresult r = encode(map, CU_TENSOR_MAP_DATA_TYPE_UINT32, 2, const_cast<void*>(p), dims, pitch, box, ones,
                            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE,
                            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

int64_t tiles_of(int64_t rows, int tile) { return (rows + tile - 1) / tile; }

// Which kernel, tile and cut of K: the least of these estimates, in cycles, which
// follow from the shape alone (as workspace sizes do).  A K tile costs its
// products, 2 cycles a column (of the pair kernel, whose tile is 256 rows on two
// SMs) or a row (of the other, 128 columns on one), or its loads at 64 bytes a
// cycle and SM, whichever is more; of a CTA by itself at least 570 cycles, the
// time from one issue to the next.  Then there is what does not overlap: the
// start, the first loads' latency, the epilogue.
struct Plan {
  int tile_n;   // of the pair kernel, else 0
  int tile_m;   // of the other
  int splits;
};

Plan plan_product(bool mx, int64_t rows, int64_t cols, int64_t k_tiles, bool r_mn) {
  Plan best{0, 0, 1};
  double least = 0;
  // cycles of an epilogue for each row of a tile of 128 columns; rows that start on no 16-byte boundary are
  // written element by element
  const double row_cost = cols % 8 == 0 ? 60.0 : 120.0;
  // the operands from memory, at 3.6 KB a cycle (6.8 TB/s)
  const double memory = double(rows + cols) * double(k_tiles) * kLine / 3600.0;
  auto offer = [&](double cost, const Plan& p) {
    if (best.tile_m == 0 || cost < least) least = cost, best = p;
  };
  for (int tm = r_mn ? 64 : 16; tm <= kSplitMostRows; tm *= 2) {
    const int64_t tiles = tiles_of(rows, tm) * tiles_of(cols, kSplitN);
    const double k_cost = std::max(2.0 * tm, (kOperandQ + tm * kLine) / 64.0);
    for (int s = 1; s <= 8 && (s == 1 || k_tiles >= (mx ? 4 : 2) * s); s *= 2) {
      const double turns = double(tiles_of(tiles * s, kPlanSms)), k_each = double(tiles_of(k_tiles, s));
      const double ends = 3000.0 + (s > 1 ? 2500.0 + (80.0 + row_cost) * tm : row_cost * tm);  // (stores to other CTAs: 4 bytes a cycle)
      // two CTAs share an SM
      const double alone = double(int64_t(turns + 1) / 2) * (ends + k_each * std::max(570.0, k_cost));
      offer(2500.0 + std::max({alone, ends + turns * (k_each * k_cost + row_cost / 2 * tm / s), ends + memory}),
            Plan{0, tm, s});
    }
    if (tm >= rows) break;
  }
  if (rows > 128 && k_tiles > 0)
    for (const int tn : {mx ? 192 : 256, 128}) {
      const int64_t turns = tiles_of(tiles_of(rows, kTileM) * tiles_of(cols, tn), kPlanSms / 2);
      const double k_cost = std::max(2.0 * tn, (kOperandM + tn / 2 * kLine) / 64.0);
      offer(std::max(double(turns) * std::max(double(k_tiles) * k_cost, row_cost / 2 * tn), memory) + 7000.0 + row_cost / 2 * tn + (mx ? 4000.0 : 0.0),
            Plan{tn, 128, 1});
    }
  return best;
}

// Bytes of the arranged scales of a product on the pair kernel.
int64_t arranged_bytes(int64_t rows, int64_t cols, int64_t k_tiles, int tile_n) {
  return (2 * tiles_of(rows, kTileM) + tiles_of(cols, tile_n) * ((tile_n + 127) / 128)) * k_tiles * 512;
}

template <bool MX, int TN>
cudaError_t fill_pair(PairProduct* a, DType t, const Operand& r, const Operand& q, const Epilogue& epi, int64_t k_tiles,
                      uint8_t* ws, int sm_count, cudaStream_t stream, int* launches) {
  using S = PairShape<MX, TN>;
  cudaError_t e;
  if ((e = make_map(&a->r, t, MX, r, 64)) != cudaSuccess) return e;
  if ((e = make_map(&a->q, t, MX, q, S::kHalfN % 64 == 0 ? 64 : S::kHalfN)) != cudaSuccess) return e;
  a->tiles_m = tiles_of(r.rows, kTileM);
  a->tiles_n = tiles_of(q.rows, TN);
  if constexpr (MX) {
    ArrangeArgs g = {};
    g.s[0] = scale_rows(r), g.s[1] = scale_rows(q);
    g.tiles[0] = 2 * a->tiles_m, g.tiles[1] = a->tiles_n;
    g.rows[0] = kHalfM, g.rows[1] = TN;
    g.blocks[0] = 1, g.blocks[1] = S::kQBlocks;
    g.k_tiles = int(k_tiles);
    g.out[0] = reinterpret_cast<uint4*>(ws);
    g.out[1] = g.out[0] + g.tiles[0] * k_tiles * 32;
    const int64_t warps = (g.tiles[0] + S::kQBlocks * g.tiles[1]) * ((k_tiles + 3) / 4);
    e = launch(k_arrange, dim3(unsigned(std::min<int64_t>((warps + 7) / 8, 8 * sm_count))), dim3(256), 0, stream, g);
    if (e != cudaSuccess) return e;
    ++*launches;
    if ((e = make_scale_map(&a->rs, g.out[0], g.tiles[0] * k_tiles, 128)) != cudaSuccess) return e;
    if ((e = make_scale_map(&a->qs, g.out[1], g.tiles[1] * k_tiles, 128 * S::kQBlocks)) != cudaSuccess) return e;
  }
  a->epi = epi;
  a->k_tiles = int(k_tiles);
  a->k_tile = MX ? 128 : 64;
  a->r_mn = r.mn;
  a->q_mn = q.mn;
  a->idesc = MX ? mma_desc_mx8(kTileM, TN) : mma_desc_f16(t == DType::BF16, r.mn, q.mn, kTileM, TN);
  return cudaSuccess;
}

template <typename T, bool MX, int TN, bool TWO>
cudaError_t launch_pair(PairArgs* a, int sm_count, cudaStream_t stream, int* launches) {
  using S = PairShape<MX, TN>;
  constexpr auto kernel = k_mm_pair<T, MX, TN, TWO>;
  a->first = a->p[0].tiles_m * a->p[0].tiles_n;
  a->tiles = a->first + (TWO ? a->p[1].tiles_m * a->p[1].tiles_n : 0);
  int pairs = 1;
  cudaError_t e = resident_clusters(kernel, kPairThreads, S::kSmem, 2, sm_count, &pairs);
  if (e != cudaSuccess) return e;
  e = launch_cluster(kernel, unsigned(2 * std::min<int64_t>(a->tiles, pairs)), kPairThreads, S::kSmem, 2, stream, *a);
  if (e == cudaSuccess) ++*launches;
  return e;
}

template <typename T, bool MX, int TN>
cudaError_t product_pair(DType t, const Operand& r, const Operand& q, const Epilogue& epi, int64_t k_tiles, uint8_t* ws,
                         int sm_count, cudaStream_t stream, int* launches) {
  PairArgs a = {};
  const cudaError_t e = fill_pair<MX, TN>(&a.p[0], t, r, q, epi, k_tiles, ws, sm_count, stream, launches);
  return e != cudaSuccess ? e : launch_pair<T, MX, TN, false>(&a, sm_count, stream, launches);
}

template <typename T, bool MX>
cudaError_t product(DType t, const Operand& r, const Operand& q, const Epilogue& epi, uint8_t* ws, int sm_count,
                    cudaStream_t stream, int* launches) {
  constexpr int kWide = MX ? 192 : 256;
  const int k_tile = MX ? 128 : 64;
  const int64_t k_tiles = tiles_of(r.depth, k_tile);
  const Plan p = plan_product(MX, r.rows, q.rows, k_tiles, r.mn);
  if (p.tile_n != 0)
    return p.tile_n == kWide ? product_pair<T, MX, kWide>(t, r, q, epi, k_tiles, ws, sm_count, stream, launches)
                             : product_pair<T, MX, 128>(t, r, q, epi, k_tiles, ws, sm_count, stream, launches);
  cudaError_t e;
  SplitArgs a = {};
  if (k_tiles > 0) {
    if ((e = make_map(&a.r, t, MX, r, std::min(p.tile_m, 64))) != cudaSuccess) return e;
    if ((e = make_map(&a.q, t, MX, q, 64)) != cudaSuccess) return e;
  }
  if (MX) a.rs = scale_rows(r), a.qs = scale_rows(q);
  a.epi = epi;
  a.tiles_m = tiles_of(r.rows, p.tile_m);
  a.tile_m = p.tile_m;
  a.k_tiles = int(k_tiles);
  a.k_tile = k_tile;
  a.r_mn = r.mn;
  a.q_mn = q.mn;
  const int stage = kOperandQ + p.tile_m * kLine, quads = MX ? kScaleQuads * kSplitQuadBytes : 0;
  const int sums = p.splits > 1 && p.tile_m <= 64 ? p.tile_m * kSplitN * 4 : 0;
  a.sums_apart = sums > 0;
  a.stages = std::min(kSplitMostStages, (kSplitBudget - 1024 - quads - sums) / stage);
  a.idesc = MX ? mma_desc_mx8(kSplitN, p.tile_m) : mma_desc_f16(t == DType::BF16, q.mn, r.mn, kSplitN, p.tile_m);
  const int64_t grid = a.tiles_m * tiles_of(q.rows, kSplitN) * p.splits;
  if (grid > INT32_MAX) return cudaErrorInvalidConfiguration;
  e = launch_cluster(k_mm_split<T, MX>, unsigned(grid), kSplitThreads,
                     size_t(1024) + size_t(a.stages) * stage + quads + sums, unsigned(p.splits), stream, a);
  if (e == cudaSuccess) ++*launches;
  return e;
}

// A gradient's two products in one launch, where both take the pair kernel with tiles
// of one width; the deeper one's tiles first.
template <typename T, int TN>
cudaError_t pair_of_products(DType t, const Operand* const (&o)[2][2], const Epilogue (&epi)[2], int sm_count,
                             cudaStream_t stream, int* launches) {
  PairArgs a = {};
  const int deep = o[1][0]->depth > o[0][0]->depth ? 1 : 0;
  for (int i = 0; i < 2; ++i) {
    const int j = i == 0 ? deep : 1 - deep;
    const cudaError_t e = fill_pair<false, TN>(&a.p[i], t, *o[j][0], *o[j][1], epi[j], tiles_of(o[j][0]->depth, 64), nullptr,
                                               sm_count, stream, launches);
    if (e != cudaSuccess) return e;
  }
  return launch_pair<T, false, TN, true>(&a, sm_count, stream, launches);
}

cudaError_t product(DType t, bool mx8, const Operand& r, const Operand& q, const Epilogue& epi, uint8_t* ws, int sm_count,
                    cudaStream_t stream, int* launches) {
  if (t == DType::F16)
    return mx8 ? product<__half, true>(t, r, q, epi, ws, sm_count, stream, launches)
               : product<__half, false>(t, r, q, epi, ws, sm_count, stream, launches);
  return mx8 ? product<__nv_bfloat16, true>(t, r, q, epi, ws, sm_count, stream, launches)
             : product<__nv_bfloat16, false>(t, r, q, epi, ws, sm_count, stream, launches);
}

// Whether rows of n elements of `es` bytes from p on can be read by TMA as they lie.
bool in_place(const void* p, int64_t n, int es) { return n * es % 16 == 0 && on(p, 16); }
int64_t pitched_bytes(int64_t rows, int64_t n, int es) { return round_up(rows * round_up(n, 16 / es) * es, 256); }

// Copies for operands that cannot be read as they lie, collected for one launch.
struct Pitcher {
  int es;
  uint8_t* ws;
  PitchArgs a = {};
  int used = 0;
  // o as it lies, or as its copy will.
  void add(Operand* o) {
    const int64_t n = o->mn ? o->rows : o->depth, rows = o->mn ? o->depth : o->rows;
    o->ld = n;
    if (n == 0 || rows == 0 || in_place(o->p, n, es)) return;
    o->ld = round_up(n, 16 / es);
    a.x[used] = o->p;
    a.y[used] = ws;
    a.rows[used] = rows;
    a.n[used] = uint32_t(n);
    a.ld[used++] = uint32_t(o->ld);
    o->p = ws;
    ws += pitched_bytes(rows, n, es);
  }
  cudaError_t run(int sm_count, cudaStream_t stream, int* launches) const {
    if (used == 0) return cudaSuccess;
    int64_t warps = 0;
    for (int i = 0; i < used; ++i) warps += a.rows[i] * ((a.ld[i] + 255) / 256);
    const dim3 grid(unsigned(std::min<int64_t>((warps + 7) / 8, int64_t(sm_count) * 16)));
    const cudaError_t e = es == 1 ? launch(k_pitch<uint8_t>, grid, dim3(256), 0, stream, a)
                                  : launch(k_pitch<uint16_t>, grid, dim3(256), 0, stream, a);
    if (e == cudaSuccess) ++*launches;
    return e;
  }
};

// Row chunks of k_act_slope: as many blocks as the device holds (three an SM) at once,
// 64 rows at least (so that few rows have one chunk, whose sums are dbias).
int64_t slope_chunks(int64_t M, int64_t N) {
  const int64_t tiles = std::max<int64_t>(1, (N + 255) / 256);
  return std::max<int64_t>(1, std::min({3 * kPlanSms / tiles, (M + 63) / 64, int64_t(65535)}));
}

template <typename T>
cudaError_t act_slope_rows(const MatmulGradArgs& a, T* dz, int64_t ld, float* partial, cudaStream_t stream,
                           int* launches) {
  const int zm = a.act == kActNone ? 0 : a.z_scales != nullptr ? 2 : 1;
  const bool vec = a.N % 8 == 0 && on(a.dy, 16) && (zm != 1 || on(a.z, 16)) && (zm != 2 || on(a.z, 8));
  const int64_t chunks = slope_chunks(a.M, a.N), per = (a.M + chunks - 1) / chunks, used = (a.M + per - 1) / per;
  const int64_t width = dz != nullptr ? ld : a.N;
  auto run = [&](auto kernel, int vw) {
    return launch(kernel, dim3(unsigned((width + 32 * vw - 1) / (32 * vw)), unsigned(used)), dim3(kSlopeThreads), 0,
                  stream, static_cast<const T*>(a.dy), a.z, a.z_scales, dz, a.M, a.N, width, per, a.act, a.alpha,
                  used > 1 ? partial : nullptr, used == 1 ? static_cast<T*>(a.dbias) : nullptr);
  };
  cudaError_t e;
  if (vec) e = zm == 0 ? run(k_act_slope<T, 8, 0>, 8) : zm == 1 ? run(k_act_slope<T, 8, 1>, 8) : run(k_act_slope<T, 8, 2>, 8);
  else e = zm == 0 ? run(k_act_slope<T, 1, 0>, 1) : zm == 1 ? run(k_act_slope<T, 1, 1>, 1) : run(k_act_slope<T, 1, 2>, 1);
  if (e != cudaSuccess) return e;
  ++*launches;
  if (partial == nullptr || used == 1) return cudaSuccess;
  e = launch(k_channel_sums<T>, dim3(unsigned(std::min<int64_t>((a.N + 31) / 32, 65535))), dim3(kSumsThreads), 0,
             stream, static_cast<const float*>(partial), used, int64_t(1), a.N, 1, static_cast<T*>(a.dbias),
             static_cast<T*>(nullptr));
  if (e == cudaSuccess) ++*launches;
  return e;
}

}  // namespace

size_t matmul_workspace_bytes(bool mx8, int64_t M, int64_t N, int64_t K, bool aligned) {
  const int es = mx8 ? 1 : 2;
  size_t b = 0;
  if (K > 0 && !(aligned && K * es % 16 == 0)) b += size_t(pitched_bytes(M, K, es) + pitched_bytes(N, K, es));
  if (mx8) {
    const Plan p = plan_product(true, M, N, tiles_of(K, 128), false);
    if (p.tile_n != 0) b += size_t(arranged_bytes(M, N, tiles_of(K, 128), p.tile_n));
  }
  return b;
}

void set_access(Epilogue* e) {
  e->vec = e->cols % 8 == 0 && on(e->y, 16) && on(e->residual, 16) && on(e->z, 16);
  e->pairs = e->cols % 2 == 0 && on(e->y, 4) && on(e->residual, 4) && on(e->z, e->z_scales != nullptr ? 2 : 4);
  e->vec_bias = on(e->bias, 16);
}

cudaError_t launch_matmul(const MatmulArgs& a, int sm_count, cudaStream_t stream, int* launches) {
  Pitcher pitch{a.mx8 ? 1 : 2, static_cast<uint8_t*>(a.workspace)};
  Operand r{a.a, a.a_scales, a.M, a.K, a.K, false}, q{a.w, a.w_scales, a.N, a.K, a.K, false};
  pitch.add(&r);
  pitch.add(&q);
  const cudaError_t e = pitch.run(sm_count, stream, launches);
  if (e != cudaSuccess) return e;
  Epilogue epi{a.bias, a.residual, a.y, a.z, a.z_scales, a.M, a.N, a.act, a.alpha, false, false, false};
  set_access(&epi);
  return product(a.t, a.mx8, r, q, epi, pitch.ws, sm_count, stream, launches);
}

size_t matmul_grad_workspace_bytes(int64_t M, int64_t N, int64_t K, bool act, bool a_mx8, bool aligned) {
  size_t b = size_t(round_up(slope_chunks(M, N) * N * 4, 256));
  if (act || !aligned || N % 8 != 0) b += size_t(pitched_bytes(M, N, 2));
  if (a_mx8 || !aligned || K % 8 != 0) b += size_t(pitched_bytes(M, K, 2));
  if (!aligned || K % 8 != 0) b += size_t(pitched_bytes(N, K, 2));
  return b;
}

cudaError_t launch_matmul_grad(const MatmulGradArgs& a, int sm_count, cudaStream_t stream, int* launches) {
  uint8_t* ws = static_cast<uint8_t*>(a.workspace);
  cudaError_t e = cudaSuccess;
  float* partial = nullptr;
  if (a.dbias != nullptr && a.M > 0 && a.N > 0) {
    partial = reinterpret_cast<float*>(ws);
    ws += round_up(slope_chunks(a.M, a.N) * a.N * 4, 256);
  }
  // dz, as it lies or made
  const void* dz = a.dy;
  int64_t ld = a.N;
  const bool make = a.M > 0 && a.N > 0 && (a.act != kActNone || !in_place(a.dy, a.N, 2));
  if (make) {
    ld = round_up(a.N, 8);
    dz = ws;
    ws += pitched_bytes(a.M, a.N, 2);
  }
  if (make || partial != nullptr) {
    void* out = make ? const_cast<void*>(dz) : nullptr;
    e = a.t == DType::F16 ? act_slope_rows(a, static_cast<__half*>(out), ld, partial, stream, launches)
                          : act_slope_rows(a, static_cast<__nv_bfloat16*>(out), ld, partial, stream, launches);
    if (e != cudaSuccess) return e;
  }
  // dA (M, K) = dz (M, N) W: W's rows are the depth.  dW (N, K) = dz^T A: both have the depth as rows.
  Operand ra{dz, nullptr, a.M, a.N, ld, false}, qa{a.w, nullptr, a.K, a.N, a.K, true};
  Operand rw{dz, nullptr, a.N, a.M, ld, true}, qw{a.a, nullptr, a.K, a.M, a.K, true};
  const bool da = a.da != nullptr && a.M > 0 && a.K > 0, dw = a.dw != nullptr && a.N > 0 && a.K > 0;
  Pitcher pitch{2, ws};
  if (da) pitch.add(&qa);
  if (dw) {
    if (a.a_scales != nullptr && a.M > 0) {
      qw.ld = round_up(a.K, 8);
      qw.p = pitch.ws;
      pitch.ws += pitched_bytes(a.M, a.K, 2);
      e = launch_dequantize_pitched(a.t, static_cast<const uint8_t*>(a.a), a.a_scales, const_cast<void*>(qw.p), a.M, a.K,
                                    qw.ld, sm_count, stream, launches);
      if (e != cudaSuccess) return e;
    } else {
      pitch.add(&qw);
    }
  }
  if ((e = pitch.run(sm_count, stream, launches)) != cudaSuccess) return e;
  auto plain = [](const Operand& r, const Operand& q, void* y) {
    Epilogue epi{nullptr, nullptr, y, nullptr, nullptr, r.rows, q.rows, kActNone, 0.f, false, false, false};
    set_access(&epi);
    return epi;
  };
  const Epilogue epi[2] = {plain(ra, qa, a.da), plain(rw, qw, a.dw)};
  if (da && dw) {
    const int width = plan_product(false, ra.rows, qa.rows, tiles_of(ra.depth, 64), false).tile_n;
    if (width != 0 && width == plan_product(false, rw.rows, qw.rows, tiles_of(rw.depth, 64), true).tile_n) {
      const Operand* const o[2][2] = {{&ra, &qa}, {&rw, &qw}};
      if (a.t == DType::F16)
        return width == 256 ? pair_of_products<__half, 256>(a.t, o, epi, sm_count, stream, launches)
                            : pair_of_products<__half, 128>(a.t, o, epi, sm_count, stream, launches);
      return width == 256 ? pair_of_products<__nv_bfloat16, 256>(a.t, o, epi, sm_count, stream, launches)
                          : pair_of_products<__nv_bfloat16, 128>(a.t, o, epi, sm_count, stream, launches);
    }
  }
  if (da) e = product(a.t, false, ra, qa, epi[0], nullptr, sm_count, stream, launches);
  if (dw && e == cudaSuccess) e = product(a.t, false, rw, qw, epi[1], nullptr, sm_count, stream, launches);
  return e;
}

cudaError_t matmul_pipe_timeouts(unsigned int* count, bool clear) { return read_pipe_timeouts(count, clear); }

}  // namespace ep

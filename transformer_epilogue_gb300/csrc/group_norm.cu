// GroupNorm over channels-last (N, S, C) tensors, with an optional SiLU, and
// its gradient.
//
// Definition (com.microsoft.GroupNorm of the contrib family, channels_last = 1):
// G groups of D = C / G neighbouring channels, M = S * D values each;
//   mu = mean(x), var = mean((x - mu)^2), r = 1 / sqrt(var + epsilon)   per (n, g)
//   h = (x - mu) r,  u = h * gamma[c] + beta[c],  y = u or u * sigmoid(u)
// and the gradient, from dy and the saved mu and r:
//   du = dy or dy * s (1 + u (1 - s)), s = sigmoid(u)
//   dbeta[c] = sum du,  dgamma[c] = sum du * h                          over n and positions
//   m1 = mean(du * gamma), m2 = mean(du * gamma * h)                    per (n, g)
//   dx = r (du * gamma - m1 - h m2)
//
// Split form (this file's general path, any C, S and alignment): the walk of
// column_walk.cuh over each sample.  Pass 1 leaves (count, mean, sum of squared
// distances) per chunk and group, a small kernel joins the chunks, pass 2 reads
// x again (from L2 where it fits) and writes y.  The statistics are taken
// relative to values near their mean throughout, so that a large mean costs the
// variance nothing.  The gradient has the same three steps, with per-channel sums of du
// and du * h beside the groups' sums.
//
// All sums and statistics are float32; results are rounded once, to T.
#include <algorithm>
#include <climits>
#include <type_traits>

#include "column_walk.cuh"
#include "device_common.cuh"
#include "ep_internal.h"
#include "group_norm.cuh"
#include "launch_util.h"

namespace ep {
namespace {

// The split kernels' forms:
//  kAny      any C and alignment: fragments are checked against the sample's
//            ends, and a sample may start off a 16-byte boundary (VEC: whole
//            fragments are loaded as 16 bytes; else value by value);
//  kChannel  C % VW == 0 and 16-byte-aligned operands: every fragment is whole
//            (and the last walk row may have fewer than the others);
//  kGroup    and D % VW == 0: a fragment lies in one group, so statistics and
//            group sums are per fragment, not per channel.
enum { kAny = 0, kChannel = 1, kGroup = 2 };

// One call's sizes, as every kernel of the split form gets them (C is at most
// kMaxGroupNormChannels, so positions in a walk row fit an int), for the
// samples of one launch.
struct GnDims {
  int64_t N, S, L;  // L = S * C
  int C, G, D;
  float eps;
  WalkPlan p;
};

// Where a sample's walk row starts: `off` elements before the sample.
template <typename T, int FORM, bool VEC>
__device__ __forceinline__ int walk_offset(const T* sample) {
  return FORM == kAny && VEC ? dev::misalignment(sample) : 0;
}

// The channel of the first element of fragment column j.
__device__ __forceinline__ int first_channel(int64_t j, int vw, int off, int C) {
  return static_cast<int>((j * vw + C - off % C) % C);
}

// The first repeat k of a group whose channels [c0, c0 + D), at the positions
// off + c + k C of a walk row, reach past position p0 (k < 0: the channels that
// the walk row's `off` leading positions hold).
__device__ __forceinline__ int first_repeat(int p0, int off, int c0, int D, int C) {
  const int a = p0 - off - c0 - D;
  return (a >= 0 ? a / C : -((-a + C - 1) / C)) + 1;
}

// Calls f(i, c) for every position p0 + i of a tile of np positions that holds a
// channel c of the group, by the lanes of a warp in turn: the lanes split into
// sets of the smallest power of two that holds D channels (at most 32), each set
// taking the repeats in turn, so that few channels still use (and sum over) all lanes.
// (kGroup: positions are fragments, and C, D, c0 count fragments too.)
template <typename F>
__device__ __forceinline__ void for_group(int p0, int np, int off, int c0, int D, int C, F f) {
  const int lane = threadIdx.x & 31;
  const int set = D >= 32 ? 32 : D <= 1 ? 1 : 1 << (32 - __clz(D - 1));
  const int64_t step = int64_t(C) * (32 / set);
  for (int64_t a = off + c0 + int64_t(first_repeat(p0, off, c0, D, C) + lane / set) * C - p0; a < np; a += step) {
    const int lo = static_cast<int>(max(int64_t(0), a)), hi = static_cast<int>(min(int64_t(np), a + D));
    for (int i = lo + (lane & (set - 1)); i < hi; i += set) f(i, c0 + (i - static_cast<int>(a)));
  }
}

__device__ __forceinline__ bool group_in_tile(int p0, int np, int off, int c0, int D, int C) {
  return off + c0 + int64_t(first_repeat(p0, off, c0, D, C)) * C < p0 + np;
}

// A CTA's place: its tile of the walk row and its thread's fragment column.
struct Tile {
  int tile, frags;   // the tile's number and fragments
  int64_t j;         // fragment column
  int64_t rows;      // walk rows of a sample that have a fragment j (kAny: all, with checks)
  bool mine;
  __device__ __forceinline__ Tile(const WalkPlan& p, int64_t sample_frags) {
    tile = p.tiles == 1 ? 0 : static_cast<int>(blockIdx.x % unsigned(p.tiles));
    frags = static_cast<int>(min(int64_t(p.tile_frags), p.row_frags - int64_t(tile) * p.tile_frags));
    j = int64_t(tile) * p.tile_frags + threadIdx.x;
    mine = int(threadIdx.x) < frags;
    rows = sample_frags < 0 ? p.rows : (sample_frags - j + p.row_frags - 1) / p.row_frags;
  }
};

// Pass 1.  partial: [item][tile][G] x (count, mean, M2), relative to the group's
// first value, or, where a sample has one item and one tile, the statistics
// themselves (partial == nullptr).  A thread sums its values and their squares
// relative to the mean of its first U rows, which is near enough to its own mean
// that nothing cancels; the threads' (count, mean, M2) are joined by two sums,
// the second relative to the first's mean.
template <typename T, int FORM>
__global__ void __launch_bounds__(kWalkThreads)
k_gn_stats(const T* x, GnDims d, float* partial, float* mean_out, float* inv_out) {
  constexpr int VW = dev::Vec16<T>::N;
  constexpr int EV = FORM == kGroup ? 1 : VW;  // sums of a thread
  constexpr int U = 4;
  __shared__ float s_cnt[kWalkThreads * EV], s_mean[kWalkThreads * EV], s_m2[kWalkThreads * EV];
  dev::pdl_wait();
  dev::pdl_trigger();
  const WalkPlan& p = d.p;
  const Tile t(p, FORM == kAny ? -1 : d.L / VW);
  const int p0 = t.tile * p.tile_frags * EV, np = t.frags * EV;
  const int Cw = FORM == kGroup ? d.C / VW : d.C, Dw = FORM == kGroup ? d.D / VW : d.D;
  const int64_t items = d.N * p.chunks;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;

  for (int64_t item = blockIdx.x / unsigned(p.tiles); item < items; item += gridDim.x / unsigned(p.tiles)) {
    const int64_t n = item / p.chunks, chunk = item - n * p.chunks;
    const T* xs = x + n * d.L;
    const int off = walk_offset<T, FORM, true>(xs);
    if (t.mine) {
      float first[EV], c[EV], s[EV], q[EV], cnt[EV];
      for_channels<VW>(first_channel(t.j, VW, off, d.C), d.C, d.D, [&](int e, int, int g) {
        if (e < EV) first[e] = dev::ld1_keep(xs + int64_t(g) * d.D);
      });
#pragma unroll
      for (int e = 0; e < EV; ++e) s[e] = q[e] = cnt[e] = 0.f;
      const int64_t ra = chunk * p.rows_per_chunk, rb = min(t.rows, ra + p.rows_per_chunk);
      const int64_t pitch = p.row_frags * VW;
      const T* px = xs + (ra * p.row_frags + t.j) * VW;
      if constexpr (FORM != kAny) {
        // centre: the first rows' mean
        if (ra < rb) {
          float m[EV];
#pragma unroll
          for (int e = 0; e < EV; ++e) m[e] = 0.f;
          const int u1 = static_cast<int>(min(int64_t(U), rb - ra));
          for (int u = 0; u < u1; ++u) {
            float v[VW];
            dev::Conv<T>::unpack(dev::ld16_keep(px + u * pitch), v);
#pragma unroll
            for (int e = 0; e < VW; ++e) m[EV == 1 ? 0 : e] += v[e] - first[EV == 1 ? 0 : e];
          }
#pragma unroll
          for (int e = 0; e < EV; ++e) c[e] = first[e] + m[e] / float(u1 * (VW / EV));
        } else {
#pragma unroll
          for (int e = 0; e < EV; ++e) c[e] = first[e];
        }
        auto add = [&](uint4 raw) {
          float v[VW];
          dev::Conv<T>::unpack(raw, v);
#pragma unroll
          for (int e = 0; e < VW; ++e) v[e] -= c[EV == 1 ? 0 : e];
          if constexpr (EV == 1) {
            float a = 0.f, b = 0.f;
#pragma unroll
            for (int e = 0; e < VW; e += 2) {
              a += v[e] + v[e + 1];
              b = fmaf(v[e], v[e], b);
              q[0] = fmaf(v[e + 1], v[e + 1], q[0]);
            }
            s[0] += a;
            q[0] += b;
          } else {
#pragma unroll
            for (int e = 0; e < VW; ++e) {
              s[e] += v[e];
              q[e] = fmaf(v[e], v[e], q[e]);
            }
          }
        };
        int64_t r = ra;
        for (; r + U <= rb; r += U, px += U * pitch) {
          uint4 raw[U];
#pragma unroll
          for (int u = 0; u < U; ++u) raw[u] = dev::ld16_keep(px + u * pitch);
#pragma unroll
          for (int u = 0; u < U; ++u) add(raw[u]);
        }
        for (; r < rb; ++r, px += pitch) add(dev::ld16_keep(px));
#pragma unroll
        for (int e = 0; e < EV; ++e) cnt[e] = ra < rb ? float(rb - ra) * (VW / EV) : 0.f;
      } else {
        // the centre is the first value a channel meets here
#pragma unroll
        for (int e = 0; e < VW; ++e) c[e] = first[e];
        for (int64_t r0 = ra; r0 < rb; r0 += U) {
          float v[U][VW];
#pragma unroll
          for (int u = 0; u < U; ++u)
            if (r0 + u < rb) dev::load_frag<T, true>(xs, ((r0 + u) * p.row_frags + t.j) * VW - off, d.L, v[u]);
#pragma unroll
          for (int u = 0; u < U; ++u) {
            const int64_t e0 = ((r0 + u) * p.row_frags + t.j) * VW - off;
#pragma unroll
            for (int e = 0; e < VW; ++e) {
              if (r0 + u < rb && e0 + e >= 0 && e0 + e < d.L) {
                if (cnt[e] == 0.f) c[e] = v[u][e];
                const float w = v[u][e] - c[e];
                cnt[e] += 1.f;
                s[e] += w;
                q[e] = fmaf(w, w, q[e]);
              }
            }
          }
        }
      }
#pragma unroll
      for (int e = 0; e < EV; ++e) {
        const float m = cnt[e] > 0.f ? s[e] / cnt[e] : 0.f;
        s_cnt[threadIdx.x * EV + e] = cnt[e];
        s_mean[threadIdx.x * EV + e] = (c[e] - first[e]) + m;
        s_m2[threadIdx.x * EV + e] = not_negative(q[e] - s[e] * m);
      }
    }
    __syncthreads();
    for (int g = warp; g < d.G; g += warps) {
      float* out = partial + ((item * p.tiles + t.tile) * d.G + g) * 3;
      if (p.tiles > 1 && !group_in_tile(p0, np, off, g * Dw, Dw, Cw)) {
        if (lane == 0) out[0] = out[1] = out[2] = 0.f;
        continue;
      }
      float c = 0.f, s = 0.f, q = 0.f;
      for_group(p0, np, off, g * Dw, Dw, Cw, [&](int i, int) {
        c += s_cnt[i];
        s = fmaf(s_cnt[i], s_mean[i], s);
      });
      c = dev::warp_sum(c);
      s = dev::warp_sum(s);
      const float mg = c > 0.f ? s / c : 0.f;
      float res = 0.f;  // what rounding s / c and the sum left out of the mean
      for_group(p0, np, off, g * Dw, Dw, Cw, [&](int i, int) {
        const float w = s_mean[i] - mg;
        res = fmaf(s_cnt[i], w, res);
        q += fmaf(s_cnt[i] * w, w, s_m2[i]);
      });
      res = dev::warp_sum(res);
      q = dev::warp_sum(q);
      if (lane == 0) {
        const float fix = c > 0.f ? res / c : 0.f;
        const float mf = mg + fix, m2g = not_negative(q - res * fix);
        if (partial == nullptr) {
          mean_out[n * d.G + g] = dev::ld1_keep(xs + int64_t(g) * d.D) + mf;
          inv_out[n * d.G + g] = 1.0f / sqrtf(m2g / c + d.eps);
        } else {
          out[0] = c;
          out[1] = mf;
          out[2] = m2g;
        }
      }
    }
    __syncthreads();
  }
}

// Joins a group's chunks and tiles: one warp for each (n, g).
template <typename T>
__global__ void __launch_bounds__(256)
k_gn_join(const T* x, const float* partial, GnDims d, float* mean_out, float* inv_out) {
  dev::pdl_wait();
  dev::pdl_trigger();
  const int lane = threadIdx.x & 31;
  const int64_t parts = int64_t(d.p.chunks) * d.p.tiles;
  for (int64_t i = int64_t(blockIdx.x) * 8 + (threadIdx.x >> 5); i < d.N * d.G; i += int64_t(gridDim.x) * 8) {
    const float* src = partial + ((i / d.G) * parts * d.G + i % d.G) * 3;
    float c = 0.f, s = 0.f, q = 0.f, res = 0.f;
#pragma unroll 4
    for (int64_t k = lane; k < parts; k += 32) {
      const float* e = src + k * d.G * 3;
      const float n = __ldcg(e);
      c += n;
      s = fmaf(n, __ldcg(e + 1), s);
    }
    c = dev::warp_sum(c);
    s = dev::warp_sum(s);
    const float mg = s / c;
#pragma unroll 4
    for (int64_t k = lane; k < parts; k += 32) {
      const float* e = src + k * d.G * 3;
      const float w = __ldcg(e + 1) - mg, n = __ldcg(e);
      res = fmaf(n, w, res);
      q += fmaf(n * w, w, __ldcg(e + 2));
    }
    res = dev::warp_sum(res);
    q = dev::warp_sum(q);
    if (lane == 0) {
      const float fix = res / c;
      mean_out[i] = dev::ld1_keep(x + i / d.G * d.L + i % d.G * d.D) + (mg + fix);
      inv_out[i] = 1.0f / sqrtf(not_negative(q - res * fix) / c + d.eps);
    }
  }
}

// Pass 2: y from x and the statistics.  Bound by the data where x comes from DRAM.
template <typename T, int FORM, bool VEC, bool SILU>
__global__ void __launch_bounds__(kWalkThreads)
k_gn_apply(const T* x, const T* __restrict__ gamma, const T* __restrict__ beta, const float* mean, const float* inv,
           T* y, GnDims d) {
  constexpr int VW = dev::Vec16<T>::N;
  constexpr int EV = FORM == kGroup ? 1 : VW;
  constexpr int U = 4;
  dev::pdl_wait();
  dev::pdl_trigger();
  const WalkPlan& p = d.p;
  const Tile t(p, FORM == kAny ? -1 : d.L / VW);
  if (!t.mine) return;
  const int64_t items = d.N * p.chunks;
  for (int64_t item = blockIdx.x / unsigned(p.tiles); item < items; item += gridDim.x / unsigned(p.tiles)) {
    const int64_t n = item / p.chunks, chunk = item - n * p.chunks;
    const T* xs = x + n * d.L;
    T* ys = y + n * d.L;
    const int off = walk_offset<T, FORM, VEC>(xs);
    float mu[EV], a[VW], b[VW];
    for_channels<VW>(first_channel(t.j, VW, off, d.C), d.C, d.D, [&](int e, int c, int g) {
      if (e < EV) mu[e] = mean[n * d.G + g];
      a[e] = inv[n * d.G + g] * dev::ld1_keep(gamma + c);
      b[e] = beta != nullptr ? dev::ld1_keep(beta + c) : 0.f;
    });
    auto value = [&](float (&v)[VW]) {
#pragma unroll
      for (int e = 0; e < VW; ++e) {
        v[e] = fmaf(v[e] - mu[EV == 1 ? 0 : e], a[e], b[e]);
        if constexpr (SILU) v[e] = silu<T>(v[e]);
      }
    };
    const int64_t ra = chunk * p.rows_per_chunk, rb = min(t.rows, ra + p.rows_per_chunk);
    if constexpr (FORM != kAny) {
      const int64_t pitch = p.row_frags * VW, at = (ra * p.row_frags + t.j) * VW;
      const T* px = xs + at;
      T* py = ys + at;
      int64_t r = ra;
      for (; r + U <= rb; r += U, px += U * pitch, py += U * pitch) {
        uint4 raw[U];
#pragma unroll
        for (int u = 0; u < U; ++u) raw[u] = dev::ld16_stream(px + u * pitch);
#pragma unroll
        for (int u = 0; u < U; ++u) {
          float v[VW];
          dev::Conv<T>::unpack(raw[u], v);
          value(v);
          dev::st16_stream(py + u * pitch, dev::Conv<T>::pack(v));
        }
      }
      for (; r < rb; ++r, px += pitch, py += pitch) {
        float v[VW];
        dev::Conv<T>::unpack(dev::ld16_stream(px), v);
        value(v);
        dev::st16_stream(py, dev::Conv<T>::pack(v));
      }
    } else {
      for (int64_t r0 = ra; r0 < rb; r0 += U) {
        float v[U][VW];
#pragma unroll
        for (int u = 0; u < U; ++u)
          if (r0 + u < rb) dev::load_frag<T, VEC>(xs, ((r0 + u) * p.row_frags + t.j) * VW - off, d.L, v[u]);
#pragma unroll
        for (int u = 0; u < U; ++u) {
          if (r0 + u < rb) {
            value(v[u]);
            dev::store_frag<T, VEC>(ys, ((r0 + u) * p.row_frags + t.j) * VW - off, d.L, v[u]);
          }
        }
      }
    }
  }
}

// What the gradient's passes make of x and dy: h and du, with a thread's channel
// values in registers.
template <typename T, int EV, bool SILU>
struct GradValues {
  static constexpr int VW = dev::Vec16<T>::N;
  float mu[EV], rs[EV], ga[VW], be[VW];
  __device__ __forceinline__ void load(int c0, int64_t ng, const GnDims& d, const T* __restrict__ gamma,
                                       const T* __restrict__ beta, const float* mean, const float* inv) {
    for_channels<VW>(c0, d.C, d.D, [&](int e, int c, int g) {
      if (e < EV) {
        mu[e] = mean[ng + g];
        rs[e] = inv[ng + g];
      }
      ga[e] = dev::ld1_keep(gamma + c);
      be[e] = SILU && beta != nullptr ? dev::ld1_keep(beta + c) : 0.f;
    });
  }
  // x -> h, dy -> du
  __device__ __forceinline__ void operator()(float (&v)[VW], float (&w)[VW]) const {
#pragma unroll
    for (int e = 0; e < VW; ++e) {
      v[e] = (v[e] - mu[EV == 1 ? 0 : e]) * rs[EV == 1 ? 0 : e];
      if constexpr (SILU) w[e] = silu_grad<T>(w[e], fmaf(v[e], ga[e], be[e]));
    }
  }
};

// Gradient, pass 1: per-channel sums of du and du * h of a CTA's items, and the
// groups' sums of each item.  A CTA's items share `off` (the launch sees to
// it), so a thread's channels stay the same and its sums run on over them.
//   gpart: [item][tile][G] x (sum du gamma, sum du gamma h)
//   cpart: 2 x [CTA row][C] (one tile) or 2 x [CTA row][walk row], position 0
//          being channel 0
template <typename T, int FORM, bool VEC, bool SILU>
__global__ void __launch_bounds__(kWalkThreads)
k_gn_grad_sums(const T* dy, const T* x, const T* __restrict__ gamma, const T* __restrict__ beta, const float* mean,
               const float* inv, GnDims d, float* gpart, float* cpart) {
  constexpr int VW = dev::Vec16<T>::N;
  constexpr int EV = FORM == kGroup ? 1 : VW;
  constexpr int U = sizeof(T) == 4 ? 4 : 2;
  __shared__ float s_a[kWalkThreads * VW], s_b[kWalkThreads * VW];
  dev::pdl_wait();
  dev::pdl_trigger();
  const WalkPlan& p = d.p;
  const Tile t(p, FORM == kAny ? -1 : d.L / VW);
  const int p0 = t.tile * p.tile_frags * EV, np = t.frags * EV;
  const int Cw = FORM == kGroup ? d.C / VW : d.C, Dw = FORM == kGroup ? d.D / VW : d.D;
  const int64_t items = d.N * p.chunks;
  const int cta_rows = gridDim.x / unsigned(p.tiles), cta_row = blockIdx.x / unsigned(p.tiles);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  float tot_a[VW], tot_b[VW];
#pragma unroll
  for (int e = 0; e < VW; ++e) tot_a[e] = tot_b[e] = 0.f;
  int off = 0;

  for (int64_t item = cta_row; item < items; item += cta_rows) {
    const int64_t n = item / p.chunks, chunk = item - n * p.chunks;
    const T* xs = x + n * d.L;
    const T* ds = dy + n * d.L;
    off = walk_offset<T, FORM, VEC>(xs);
    if (t.mine) {
      GradValues<T, EV, SILU> val;
      val.load(first_channel(t.j, VW, off, d.C), n * d.G, d, gamma, beta, mean, inv);
      float sa[VW], sb[VW];
#pragma unroll
      for (int e = 0; e < VW; ++e) sa[e] = sb[e] = 0.f;
      auto add = [&](float (&v)[VW], float (&w)[VW]) {
        val(v, w);
#pragma unroll
        for (int e = 0; e < VW; ++e) {
          sa[e] += w[e];
          sb[e] = fmaf(w[e], v[e], sb[e]);
        }
      };
      const int64_t ra = chunk * p.rows_per_chunk, rb = min(t.rows, ra + p.rows_per_chunk);
      if constexpr (FORM != kAny) {
        const int64_t pitch = p.row_frags * VW, at = (ra * p.row_frags + t.j) * VW;
        const T* px = xs + at;
        const T* pd = ds + at;
        int64_t r = ra;
        for (; r + U <= rb; r += U, px += U * pitch, pd += U * pitch) {
          uint4 rx[U], rd[U];
#pragma unroll
          for (int u = 0; u < U; ++u) {
            rx[u] = dev::ld16_keep(px + u * pitch);
            rd[u] = dev::ld16_keep(pd + u * pitch);
          }
#pragma unroll
          for (int u = 0; u < U; ++u) {
            float v[VW], w[VW];
            dev::Conv<T>::unpack(rx[u], v);
            dev::Conv<T>::unpack(rd[u], w);
            add(v, w);
          }
        }
        for (; r < rb; ++r, px += pitch, pd += pitch) {
          float v[VW], w[VW];
          dev::Conv<T>::unpack(dev::ld16_keep(px), v);
          dev::Conv<T>::unpack(dev::ld16_keep(pd), w);
          add(v, w);
        }
      } else {
        for (int64_t r = ra; r < rb; ++r) {
          const int64_t e0 = (r * p.row_frags + t.j) * VW - off;
          float v[VW], w[VW];
          dev::load_frag<T, VEC>(xs, e0, d.L, v);
          dev::load_frag<T, VEC>(ds, e0, d.L, w);  // 0 outside the sample: adds nothing
          add(v, w);
        }
      }
      if constexpr (FORM == kGroup) {
        float a = 0.f, b = 0.f;
#pragma unroll
        for (int e = 0; e < VW; ++e) {
          a = fmaf(sa[e], val.ga[e], a);
          b = fmaf(sb[e], val.ga[e], b);
        }
        s_a[threadIdx.x] = a;
        s_b[threadIdx.x] = b;
      } else {
#pragma unroll
        for (int e = 0; e < VW; ++e) {
          s_a[threadIdx.x * VW + e] = sa[e] * val.ga[e];
          s_b[threadIdx.x * VW + e] = sb[e] * val.ga[e];
        }
      }
#pragma unroll
      for (int e = 0; e < VW; ++e) {
        tot_a[e] += sa[e];
        tot_b[e] += sb[e];
      }
    }
    __syncthreads();
    for (int g = warp; g < d.G; g += warps) {
      float a = 0.f, b = 0.f;
      if (p.tiles == 1 || group_in_tile(p0, np, off, g * Dw, Dw, Cw)) {
        for_group(p0, np, off, g * Dw, Dw, Cw, [&](int i, int) {
          a += s_a[i];
          b += s_b[i];
        });
        a = dev::warp_sum(a);
        b = dev::warp_sum(b);
      }
      if (lane == 0) {
        float* out = gpart + ((item * p.tiles + t.tile) * d.G + g) * 2;
        out[0] = a;
        out[1] = b;
      }
    }
    __syncthreads();
  }
  if (cpart == nullptr) return;
  if (p.tiles > 1) {
    if (t.mine) {
      const int64_t P = p.row_frags * VW;
      float* oa = cpart + cta_row * P;
      float* ob = oa + cta_rows * P;
#pragma unroll
      for (int e = 0; e < VW; ++e) {
        int64_t q = t.j * VW + e - off;
        if (q < 0) q += P;
        oa[q] = tot_a[e];
        ob[q] = tot_b[e];
      }
    }
    return;
  }
  if (t.mine) {
#pragma unroll
    for (int e = 0; e < VW; ++e) {
      s_a[threadIdx.x * VW + e] = tot_a[e];
      s_b[threadIdx.x * VW + e] = tot_b[e];
    }
  }
  __syncthreads();
  const int reps = static_cast<int>(p.reps), P = t.frags * VW;
  float* oa = cpart + int64_t(cta_row) * d.C;
  float* ob = oa + int64_t(cta_rows) * d.C;
  if (reps <= 16) {
    for (int c = threadIdx.x; c < d.C; c += blockDim.x) {
      float a = 0.f, b = 0.f;
      for (int k = 0; k < reps; ++k) {
        int q = c + off + k * d.C;
        if (q >= P) q -= P;
        a += s_a[q];
        b += s_b[q];
      }
      oa[c] = a;
      ob[c] = b;
    }
  } else {
    for (int c = warp; c < d.C; c += warps) {
      float a = 0.f, b = 0.f;
      for (int k = lane; k < reps; k += 32) {
        int q = c + off + k * d.C;
        if (q >= P) q -= P;
        a += s_a[q];
        b += s_b[q];
      }
      a = dev::warp_sum(a);
      b = dev::warp_sum(b);
      if (lane == 0) {
        oa[c] = a;
        ob[c] = b;
      }
    }
  }
}

// Joins the groups' sums over chunks and tiles: m1, m2 of each (n, g).
__global__ void __launch_bounds__(256)
k_gn_grad_join(const float* gpart, GnDims d, float* m1, float* m2) {
  dev::pdl_wait();
  dev::pdl_trigger();
  const int lane = threadIdx.x & 31;
  const int64_t parts = int64_t(d.p.chunks) * d.p.tiles;
  const float scale = 1.0f / (float(d.S) * float(d.D));
  for (int64_t i = int64_t(blockIdx.x) * 8 + (threadIdx.x >> 5); i < d.N * d.G; i += int64_t(gridDim.x) * 8) {
    const float2* src = reinterpret_cast<const float2*>(gpart) + (i / d.G) * parts * d.G + i % d.G;
    float a = 0.f, b = 0.f;
#pragma unroll 4
    for (int64_t k = lane; k < parts; k += 32) {
      const float2 v = __ldcg(src + k * d.G);
      a += v.x;
      b += v.y;
    }
    a = dev::warp_sum(a);
    b = dev::warp_sum(b);
    if (lane == 0) {
      m1[i] = a * scale;
      m2[i] = b * scale;
    }
  }
}

// Gradient, pass 2: dx.
template <typename T, int FORM, bool VEC, bool SILU>
__global__ void __launch_bounds__(kWalkThreads)
k_gn_grad_apply(const T* dy, const T* x, const T* __restrict__ gamma, const T* __restrict__ beta, const float* mean,
                const float* inv, const float* m1, const float* m2, T* dx, GnDims d) {
  constexpr int VW = dev::Vec16<T>::N;
  constexpr int EV = FORM == kGroup ? 1 : VW;
  constexpr int U = sizeof(T) == 4 ? 4 : 2;
  dev::pdl_wait();
  dev::pdl_trigger();
  const WalkPlan& p = d.p;
  const Tile t(p, FORM == kAny ? -1 : d.L / VW);
  if (!t.mine) return;
  const int64_t items = d.N * p.chunks;
  for (int64_t item = blockIdx.x / unsigned(p.tiles); item < items; item += gridDim.x / unsigned(p.tiles)) {
    const int64_t n = item / p.chunks, chunk = item - n * p.chunks;
    const T* xs = x + n * d.L;
    const T* ds = dy + n * d.L;
    T* os = dx + n * d.L;
    const int off = walk_offset<T, FORM, VEC>(xs);
    const int c0 = first_channel(t.j, VW, off, d.C);
    GradValues<T, EV, SILU> val;
    val.load(c0, n * d.G, d, gamma, beta, mean, inv);
    float a1[EV], a2[EV];
    for_channels<VW>(c0, d.C, d.D, [&](int e, int, int g) {
      if (e < EV) {
        a1[e] = __ldcg(m1 + n * d.G + g);
        a2[e] = __ldcg(m2 + n * d.G + g);
      }
    });
    auto value = [&](float (&v)[VW], float (&w)[VW]) {  // x, dy -> dx in v
      val(v, w);
#pragma unroll
      for (int e = 0; e < VW; ++e) {
        const int i = EV == 1 ? 0 : e;
        v[e] = val.rs[i] * (fmaf(w[e], val.ga[e], -a1[i]) - v[e] * a2[i]);
      }
    };
    const int64_t ra = chunk * p.rows_per_chunk, rb = min(t.rows, ra + p.rows_per_chunk);
    if constexpr (FORM != kAny) {
      const int64_t pitch = p.row_frags * VW, at = (ra * p.row_frags + t.j) * VW;
      const T* px = xs + at;
      const T* pd = ds + at;
      T* po = os + at;
      int64_t r = ra;
      for (; r + U <= rb; r += U, px += U * pitch, pd += U * pitch, po += U * pitch) {
        uint4 rx[U], rd[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
          rx[u] = dev::ld16_stream(px + u * pitch);
          rd[u] = dev::ld16_stream(pd + u * pitch);
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
          float v[VW], w[VW];
          dev::Conv<T>::unpack(rx[u], v);
          dev::Conv<T>::unpack(rd[u], w);
          value(v, w);
          dev::st16_stream(po + u * pitch, dev::Conv<T>::pack(v));
        }
      }
      for (; r < rb; ++r, px += pitch, pd += pitch, po += pitch) {
        float v[VW], w[VW];
        dev::Conv<T>::unpack(dev::ld16_stream(px), v);
        dev::Conv<T>::unpack(dev::ld16_stream(pd), w);
        value(v, w);
        dev::st16_stream(po, dev::Conv<T>::pack(v));
      }
    } else {
      for (int64_t r = ra; r < rb; ++r) {
        const int64_t e0 = (r * p.row_frags + t.j) * VW - off;
        float v[VW], w[VW];
        dev::load_frag<T, VEC>(xs, e0, d.L, v);
        dev::load_frag<T, VEC>(ds, e0, d.L, w);
        value(v, w);
        dev::store_frag<T, VEC>(os, e0, d.L, v);
      }
    }
  }
}

int64_t vec_width(DType t) { return t == DType::F32 ? 4 : 8; }

GnDims dims_of(DType t, int64_t N, int64_t S, int64_t C, int64_t G, float eps) {
  GnDims d{N, S, S * C, int(C), int(G), int(C / G), eps, {}};
  d.p = make_walk(d.L, C, int(vec_width(t)), N, kPlanSms * 4, 4);
  return d;
}

// CTA rows (of `tiles` CTAs) of a launch over N * chunks items.
int64_t cta_rows_of(const GnDims& d, int64_t most_ctas) {
  return std::max<int64_t>(1, std::min(d.N * d.p.chunks, most_ctas / d.p.tiles));
}

bool split_parts(const GnDims& d) { return d.p.chunks > 1 || d.p.tiles > 1; }
int64_t grad_rows(const GnDims& d) { return cta_rows_of(d, kPlanSms * 4); }

// Offset in bytes of the next array in a workspace: each starts on 16 bytes.
size_t pad16(size_t b) { return (b + 15) / 16 * 16; }

struct GnWorkspace {
  size_t partial, mean, inv, total;
};
GnWorkspace gn_workspace(const GnDims& d) {
  GnWorkspace w;
  const size_t stats = pad16(size_t(d.N) * d.G * 4);
  w.partial = 0;
  w.mean = split_parts(d) ? pad16(size_t(d.N) * d.p.chunks * d.p.tiles * d.G * 12) : 0;
  w.inv = w.mean + stats;
  w.total = w.inv + stats;
  return w;
}

struct GnGradWorkspace {
  size_t gpart, m1, m2, cpart, total;
};
GnGradWorkspace gn_grad_workspace(const GnDims& d, DType t) {
  GnGradWorkspace w;
  const size_t stats = pad16(size_t(d.N) * d.G * 4);
  const int64_t width = d.p.tiles > 1 ? d.p.row_frags * vec_width(t) : d.C;
  w.gpart = 0;
  w.m1 = pad16(size_t(d.N) * d.p.chunks * d.p.tiles * d.G * 8);
  w.m2 = w.m1 + stats;
  w.cpart = w.m2 + stats;
  w.total = w.cpart + size_t(grad_rows(d)) * width * 8;
  return w;
}

inline unsigned misalign16(const void* p) { return unsigned(reinterpret_cast<uintptr_t>(p) & 15u); }

inline unsigned join_grid(const GnDims& d) {
  return unsigned(std::min<int64_t>((d.N * d.G + 7) / 8, kPlanSms * 8));
}

template <typename T>
cudaError_t group_norm_t(const GroupNormArgs& a, int sm_count, cudaStream_t stream, int* launches) {
  const GnDims d = dims_of(a.t, a.N, a.S, a.C, a.G, a.eps);
  const GnWorkspace w = gn_workspace(d);
  char* ws = static_cast<char*>(a.workspace);
  float* mean = a.mean != nullptr ? a.mean : reinterpret_cast<float*>(ws + w.mean);
  float* inv = a.inv != nullptr ? a.inv : reinterpret_cast<float*>(ws + w.inv);
  float* partial = split_parts(d) ? reinterpret_cast<float*>(ws + w.partial) : nullptr;
  const T* x = static_cast<const T*>(a.x);
  const T* gamma = static_cast<const T*>(a.gamma);
  const T* beta = static_cast<const T*>(a.beta);
  T* y = static_cast<T*>(a.y);
  const dim3 grid(unsigned(cta_rows_of(d, int64_t(sm_count) * 8) * d.p.tiles)), block(d.p.threads);
  const int whole = a.C % dev::Vec16<T>::N == 0 ? (d.D % dev::Vec16<T>::N == 0 ? kGroup : kChannel) : kAny;
  const int form1 = misalign16(x) == 0 ? whole : kAny;  // statistics need no alignment of y
  auto f1 = form1 == kGroup ? k_gn_stats<T, kGroup> : form1 == kChannel ? k_gn_stats<T, kChannel> : k_gn_stats<T, kAny>;
  cudaError_t e = launch(f1, grid, block, 0, stream, x, d, partial, mean, inv);
  if (e != cudaSuccess) return e;
  *launches += 1;
  if (partial != nullptr) {
    e = launch(k_gn_join<T>, dim3(join_grid(d)), dim3(256), 0, stream, x, partial, d, mean, inv);
    if (e != cudaSuccess) return e;
    *launches += 1;
  }
  const bool vec = misalign16(x) == misalign16(y);
  auto pick = [&](auto silu) {
    constexpr bool kSilu = decltype(silu)::value;
    if (!vec) return k_gn_apply<T, kAny, false, kSilu>;
    return form1 == kGroup     ? k_gn_apply<T, kGroup, true, kSilu>
           : form1 == kChannel ? k_gn_apply<T, kChannel, true, kSilu>
                               : k_gn_apply<T, kAny, true, kSilu>;
  };
  auto fn = a.silu ? pick(std::true_type{}) : pick(std::false_type{});
  e = launch(fn, grid, block, 0, stream, x, gamma, beta, mean, inv, y, d);
  if (e == cudaSuccess) *launches += 1;
  return e;
}

template <typename T>
cudaError_t group_norm_grad_t(const GroupNormGradArgs& a, int sm_count, cudaStream_t stream, int* launches) {
  constexpr int VW = dev::Vec16<T>::N;
  const GnDims d = dims_of(a.t, a.N, a.S, a.C, a.G, 0.f);
  const GnGradWorkspace w = gn_grad_workspace(d, a.t);
  char* ws = static_cast<char*>(a.workspace);
  float* gpart = reinterpret_cast<float*>(ws + w.gpart);
  float* m1 = reinterpret_cast<float*>(ws + w.m1);
  float* m2 = reinterpret_cast<float*>(ws + w.m2);
  float* cpart = a.dgamma != nullptr || a.dbeta != nullptr ? reinterpret_cast<float*>(ws + w.cpart) : nullptr;
  const T* x = static_cast<const T*>(a.x);
  const T* dy = static_cast<const T*>(a.dy);
  const T* gamma = static_cast<const T*>(a.gamma);
  const T* beta = static_cast<const T*>(a.beta);
  T* dx = static_cast<T*>(a.dx);
  const int64_t rows = grad_rows(d);
  // whole fragments need x and dy (and dx) at one offset within 16 bytes, and
  // one walk offset for all the samples that a CTA takes
  const bool one_off = d.L % VW == 0 || rows >= d.N * d.p.chunks;
  const bool vec1 = misalign16(x) == misalign16(dy) && one_off;
  const bool vec2 = misalign16(x) == misalign16(dy) && misalign16(x) == misalign16(dx);
  const int whole = misalign16(x) != 0 || a.C % VW != 0 ? kAny : d.D % VW == 0 ? kGroup : kChannel;
  auto pick1 = [&](auto silu) {
    constexpr bool kSilu = decltype(silu)::value;
    if (!vec1) return k_gn_grad_sums<T, kAny, false, kSilu>;
    return whole == kGroup     ? k_gn_grad_sums<T, kGroup, true, kSilu>
           : whole == kChannel ? k_gn_grad_sums<T, kChannel, true, kSilu>
                               : k_gn_grad_sums<T, kAny, true, kSilu>;
  };
  auto f1 = a.silu ? pick1(std::true_type{}) : pick1(std::false_type{});
  cudaError_t e = launch(f1, dim3(unsigned(rows * d.p.tiles)), dim3(d.p.threads), 0, stream, dy, x, gamma, beta, a.mean,
                         a.inv, d, gpart, cpart);
  if (e != cudaSuccess) return e;
  *launches += 1;
  e = launch(k_gn_grad_join, dim3(join_grid(d)), dim3(256), 0, stream, gpart, d, m1, m2);
  if (e != cudaSuccess) return e;
  *launches += 1;
  auto pick2 = [&](auto silu) {
    constexpr bool kSilu = decltype(silu)::value;
    if (!vec2) return k_gn_grad_apply<T, kAny, false, kSilu>;
    return whole == kGroup     ? k_gn_grad_apply<T, kGroup, true, kSilu>
           : whole == kChannel ? k_gn_grad_apply<T, kChannel, true, kSilu>
                               : k_gn_grad_apply<T, kAny, true, kSilu>;
  };
  auto f2 = a.silu ? pick2(std::true_type{}) : pick2(std::false_type{});
  const dim3 grid(unsigned(cta_rows_of(d, int64_t(sm_count) * 8) * d.p.tiles));
  e = launch(f2, grid, dim3(d.p.threads), 0, stream, dy, x, gamma, beta, a.mean, a.inv, m1, m2, dx, d);
  if (e != cudaSuccess) return e;
  *launches += 1;
  if (cpart != nullptr) {
    const int64_t jobs = std::min<int64_t>((int64_t(d.C) + 31) / 32 * 2, INT_MAX);
    // the sums of du are dbeta, those of du * h are dgamma
    e = launch(k_channel_sums<T>, dim3(unsigned(jobs)), dim3(kSumsThreads), 0, stream, cpart, rows,
               d.p.tiles > 1 ? d.p.reps : int64_t(1), int64_t(d.C), 2, static_cast<T*>(a.dbeta), static_cast<T*>(a.dgamma));
    if (e == cudaSuccess) *launches += 1;
  }
  return e;
}

}  // namespace

size_t group_norm_workspace_bytes(DType t, int64_t N, int64_t S, int64_t C, int64_t G) {
  return gn_workspace(dims_of(t, N, S, C, G, 0.f)).total;
}

size_t group_norm_grad_workspace_bytes(DType t, int64_t N, int64_t S, int64_t C, int64_t G) {
  return std::max(gn_grad_workspace(dims_of(t, N, S, C, G, 0.f), t).total,
                  group_norm_grad_fused_bytes(t, N, S, C, G));
}

cudaError_t launch_group_norm(const GroupNormArgs& a, int sm_count, cudaStream_t stream, int* launches) {
  bool done = false;
  const cudaError_t e = launch_group_norm_fused(a, sm_count, stream, launches, &done);
  if (done || e != cudaSuccess) return e;
  switch (a.t) {
    case DType::F32: return group_norm_t<float>(a, sm_count, stream, launches);
    case DType::F16: return group_norm_t<__half>(a, sm_count, stream, launches);
    default: return group_norm_t<__nv_bfloat16>(a, sm_count, stream, launches);
  }
}

cudaError_t launch_group_norm_grad(const GroupNormGradArgs& a, int sm_count, cudaStream_t stream, int* launches) {
  bool done = false;
  const cudaError_t e = launch_group_norm_grad_fused(a, sm_count, stream, launches, &done);
  if (done || e != cudaSuccess) return e;
  switch (a.t) {
    case DType::F32: return group_norm_grad_t<float>(a, sm_count, stream, launches);
    case DType::F16: return group_norm_grad_t<__half>(a, sm_count, stream, launches);
    default: return group_norm_grad_t<__nv_bfloat16>(a, sm_count, stream, launches);
  }
}

}  // namespace ep

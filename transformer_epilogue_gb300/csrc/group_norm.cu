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
// Five forms, in the order in which they are tried:
//   staged tokens (here)    S = 1, groups of 1, 2, 4 ... 32 fragments, from 1 MB (the
//                           gradient 2 MB) on: one launch at the copy rate's 75 %
//                           (bf16 8192x1x4096 27 us; the gradient 8192x1x2048 25)
//   tokens                  group_norm_fused.cu: S = 1, groups of whole fragments
//   fused                   group_norm_fused.cu: a sample fits a block's registers
//   staged split (here)     any other size with 16-byte-aligned tensors whose channels
//                           repeat within a block's 256 fragments (or C % VW == 0)
//   general split (here)    everything else
// The split forms walk each sample as column_walk.cuh describes.  Pass 1 leaves
// (count, centre, mean - centre, sum of squared distances from the mean) per chunk
// and group, a small kernel (or pass 2 itself) joins the chunks, pass 2 reads x again,
// from L2 where it fits, and writes y.  The statistics are taken relative to values
// near their mean throughout, and a part keeps its own centre beside the distance
// from it, so that neither a large mean nor an outlying value costs them digits.  The gradient has
// the same three steps, with per-channel sums of du and du * h beside the groups'.
// A split form's floor is three reads and writes, not two, where x is larger than
// L2: bf16 8x16384x512 (134 MB) takes 65 us, 60 at the copy rate; small ones are
// bound by the latency of their launches (f16 2x4096x320 9.4 us, of which 1.6 are
// its bytes).  Scratch: a part for each chunk and each group that a tile of it meets.
//
// All sums and statistics are float32; results are rounded once, to T.
#include <algorithm>
#include <climits>
#include <type_traits>

#include "column_walk.cuh"
#include "device_common.cuh"
#include "group_norm.cuh"
#include "launch_util.h"
#include "smem_limit.h"
#include "tma_pipe.cuh"
#include "training_internal.h"

namespace ep {
namespace {

// One call's sizes, as every kernel of the split form gets them (C is at most
// kMaxGroupNormChannels, so positions in a walk row fit an int).
struct GnDims {
  int64_t N, S, L;  // L = S * C
  int C, G, D;
  float eps;
  // whole fragments of a sample, the walk rows that are full and the rest
  int64_t frags, full_rows;
  int rest;
  bool pvec;  // gamma and beta 16-byte aligned (and every fragment's channels one after another)
  bool here;  // pass 2 joins the chunks itself
  int slots;  // groups that a tile of the walk row can meet: its parts of an item
  bool staged, shifted;  // how the parts lie: see Slots; shifted: walks start before their sample
  int64_t ctas;  // CTAs that the plan is made for
  WalkPlan p;
};

// a / b where a mostly fits 32 bits.
__device__ __forceinline__ int64_t quotient(int64_t a, int b) {
  return a <= int64_t(0xffffffffu) ? int64_t(uint32_t(a) / uint32_t(b)) : a / b;
}

// Where a sample's walk row starts: `off` elements before the sample.
template <typename T, bool VEC>
__device__ __forceinline__ int walk_offset(const T* sample) {
  return VEC ? dev::misalignment(sample) : 0;
}

// The channel of the first element of fragment column j.
__device__ __forceinline__ int first_channel(int64_t j, int vw, int off, int C) {
  return static_cast<int>((unsigned(j) * unsigned(vw) + unsigned(C - off % C)) % unsigned(C));
}

// The first repeat k of a group whose channels [c0, c0 + D), at the positions
// off + c + k C of a walk row, reach past position p0 (k < 0: the channels that
// the walk row's `off` leading positions hold).
__device__ __forceinline__ int first_repeat(int p0, int off, int c0, int D, int C) {
  const int a = p0 - off - c0 - D;
  return (a >= 0 ? a / C : -((-a + C - 1) / C)) + 1;
}

// The positions of a tile that hold a group's channels, by the lanes of a warp.
// `cols` lanes (a power of two) stand side
// by side over the group's channels, and as many of its repeats as fit a warp
// next to each other, so that few channels still use (and sum over) all lanes.
struct GroupWalk {
  int np, C, D, reps, cols;
  int p0;         // the tile's first position
  bool whole;     // the tile is the walk row: positions wrap around
  __device__ __forceinline__ GroupWalk(const WalkPlan& p, int tile, int frags, int C_, int D_, int vw) {
    np = frags * vw;
    C = C_;
    D = D_;
    whole = p.tiles == 1;
    p0 = tile * p.tile_frags * vw;
    reps = whole ? static_cast<int>(p.reps) : 0;
    cols = D >= 32 ? 32 : D <= 1 ? 1 : 1 << (32 - __clz(D - 1));
  }
  template <typename F>
  __device__ __forceinline__ void run(int g, int off, F f) const {
    const int lane = threadIdx.x & 31, j0 = lane & (cols - 1), ks = 32 / cols;
    if (whole) {
      const int start = off + g * D;
      for (int k = lane / cols; k < reps; k += ks) {
        for (int j = j0; j < D; j += cols) {
          int pos = start + j + k * C;
          if (pos >= np) pos -= np;
          f(pos);
        }
      }
    } else {
      const int c0 = g * D;
      for (int64_t a = off + c0 + int64_t(first_repeat(p0, off, c0, D, C) + lane / cols) * C - p0; a < np;
           a += int64_t(C) * ks) {
        const int lo = static_cast<int>(max(int64_t(0), a)), hi = static_cast<int>(min(int64_t(np), a + D));
        for (int i = lo + j0; i < hi; i += cols) f(i);
      }
    }
  }
  __device__ __forceinline__ bool has(int g, int off) const {
    return whole || off + g * D + int64_t(first_repeat(p0, off, g * D, D, C)) * C < p0 + np;
  }
};

// A CTA's place: its tile of the walk row and its thread's fragment column.
struct Tile {
  int tile, frags;   // the tile's number and fragments
  int64_t j;         // fragment column
  bool mine;
  __device__ __forceinline__ explicit Tile(const WalkPlan& p) {
    tile = p.tiles == 1 ? 0 : static_cast<int>(blockIdx.x % unsigned(p.tiles));
    frags = static_cast<int>(min(int64_t(p.tile_frags), p.row_frags - int64_t(tile) * p.tile_frags));
    j = int64_t(tile) * p.tile_frags + threadIdx.x;
    mine = int(threadIdx.x) < frags;
  }
};

// Items of a CTA, first to last or (reversed: the pass that finds in L2 what
// the pass before read last) last to first.
struct Items {
  int64_t items, step, at;
  bool reversed;
  __device__ __forceinline__ Items(const GnDims& d, bool rev) : items(d.N * d.p.chunks), reversed(rev) {
    at = blockIdx.x / unsigned(d.p.tiles);
    step = gridDim.x / unsigned(d.p.tiles);
  }
  __device__ __forceinline__ bool more() const { return at < items; }
  __device__ __forceinline__ int64_t item() const { return reversed ? items - 1 - at : at; }
  __device__ __forceinline__ void next() { at += step; }
};

// The walk rows [ra, rb) of an item, and its sample.  `rows`: of a sample.
struct Range {
  int64_t n, ra, rb;
  __device__ __forceinline__ Range(const WalkPlan& p, int64_t item, int64_t rows) {
    n = p.chunks == 1 ? item : quotient(item, p.chunks);
    ra = (item - n * p.chunks) * p.rows_per_chunk;
    rb = min(rows, ra + p.rows_per_chunk);
  }
};

// A sample as the staged kernels read it: `nf` fragments from fragment f0 of the
// tensor on, the first `off` elements of which belong to the sample before.
// (Off and the ends matter where C % VW != 0: ODD.)
struct Sample {
  int off;
  int64_t f0, nf;
};

// An item's parts: `slots` for each tile of the walk row, from the tile's first group
// on (modulo G), so that scratch grows with the groups and not with groups x tiles
// (f16 1x64x65536 in 65536 groups: 303 MB to 10).
//  staged: channels do not wrap around in a tile, so group g is in the tiles t0 ...
//  that its channels reach, in all but the first of them as the first group;
//  general: a tile's channels may wrap around and start off the sample; the join looks
//  at every tile.  Where a tile has a slot for every group, slot g is group g.
struct Slots {
  int slots, G, first;
  __device__ __forceinline__ Slots(const GnDims& d, int tile, int off, int vw) : slots(d.slots), G(d.G), first(0) {
    if (slots < G || (d.staged && d.p.tiles > 1))
      first = first_channel(int64_t(tile) * d.p.tile_frags, vw, off, d.C) / d.D;
  }
  __device__ __forceinline__ int group(int s) const { return first + s < G ? first + s : first + s - G; }
  __device__ __forceinline__ int slot(int g) const { return g >= first ? g - first : g - first + G; }
};

// The parts of group g of a sample on staged rows of several tiles, by index: where part
// k stands, counted in slots from the sample's first.  No branches: the join's loads go
// out together.
struct GroupParts {
  unsigned count, of_chunk, magic;  // magic: 2^32 / of_chunk, rounded up
  int tiles, slots, base0, base1;   // the first and the other parts of a chunk
  __device__ __forceinline__ GroupParts(const GnDims& d, int g, int vw) : tiles(d.p.tiles), slots(d.slots) {
    const int e0 = g * d.D, tile = d.p.tile_frags * vw, t0 = e0 / tile;
    of_chunk = (e0 + d.D - 1) / tile - t0 + 1;
    base1 = t0 * slots;
    base0 = base1 + g - t0 * tile / d.D;
    count = unsigned(d.p.chunks) * of_chunk;
    magic = of_chunk > 1 ? 0xffffffffu / of_chunk + 1u : 0u;
  }
  template <typename F>
  __device__ __forceinline__ F load(const F* src, unsigned k) const {
    unsigned chunk = of_chunk > 1 ? __umulhi(k, magic) : k;
    if (chunk * of_chunk > k) --chunk;  // (k of_chunk from 2^32 on: one too many at most)
    const unsigned i = k - chunk * of_chunk;
    return k < count ? __ldcg(src + int64_t(chunk * unsigned(tiles) + i) * slots + (i == 0 ? base0 : base1)) : F{};
  }
};

// The same where a tile meets some of the groups and channels wrap around in it:
// every tile is looked at.
struct ScannedParts {
  const GnDims& d;
  int g, vw, off;
  unsigned count;
  __device__ __forceinline__ ScannedParts(const GnDims& d_, int g_, int vw_, int off_)
      : d(d_), g(g_), vw(vw_), off(off_), count(unsigned(d_.p.chunks) * d_.p.tiles) {}
  template <typename F>
  __device__ __forceinline__ F load(const F* src, unsigned k) const {
    if (k >= count) return F{};
    const int s = Slots(d, static_cast<int>(k % unsigned(d.p.tiles)), off, vw).slot(g);
    return s < d.slots ? __ldcg(src + int64_t(k) * d.slots + s) : F{};
  }
};

// The same where slot g is group g in every tile.
struct LinearParts {
  unsigned count;
  int slots, g;
  __device__ __forceinline__ LinearParts(const GnDims& d, int g_)
      : count(unsigned(d.p.chunks) * d.p.tiles), slots(d.slots), g(g_) {}
  template <typename F>
  __device__ __forceinline__ F load(const F* src, unsigned k) const {
    return k < count ? __ldcg(src + int64_t(k) * slots + g) : F{};
  }
};

// f(parts) for those of group g of the sample that starts at xs.  How they are found is
// the kernel's own (WAY): a join runs once, and code that it does not need costs it
// instruction fetches (f16 2x4096x320 with all ways in one kernel 10.5 us, 10.1 apart).
template <typename T, int WAY, typename F>
__device__ __forceinline__ void with_parts(const GnDims& d, int g, const T* xs, F f) {
  constexpr int VW = dev::Vec16<T>::N;
  if constexpr (WAY == 0) {
    f(LinearParts(d, g));
  } else if constexpr (WAY == 1) {
    f(GroupParts(d, g, VW));
  } else {
    f(ScannedParts(d, g, VW, d.shifted ? dev::misalignment(xs) : 0));
  }
}
inline int way_of(const GnDims& d) { return d.p.tiles == 1 || (!d.staged && d.slots == d.G) ? 0 : d.staged ? 1 : 2; }

// An item's partial fragments, if this thread has one: the sample's first (before
// `lo` outside) and last (from `hi` on), by their row in the item.  They are
// read from global memory, value by value: the tensor's last one is not staged.
struct Ends {
  int first = -1, last = -1, lo = 0, hi = 0;
  int64_t e0 = 0, pitch = 0;  // the thread's first element in the item, from the sample's start
  __device__ __forceinline__ bool has(int row) const { return row == first || row == last; }
  __device__ __forceinline__ bool inside(int row, int e) const {
    return !(row == first && e < lo) && !(row == last && e >= hi);
  }
};

// ---------------------------------------------------------------------------
// Block epilogues of the general kernels: a warp to a group, with the walk row's
// offset and repeats.
// ---------------------------------------------------------------------------

// The threads' (count, centre, mean - centre, M2) for each position, in shared memory,
// to the item's groups: two sums, of the means' distances from one of them and then
// relative to the first's mean.
template <typename T>
__device__ __forceinline__ void join_statistics(const GnDims& d, const Tile& t, const Range& r, int64_t item, int off,
                                                int warps, const float* s_cnt, const float* s_ref, const float* s_mean,
                                                const float* s_m2, float4* partial, float* mean_out, float* inv_out) {
  const WalkPlan& p = d.p;
  const GroupWalk walk(p, t.tile, t.frags, d.C, d.D, dev::Vec16<T>::N);
  const int lane = threadIdx.x & 31;
  const Slots slots(d, t.tile, off, dev::Vec16<T>::N);
  for (int i = threadIdx.x >> 5; i < d.slots; i += warps) {
    const int g = slots.group(i);
    float4* out = partial + (item * p.tiles + t.tile) * d.slots + i;
    if (!walk.has(g, off)) {
      if (lane == 0) *out = make_float4(0.f, 0.f, 0.f, 0.f);
      continue;
    }
    float c = 0.f, s = 0.f, q = 0.f, ref = 0.f;
    walk.run(g, off, [&](int i) {  // relative to the lane's first mean
      const float n = s_cnt[i], z = s_ref[i], m = s_mean[i];
      if (c == 0.f) ref = z + m;
      c += n;
      s = fmaf(n, (z - ref) + m, s);
    });
    const float own = ref;
    ref = __shfl_sync(0xffffffffu, own, max(0, __ffs(__ballot_sync(0xffffffffu, c > 0.f)) - 1));
    s = dev::warp_sum(c > 0.f ? fmaf(c, own - ref, s) : 0.f);
    c = dev::warp_sum(c);
    const float mg = c > 0.f ? s / c : 0.f;
    float res = 0.f;  // what rounding s / c and the sum left out of the mean
    walk.run(g, off, [&](int i) {
      const float w = ((s_ref[i] - ref) + s_mean[i]) - mg;
      res = fmaf(s_cnt[i], w, res);
      q += fmaf(s_cnt[i] * w, w, s_m2[i]);
    });
    res = dev::warp_sum(res);
    q = dev::warp_sum(q);
    if (lane == 0) {
      const float fix = c > 0.f ? res / c : 0.f;
      const float mf = mg + fix, m2g = not_negative(q - res * fix);
      if (partial == nullptr) {
        mean_out[r.n * d.G + g] = ref + mf;
        inv_out[r.n * d.G + g] = 1.0f / sqrtf(m2g / c + d.eps);
      } else {
        *out = make_float4(c, ref, mf, m2g);
      }
    }
  }
}

// The positions' (sum du gamma, sum du gamma h), in shared memory, to the item's groups.
template <typename T>
__device__ __forceinline__ void join_group_sums(const GnDims& d, const Tile& t, int64_t item, int off, int warps,
                                                const float* s_a, const float* s_b, float* gpart) {
  const WalkPlan& p = d.p;
  const GroupWalk walk(p, t.tile, t.frags, d.C, d.D, dev::Vec16<T>::N);
  const int lane = threadIdx.x & 31;
  const Slots slots(d, t.tile, off, dev::Vec16<T>::N);
  for (int i = threadIdx.x >> 5; i < d.slots; i += warps) {
    const int g = slots.group(i);
    float a = 0.f, b = 0.f;
    if (walk.has(g, off)) {
      walk.run(g, off, [&](int i) {
        a += s_a[i];
        b += s_b[i];
      });
      a = dev::warp_sum(a);
      b = dev::warp_sum(b);
    }
    if (lane == 0) {
      float* out = gpart + ((item * p.tiles + t.tile) * d.slots + i) * 2;
      out[0] = a;
      out[1] = b;
    }
  }
}

// VW floats to their places in shared memory, 16 bytes at a time.
template <int VW>
__device__ __forceinline__ void put(float* s, const float (&v)[VW]) {
#pragma unroll
  for (int e = 0; e < VW; e += 4)
    *reinterpret_cast<float4*>(s + threadIdx.x * VW + e) = make_float4(v[e], v[e + 1], v[e + 2], v[e + 3]);
}

// v += a thread's places, as put left them.
template <int VW>
__device__ __forceinline__ void get_more(const float* s, float (&v)[VW]) {
#pragma unroll
  for (int e = 0; e < VW; e += 4) {
    const float4 t = *reinterpret_cast<const float4*>(s + threadIdx.x * VW + e);
    v[e] += t.x;
    v[e + 1] += t.y;
    v[e + 2] += t.z;
    v[e + 3] += t.w;
  }
}

// A CTA's channel sums, which its threads left at their positions in tot_a and
// tot_b, to row cta_row of cpart: 2 x [CTA row][C] (one tile), or 2 x [CTA row]
// [walk row], position 0 being channel 0.
template <typename T, typename SYNC>
__device__ __forceinline__ void leave_channel_sums(const GnDims& d, const Tile& t, int off, int threads,
                                                   const float* tot_a, const float* tot_b, float* cpart, SYNC sync) {
  constexpr int VW = dev::Vec16<T>::N;
  const WalkPlan& p = d.p;
  const int64_t cta_rows = gridDim.x / unsigned(p.tiles), cta_row = blockIdx.x / unsigned(p.tiles);
  if (p.tiles > 1) {
    if (t.mine) {
      const int64_t P = p.row_frags * VW;
      float* oa = cpart + cta_row * P;
      float* ob = oa + cta_rows * P;
#pragma unroll
      for (int e = 0; e < VW; ++e) {
        int64_t q = t.j * VW + e - off;
        if (q < 0) q += P;
        oa[q] = tot_a[threadIdx.x * VW + e];
        ob[q] = tot_b[threadIdx.x * VW + e];
      }
    }
    return;
  }
  sync();
  const int reps = static_cast<int>(p.reps), P = t.frags * VW, lane = threadIdx.x & 31;
  float* oa = cpart + cta_row * d.C;
  float* ob = oa + cta_rows * d.C;
  const int lanes = reps <= 16 ? 1 : 32;  // to a channel
  for (int c = threadIdx.x / lanes; c < d.C; c += threads / lanes) {
    float a = 0.f, b = 0.f;
    for (int k = lanes == 1 ? 0 : lane; k < reps; k += lanes) {
      int q = c + off + k * d.C;
      if (q >= P) q -= P;
      a += tot_a[q];
      b += tot_b[q];
    }
    if (lanes == 32) {
      a = dev::warp_sum(a);
      b = dev::warp_sum(b);
    }
    if (lanes == 1 || lane == 0) {
      oa[c] = a;
      ob[c] = b;
    }
  }
}

// The staged kernels' block sums, in two steps with all threads in both: over the
// repeats of each column (a channel, or a fragment of one group) in the tile, then
// over each group's columns.  (One warp to a group took 2400 instructions a warp
// for 2 x 4096 x 320, six times the streaming itself.)  Column i of the tile is
// at positions i + k cols; its group is i / D, counted from the tile's first column.
struct Columns {
  int cols, reps, D;       // in the tile, with D columns to a group
  int g0, n_groups, in0;   // the tile's first group, groups in it, columns of g0 before it
  __device__ __forceinline__ Columns(const GnDims& d, const Tile& t, int ev, int per) {
    const bool whole = d.p.tiles == 1;
    D = d.D / per;
    reps = whole ? static_cast<int>(d.p.reps) : 1;  // (more tiles: C % VW == 0, a walk row is C)
    cols = whole ? d.C / per : t.frags * ev;
    const int first = t.tile * d.p.tile_frags * ev;
    g0 = whole ? 0 : first / D;
    in0 = whole ? 0 : first - g0 * D;
    n_groups = whole ? d.G : (in0 + cols + D - 1) / D;
  }
  // The position of column i's repeat k (ODD: behind the first `off`, around the walk row's end).
  template <bool ODD>
  __device__ __forceinline__ int at(int i, int k, int off) const {
    int pos = i + k * cols;
    if constexpr (ODD) {
      pos += off;
      if (pos >= reps * cols) pos -= reps * cols;
    }
    return pos;
  }
  // Columns [lo, hi) of the tile's group g (from g0).
  __device__ __forceinline__ int lo(int g) const { return max(0, g * D - in0); }
  __device__ __forceinline__ int hi(int g) const { return min(cols, (g + 1) * D - in0); }
};

// ---------------------------------------------------------------------------
// What a thread does with its fragments.
// ---------------------------------------------------------------------------

// The VW channels of a parameter from c on (modulo C), `vec`: 16 bytes at once.
template <typename T>
__device__ __forceinline__ void load_param(const T* __restrict__ param, int c, int C, bool vec,
                                           float (&v)[dev::Vec16<T>::N]) {
  if (vec) {
    dev::Conv<T>::unpack(dev::ld16_keep(param + c), v);
  } else {
#pragma unroll
    for (int e = 0; e < dev::Vec16<T>::N; ++e) {
      v[e] = dev::ld1_keep(param + c);
      if (++c == C) c = 0;
    }
  }
}

// mu of the thread's groups, and k scaled by their 1/sqrt(var + eps).  ld: how they
// are read.  What a join writes while this kernel may already have been launched is
// read by plain cached loads (__ldca, or through a generic pointer), never as
// read-only data.
struct PlainLoad {
  __device__ __forceinline__ float operator()(const float* p) const { return *p; }
};
struct CachedLoad {
  __device__ __forceinline__ float operator()(const float* p) const { return __ldca(p); }
};
template <int EV, int VW, typename LD>
__device__ __forceinline__ void scale_by_group(int c0, int64_t ng, const GnDims& d, const float* mean,
                                               const float* inv, float (&mu)[EV], float (&k)[VW], LD ld) {
  const float* m = mean + ng;
  const float* r = inv + ng;
  if constexpr (EV == 1) {
    const int g = c0 / d.D;
    mu[0] = ld(m + g);
    const float rg = ld(r + g);
#pragma unroll
    for (int e = 0; e < VW; ++e) k[e] *= rg;
  } else {
    for_channels<VW>(c0, d.C, d.D, [&](int e, int, int g) {
      mu[e] = ld(m + g);
      k[e] *= ld(r + g);
    });
  }
}

// A thread's channel values for the forward pass.
template <typename T, int EV, bool SILU>
struct ApplyValues {
  static constexpr int VW = dev::Vec16<T>::N;
  float mu[EV], a[VW], b[VW];
  __device__ __forceinline__ void load_params(int c0, const GnDims& d, const T* __restrict__ gamma,
                                              const T* __restrict__ beta) {
#pragma unroll
    for (int e = 0; e < VW; ++e) b[e] = 0.f;
    load_param(gamma, c0, d.C, d.pvec, a);
    if (beta != nullptr) load_param(beta, c0, d.C, d.pvec, b);
  }
  template <typename LD>
  __device__ __forceinline__ void scale(int c0, int64_t ng, const GnDims& d, const float* mean, const float* inv,
                                        LD ld) {
    scale_by_group(c0, ng, d, mean, inv, mu, a, ld);
  }
  __device__ __forceinline__ void operator()(float (&v)[VW]) const {
    centre_scale_add(v, mu, a, b);
    if constexpr (SILU) activate<T>(v);
  }
};

// The same for the gradient: x -> t = x - mu, dy -> du, with u = t (r gamma) + beta.
template <typename T, int EV, bool SILU>
struct GradValues {
  static constexpr int VW = dev::Vec16<T>::N;
  float mu[EV], k[VW], be[VW];  // k = r gamma
  __device__ __forceinline__ void load(int c0, int64_t ng, const GnDims& d, const T* __restrict__ gamma,
                                       const T* __restrict__ beta, const float* mean, const float* inv) {
#pragma unroll
    for (int e = 0; e < VW; ++e) be[e] = 0.f;
    load_param(gamma, c0, d.C, d.pvec, k);
    if (SILU && beta != nullptr) load_param(beta, c0, d.C, d.pvec, be);
    scale_by_group(c0, ng, d, mean, inv, mu, k, PlainLoad{});
  }
  __device__ __forceinline__ void operator()(float (&v)[VW], float (&w)[VW]) const {
#pragma unroll
    for (int e = 0; e < VW; e += 2) {
      const float2 m = pair_of<VW>(mu, e);
      const float2 t = __fadd2_rn(make_float2(v[e], v[e + 1]), make_float2(-m.x, -m.y));
      v[e] = t.x;
      v[e + 1] = t.y;
    }
    if constexpr (SILU) {
      float u[VW];
#pragma unroll
      for (int e = 0; e < VW; ++e) u[e] = be[e];
      fma_pairs(v, k, u);
      activate_grad<T>(w, u);
    }
  }
};

// dx = r (du gamma - m1 - h m2) = du k + (t q2 + q1), q2 = -r^2 m2, q1 = -r m1.
template <typename T, int EV, bool SILU>
struct GradApplyValues : GradValues<T, EV, SILU> {
  static constexpr int VW = dev::Vec16<T>::N;
  using Base = GradValues<T, EV, SILU>;
  float q1[EV], q2[EV];
  __device__ __forceinline__ void load_means(int c0, int64_t ng, const GnDims& d, const float* inv, const float* m1,
                                             const float* m2) {
    for_channels<VW>(c0, d.C, d.D, [&](int e, int, int g) {
      if (e < EV) {
        const float r = inv[ng + g];
        q1[e] = -r * __ldca(m1 + ng + g);
        q2[e] = -r * (r * __ldca(m2 + ng + g));
      }
    });
  }
  __device__ __forceinline__ void dx(float (&v)[VW], float (&w)[VW]) const {
    (*this)(v, w);
#pragma unroll
    for (int e = 0; e < VW; e += 2) {
      const float2 t = __ffma2_rn(make_float2(v[e], v[e + 1]), pair_of<VW>(q2, e), pair_of<VW>(q1, e));
      const float2 r = __ffma2_rn(make_float2(w[e], w[e + 1]), make_float2(Base::k[e], Base::k[e + 1]), t);
      v[e] = r.x;
      v[e + 1] = r.y;
    }
  }
};

// ---------------------------------------------------------------------------
// Staged walk rows (16-byte-aligned operands): a producer thread bulk-copies the
// rows of its CTA's items into a ring of shared-memory stages, the consumers (one to
// a fragment column) read them from there.  C % VW == 0: every fragment is whole,
// and a sample's last walk row may be shorter.  ODD, any other C whose period is one
// tile: samples start anywhere in a fragment, and the two partial fragments of a
// sample are read and written value by value (f16 3x13310x189 18 us; 36 with the
// general kernels).  The copies in flight cost no registers: with loads into
// registers two CTAs an SM had 32 KB in flight, and the passes took twice the time.
// Two stages of 32 KB and two CTAs an SM were best; three CTAs gave nothing.
// Stages are handed over by mbarriers (tma_pipe.cuh), with bounded waits; a
// consumer whose wait ran out takes no more rows but stays in step with the
// block's barriers.
// ---------------------------------------------------------------------------

constexpr int kStageBytes = 32768;   // of all operands together
constexpr int kStages = 2;
constexpr int kStageSmem = kStages * kStageBytes;

struct StageBars {
  uint64_t full[kStages], empty[kStages];
};

__device__ __forceinline__ uint64_t policy_evict_normal() {
  uint64_t pol;
  asm volatile("createpolicy.fractional.L2::evict_normal.b64 %0, 1.0;" : "=l"(pol));
  return pol;
}

template <typename T, int NOPS, bool ODD = false>
struct RowStream {
  static constexpr int VW = dev::Vec16<T>::N;
  StageBars* bars;
  unsigned char* smem;
  int rows;            // walk rows in a stage
  int row_bytes;       // of this tile
  int place;           // this thread's in a row (threads beyond the tile read its first fragment)
  int64_t total;       // walk rows of a sample (ODD: at most)
  int64_t frags, full_rows, row_frags, L, whole;
  int rest;
  dev::Ring ring;
  bool ok = true;

  __device__ __forceinline__ RowStream(StageBars* b, unsigned char* m, const GnDims& d, const Tile& t)
      : bars(b), smem(m), row_bytes(t.frags * 16), place(t.mine ? int(threadIdx.x) * 16 : 0), ring(kStages) {
    rows = kStageBytes / NOPS / row_bytes;  // >= 2: a tile has at most kWalkThreads fragments
    frags = d.frags;
    full_rows = d.full_rows;
    rest = d.rest;
    row_frags = d.p.row_frags;
    L = d.L;
    whole = d.N * d.L / VW;  // whole fragments of the tensor
    total = ODD ? d.p.rows : full_rows + (rest > 0 ? 1 : 0);
    if (threadIdx.x == 0) {
      for (int i = 0; i < kStages; ++i) {
        dev::mbar_init(&bars->full[i], 1);
        dev::mbar_init(&bars->empty[i], (blockDim.x - 32) / 32);
      }
      dev::mbar_init_fence();
    }
    __syncthreads();
  }

  __device__ __forceinline__ Sample sample(int64_t n) const {
    if constexpr (!ODD) return Sample{0, n * frags, frags};
    const int64_t e = n * L;
    const int off = static_cast<int>(e & (VW - 1));
    return Sample{off, e / VW, (off + L + VW - 1) / VW};
  }
  // An item's rows (ODD: the sample's own count of them).
  __device__ __forceinline__ Range range(const WalkPlan& p, int64_t item) const {
    Range r(p, item, total);
    if constexpr (ODD) r.rb = min(r.rb, quotient(sample(r.n).nf + row_frags - 1, int(row_frags)));
    return r;
  }
  // Walk rows of a sample that have a fragment j.
  __device__ __forceinline__ int64_t of_column(const Sample& s, int64_t j) const {
    if constexpr (ODD) return quotient(s.nf - j + row_frags - 1, int(row_frags));
    return full_rows + (j < rest ? 1 : 0);
  }
  __device__ __forceinline__ Ends ends(const Range& r, const Tile& t) const {
    Ends en;
    if constexpr (ODD) {
      const Sample s = sample(r.n);
      en.e0 = (r.ra * row_frags + t.j) * VW - s.off;
      en.pitch = row_frags * VW;
      if (t.mine) {
        if (s.off > 0 && t.j == 0 && r.ra == 0) en.first = 0;
        const int64_t last_row = quotient(s.nf - 1, int(row_frags));
        en.lo = s.off;
        en.hi = static_cast<int>(s.off + L - (s.nf - 1) * VW);
        if (en.hi < VW && t.j == s.nf - 1 - last_row * row_frags && last_row >= r.ra && last_row < r.rb)
          en.last = static_cast<int>(last_row - r.ra);
      }
    }
    return en;
  }

  // The producer: the rows of all the CTA's items.
  __device__ __forceinline__ void produce(const T* const (&base)[NOPS], const GnDims& d, const Tile& t, bool reversed,
                                          uint64_t policy) {
    const WalkPlan& p = d.p;
    int64_t n_filled = 0;
    for (Items it(d, reversed); it.more(); it.next()) {
      const Range range = this->range(p, it.item());
      const Sample s = sample(range.n);
      for (int64_t r = range.ra; r < range.rb; r += rows, ring.next(), ++n_filled) {
        if (n_filled >= kStages && !dev::mbar_wait(&bars->empty[ring.st], ring.phase ^ 1u)) {
          // the copies in flight land before the block ends
          for (int64_t k = n_filled - kStages; k < n_filled; ++k)
            dev::mbar_wait(&bars->full[k % kStages], uint32_t((k / kStages) & 1));
          return;
        }
        const int64_t f0 = s.f0 + r * p.row_frags + int64_t(t.tile) * p.tile_frags;
        const int k = static_cast<int>(min(int64_t(rows), range.rb - r));
        unsigned char* dst = smem + ring.st * kStageBytes;
        if (p.tiles == 1) {  // contiguous; the sample's last walk row may be short
          const int64_t left = ODD ? min(s.nf - r * p.row_frags, whole - f0) : frags - r * p.row_frags;
          const uint32_t bytes = uint32_t(min(int64_t(k) * p.row_frags, left)) * 16u;
          dev::mbar_arrive_expect_tx(&bars->full[ring.st], NOPS * bytes);
#pragma unroll
          for (int o = 0; o < NOPS && bytes > 0; ++o)
            dev::bulk_g2s(dst + o * (kStageBytes / NOPS), base[o] + f0 * VW, bytes, &bars->full[ring.st], policy);
        } else {
          dev::mbar_arrive_expect_tx(&bars->full[ring.st], uint32_t(NOPS * k * row_bytes));
          for (int i = 0; i < k; ++i)
#pragma unroll
            for (int o = 0; o < NOPS; ++o)
              dev::bulk_g2s(dst + o * (kStageBytes / NOPS) + i * row_bytes, base[o] + (f0 + i * p.row_frags) * VW,
                            uint32_t(row_bytes), &bars->full[ring.st], policy);
        }
      }
    }
  }

  // A consumer: f(row, src) for each stage of an item, row the stage's first,
  // counted from the item's first, and src the thread's place in it.
  template <typename F>
  __device__ __forceinline__ void stages(const Range& range, F f) {
    const int n = static_cast<int>(range.rb - range.ra);
    for (int r = 0; r < n; r += rows, ring.next()) {
      ok = ok && dev::mbar_wait(&bars->full[ring.st], ring.phase);
      if (!__all_sync(0xffffffffu, ok)) {
        ok = false;
        continue;
      }
      f(r, smem + ring.st * kStageBytes + place);
      dev::release_stage(&bars->empty[ring.st]);
    }
  }
  template <int R>
  __device__ __forceinline__ void load(const unsigned char* src, int i, uint4 (&raw)[R][NOPS]) const {
#pragma unroll
    for (int u = 0; u < R; ++u)
#pragma unroll
      for (int o = 0; o < NOPS; ++o)
        raw[u][o] = dev::lds16(src + o * (kStageBytes / NOPS) + (i + u) * row_bytes);
  }
  // f(row, raw) for the walk rows of an item that have a fragment in the thread's
  // column; raw holds four (or at most MOST), two or one rows, so that one row's
  // arithmetic covers another's latency.  start(row): before each stage.
  struct Nothing {
    __device__ __forceinline__ void operator()(int) const {}
  };
  template <int MOST = 4, typename F, typename S = Nothing>
  __device__ __forceinline__ void consume(const Range& range, int mine, F f, S start = S{}) {
    stages(range, [&](int r, const unsigned char* src) {
      start(r);
      const int k = min(rows, mine - r);
      int i = 0;
      for (; i + MOST <= k; i += MOST) {
        uint4 raw[MOST][NOPS];
        load(src, i, raw);
        f(r + i, raw);
      }
      if (MOST > 2 && i + 1 < k) {
        uint4 raw[2][NOPS];
        load(src, i, raw);
        f(r + i, raw);
        i += 2;
      }
      if (MOST > 1 && i < k) {
        uint4 raw[1][NOPS];
        load(src, i, raw);
        f(r + i, raw);
      }
    });
  }
  // Rows of an item that have a fragment in column j (0 where the thread has none).
  __device__ __forceinline__ int mine(const Range& range, const Tile& t) const {
    return t.mine ? static_cast<int>(max(int64_t(0), min(range.rb, of_column(sample(range.n), t.j)) - range.ra)) : 0;
  }
};

// The barrier of a staged kernel's consumers.
__device__ __forceinline__ void consumer_sync() { dev::named_barrier_sync(1, blockDim.x - 32); }

// Pass 1.  partial: [item][tile][slot] x (count, centre, mean - centre, M2).  The block
// takes its values relative to a centre of each group, so that its sums and sums of
// squares simply add up: the median of three of the group's values in the item's first,
// middle and last position.  Off by k standard deviations it multiplies the rounding of
// the sums by 1 + k^2; where far_off() shows k > 4 (two of the three are outliers) the
// item is gone over again about the mean so found, from L2, and the groups whose
// centre stays get the same sums again (where every item has to: f32 160x1024x516 in 4
// groups 197 us to 437, bf16 8x16384x512 80 to 124).  A thread adds kSumRows rows one after
// another, then those sums.  (Items of so many rows at most instead: f16 1x8388608x256
// 2023 us, not 1915.)
constexpr int kSumRows = 256;

template <typename T, bool GROUP, bool ODD>
__global__ void __launch_bounds__(kWalkThreads + 32, 2)
k_gn_stats_staged(const T* x, GnDims d, float4* partial) {
  constexpr int VW = dev::Vec16<T>::N;
  constexpr int EV = GROUP ? 1 : VW;
  extern __shared__ __align__(128) unsigned char smem[];
  __shared__ __align__(8) StageBars bars;
  // after the stages: two sums by position, the centres of the tile's groups
  float* s_a = reinterpret_cast<float*>(smem + kStageSmem);
  float* s_b = s_a + kWalkThreads * EV;
  float* centre = s_b + kWalkThreads * EV;
  const WalkPlan& p = d.p;
  const Tile t(p);
  RowStream<T, 1, ODD> rows(&bars, smem, d, t);
  dev::pdl_wait();
  dev::pdl_trigger();
  const int consumers = blockDim.x - 32;
  if (int(threadIdx.x) >= consumers) {
    const T* const base[1] = {x};
    if (int(threadIdx.x) == consumers) rows.produce(base, d, t, false, policy_evict_normal());
    return;
  }
  const Columns cols(d, t, EV, GROUP ? VW : 1);
  const int per = GROUP ? VW : 1;  // elements of a column
  int grp[EV];
  {
    int g = (t.mine ? int(threadIdx.x) * EV % cols.cols : 0) + cols.in0, in = g % cols.D;
    g /= cols.D;
#pragma unroll
    for (int e = 0; e < EV; ++e) {
      grp[e] = g;
      if (++in == cols.D) {
        in = 0;
        if (++g == cols.n_groups) g = 0;  // the next repeat of the channels
      }
    }
  }
  for (Items it(d, false); it.more(); it.next()) {
    const Range r = rows.range(p, it.item());
    float4* out = partial + (it.item() * p.tiles + t.tile) * d.slots;
    if (r.ra >= r.rb) {  // the plan's rows may be one more than there are
      for (int g = threadIdx.x; g < d.slots; g += consumers) out[g] = make_float4(0.f, 0.f, 0.f, 0.f);
      continue;
    }
    const int off = ODD ? rows.sample(r.n).off : 0;
    const Ends ends = rows.ends(r, t);
    const T* xs = x + r.n * d.L;
    // ODD: the item's elements of the sample
    auto from = [&] { return max(int64_t(0), r.ra * p.row_frags * VW - off); };
    auto to = [&] { return min(d.L, r.rb * p.row_frags * VW - off); };
    {
      // positions of the sample (repeats of the channels) in the item (ODD: that begin in it)
      int64_t pos0 = r.ra * p.reps, pos1 = min(r.rb * p.reps, d.S);
      if constexpr (ODD) {
        pos0 = min(quotient(from() + d.C - 1, d.C), d.S - 1);
        pos1 = max(pos0 + 1, quotient(to(), d.C));
        if (t.mine) for_channels<VW>(first_channel(t.j, VW, off, d.C), d.C, d.D, [&](int e, int, int g) { if (e < EV) grp[e] = g; });
      }
      const T* first = xs + pos0 * d.C + int64_t(t.tile) * p.tile_frags * VW;
      const int64_t mid = (pos1 - 1 - pos0) / 2 * d.C, last = (pos1 - 1 - pos0) * d.C;
      for (int g = threadIdx.x; g < cols.n_groups; g += consumers) {
        const int lo = cols.lo(g) * per, n = (cols.hi(g) - cols.lo(g)) * per;
        centre[g] = centre3(dev::to_float(first[lo]), dev::to_float(first[mid + lo + n / 2]),
                            dev::to_float(first[last + lo + n - 1]));
      }
    }
    consumer_sync();
    const int mine = rows.mine(r, t);
    bool far = false;
    auto statistics = [&](auto second) {
      constexpr bool again = decltype(second)::value;
      float c[EV], s[VW], q[VW];
#pragma unroll
      for (int e = 0; e < VW; ++e) s[e] = q[e] = 0.f;
#pragma unroll
      for (int e = 0; e < EV; ++e) c[e] = centre[grp[e]];
      int begun = 0;  // the first row of these sums: earlier ones are in the thread's places
      auto leave = [&](int row) {
        if constexpr (EV == 1) {
#pragma unroll
          for (int e = 1; e < VW; ++e) {
            s[0] += s[e];
            q[0] += q[e];
          }
          s_a[threadIdx.x] = begun > 0 ? s_a[threadIdx.x] + s[0] : s[0];
          s_b[threadIdx.x] = begun > 0 ? s_b[threadIdx.x] + q[0] : q[0];
        } else {
          if (begun > 0) {
            get_more(s_a, s);
            get_more(s_b, q);
          }
          put(s_a, s);
          put(s_b, q);
        }
#pragma unroll
        for (int e = 0; e < VW; ++e) s[e] = q[e] = 0.f;
        begun = row;
      };
      auto add = [&](float (&v)[VW]) {
#pragma unroll
        for (int e = 0; e < VW; e += 2) {
          const float2 m = pair_of<VW>(c, e);
          const float2 w = __fadd2_rn(make_float2(v[e], v[e + 1]), make_float2(-m.x, -m.y));
          v[e] = w.x;
          v[e + 1] = w.y;
        }
        dev::add_pairs(s, v);
        fma_pairs(v, v, q);
      };
      auto centre_outside = [&](int row, float (&v)[VW]) {  // what is outside counts as the centre
#pragma unroll
        for (int e = 0; e < VW; ++e)
          if (!ends.inside(row, e)) v[e] = c[EV == 1 ? 0 : e];
      };
      if constexpr (!again) {
        auto take = [&](int row, const auto& raw) {
#pragma unroll
          for (const auto& one : raw) {
            float v[VW];
            dev::Conv<T>::unpack(one[0], v);
            if (ODD && ends.has(row)) {
              dev::load_frag<T, false>(xs, ends.e0 + row * ends.pitch, d.L, v);
              centre_outside(row, v);
            }
            ++row;
            add(v);
          }
        };
        rows.consume(r, mine, take, [&](int row) {
          if (row - begun >= kSumRows && t.mine) leave(row);
        });
      } else {
        const int64_t pitch = p.row_frags * VW, e0 = (r.ra * p.row_frags + t.j) * VW - off;
#pragma unroll 2
        for (int row = 0; row < mine; ++row) {
          if (row - begun >= kSumRows) leave(row);
          float v[VW];
          dev::load_frag<T, true>(xs, e0 + row * pitch, d.L, v);
          if (ODD && ends.has(row)) centre_outside(row, v);
          add(v);
        }
      }
      if (t.mine) leave(0);
      consumer_sync();
      // to the first repeat's place (ODD: to the centre's other side, after all places have been read)
      float* t_a = s_a;
      float* t_b = s_b;
      if (ODD) {
        t_a = centre + kWalkThreads * EV;
        t_b = t_a + kWalkThreads * EV;
      }
      if (ODD || cols.reps > 1) {
        sum_sets(consumers, cols.cols, cols.reps,
                 [&](int i, int k, float& a, float& b) {
                   const int pos = cols.at<ODD>(i, k, off);
                   a += s_a[pos];
                   b += s_b[pos];
                 },
                 [&](int i, float a, float b) {
                   t_a[i] = a;
                   t_b[i] = b;
                 });
        consumer_sync();
      }
      sum_sets(consumers, cols.n_groups, cols.D,
               [&](int g, int k, float& a, float& b) {
                 const int i = cols.lo(g) + k;
                 if (i < cols.hi(g)) {
                   a += t_a[i];
                   b += t_b[i];
                 }
               },
               [&](int g, float a, float b) {
                 float n;
                 if constexpr (ODD) {  // the group's values among the sample's first from(), first to()
                   const int64_t ea = from(), eb = to(), qa = quotient(ea, d.C), qb = quotient(eb, d.C);
                   const int ia = min(max(int(ea - qa * d.C) - g * d.D, 0), d.D);
                   const int ib = min(max(int(eb - qb * d.C) - g * d.D, 0), d.D);
                   n = float((qb - qa) * d.D + (ib - ia));
                 } else {
                   n = float(min(r.rb * p.reps, d.S) - r.ra * p.reps) * float((cols.hi(g) - cols.lo(g)) * per);
                 }
                 const float m = n > 0.f ? a / n : 0.f, m2 = not_negative(b - a * m);
                 out[g] = make_float4(n, centre[g], m, m2);
                 if (!again && far_off(a * m, m2)) {
                   centre[g] += m;
                   far = true;
                 }
               });
    };
    statistics(std::false_type{});
    if (!dev::named_barrier_and(1, consumers, !far)) {
      statistics(std::true_type{});
      consumer_sync();
    }
  }
}

// The statistics of sample n, joined by pass 2 itself (GnDims::here), by all
// consumers: neighbouring threads take neighbouring groups, the rest of the block
// the other parts.  The parts' means are taken relative to the median of three of
// them: one centre, and no part read twice.  Off by k of the group's standard
// deviations it costs the variance k^2 2^-24 of its value, and k^2 is less than
// the number of parts.
struct JoinHere {
  float a[kWalkThreads], b[kWalkThreads];       // by thread
  float mean[kWalkThreads], inv[kWalkThreads];  // by group
};
__device__ __forceinline__ void join_stats_here(const float4* partial, const GnDims& d, int64_t n, int threads,
                                                JoinHere& js) {
  const int slices = static_cast<int>(unsigned(threads) / unsigned(d.G));
  const int slice = static_cast<int>(threadIdx.x / unsigned(d.G)), g = threadIdx.x - slice * d.G;
  const float4* src = partial + n * d.p.chunks * d.G + g;
  const float4 first = __ldcg(src), last = __ldcg(src + (d.p.chunks - 1) * d.G);
  const float4 mid = __ldcg(src + (d.p.chunks - 1) / 2 * d.G);
  const float mean0 = first.y + first.z;
  const float centre = median3(mean0, mid.y + mid.z, last.x > 0.f ? last.y + last.z : mean0);  // (the last may be empty)
  float a = 0.f, b = 0.f;
  if (slice < slices) {
#pragma unroll 8
    for (int k = slice; k < d.p.chunks; k += slices) {
      const float4 v = __ldcg(src + k * d.G);
      const float w = (v.y - centre) + v.z, cw = v.x * w;
      a += cw;
      b += fmaf(cw, w, v.w);
    }
  }
  consumer_sync();  // (the sample before has been read)
  js.a[threadIdx.x] = a;
  js.b[threadIdx.x] = b;
  if (slice == 0) js.mean[g] = centre;
  consumer_sync();
  const float total = float(d.S) * float(d.D);
  sum_sets(threads, d.G, slices,
           [&](int i, int k, float& sa, float& sb) {
             sa += js.a[k * d.G + i];
             sb += js.b[k * d.G + i];
           },
           [&](int i, float sa, float sb) {
             const float m = sa / total;
             js.mean[i] += m;
             js.inv[i] = 1.0f / sqrtf(not_negative(sb - sa * m) / total + d.eps);
           });
  consumer_sync();
}

// Pass 2: y from x and the statistics, over the items in reverse: what pass 1
// read last is in L2.
template <typename T, bool GROUP, bool ODD, bool SILU>
__global__ void __launch_bounds__(kWalkThreads + 32, 2)
k_gn_apply_staged(const T* x, const T* __restrict__ gamma, const T* __restrict__ beta, const float4* partial,
                  float* mean, float* inv, T* y, GnDims d) {
  constexpr int VW = dev::Vec16<T>::N;
  extern __shared__ __align__(128) unsigned char smem[];
  __shared__ __align__(8) StageBars bars;
  __shared__ JoinHere js;
  const WalkPlan& p = d.p;
  const Tile t(p);
  RowStream<T, 1, ODD> rows(&bars, smem, d, t);
  const int consumers = blockDim.x - 32;
  if (int(threadIdx.x) >= consumers) {  // (the inputs: before the join's end)
    const T* const base[1] = {x};
    if (int(threadIdx.x) == consumers) rows.produce(base, d, t, true, dev::policy_evict_first());
    return;
  }
  int c0 = first_channel(t.j, VW, 0, d.C);
  bool waited = false;
  int64_t joined = -1;
  for (Items it(d, true); it.more(); it.next()) {  // (every CTA has an item)
    const Range r = rows.range(p, it.item());
    const int off = ODD ? rows.sample(r.n).off : 0;
    const Ends ends = rows.ends(r, t);
    if constexpr (ODD) c0 = first_channel(t.j, VW, off, d.C);
    ApplyValues<T, GROUP ? 1 : VW, SILU> val;
    if (t.mine) val.load_params(c0, d, gamma, beta);
    if (!waited) {
      waited = true;
      dev::pdl_wait();
      dev::pdl_trigger();
    }
    if (d.here && joined != r.n) {
      joined = r.n;
      join_stats_here(partial, d, r.n, consumers, js);
    }
    if (d.here && r.ra == 0 && int(threadIdx.x) < d.G) {
      if (mean != nullptr) mean[r.n * d.G + threadIdx.x] = js.mean[threadIdx.x];
      if (inv != nullptr) inv[r.n * d.G + threadIdx.x] = js.inv[threadIdx.x];
    }
    if (t.mine) val.scale(c0, d.here ? 0 : r.n * d.G, d, d.here ? js.mean : mean, d.here ? js.inv : inv, PlainLoad{});
    const int64_t pitch = p.row_frags * VW;
    T* py = y + r.n * d.L - off + r.ra * pitch + t.j * VW;
    rows.consume(r, rows.mine(r, t), [&](int row, const auto& raw) {
#pragma unroll
      for (const auto& one : raw) {
        float v[VW];
        dev::Conv<T>::unpack(one[0], v);
        if (ODD && ends.has(row)) {
          const int64_t e0 = ends.e0 + row * ends.pitch;
          dev::load_frag<T, false>(x + r.n * d.L, e0, d.L, v);
          val(v);
          dev::store_frag<T, false>(y + r.n * d.L, e0, d.L, v);
        } else {
          val(v);
          dev::st16_stream(py + row * pitch, dev::Conv<T>::pack(v));
        }
        ++row;
      }
    });
  }
}

// Gradient, pass 1: per-channel sums of du and du * h of a CTA's items, and the
// groups' sums of each item.
//   gpart: [item][tile][slot] x (sum du gamma, sum du gamma h); cpart: leave_channel_sums
template <typename T, bool GROUP, bool ODD, bool SILU>
__global__ void __launch_bounds__(kWalkThreads + 32, 2)
k_gn_grad_sums_staged(const T* dy, const T* x, const T* __restrict__ gamma, const T* __restrict__ beta,
                      const float* mean, const float* inv, GnDims d, float* gpart, float* cpart) {
  constexpr int VW = dev::Vec16<T>::N;
  constexpr int EV = GROUP ? 1 : VW;
  extern __shared__ __align__(128) unsigned char smem[];
  __shared__ __align__(8) StageBars bars;
  // after the stages: the sums by position, and by channel over the CTA's items
  float* s_a = reinterpret_cast<float*>(smem + kStageSmem);
  float* s_b = s_a + kWalkThreads * VW;
  float* tot_a = s_b + kWalkThreads * VW;
  float* tot_b = tot_a + kWalkThreads * VW;
  float* t_a = ODD ? tot_b + kWalkThreads * VW : s_a;
  float* t_b = ODD ? t_a + kWalkThreads * VW : s_b;
  const WalkPlan& p = d.p;
  const Tile t(p);
  RowStream<T, 2, ODD> rows(&bars, smem, d, t);
  dev::pdl_wait();
  dev::pdl_trigger();
  const int consumers = blockDim.x - 32;
  if (int(threadIdx.x) >= consumers) {
    const T* const base[2] = {x, dy};
    if (int(threadIdx.x) == consumers) rows.produce(base, d, t, false, policy_evict_normal());
    return;
  }
  int c0 = first_channel(t.j, VW, 0, d.C);
  const Columns cols(d, t, VW, 1);
  bool once = true;
  for (Items it(d, false); it.more(); it.next()) {
    const Range r = rows.range(p, it.item());
    const int off = ODD ? rows.sample(r.n).off : 0;
    const Ends ends = rows.ends(r, t);
    if constexpr (ODD) c0 = first_channel(t.j, VW, off, d.C);
    GradValues<T, EV, SILU> val;
    if (t.mine) val.load(c0, r.n * d.G, d, gamma, beta, mean, inv);
    float sa[VW], sb[VW];
#pragma unroll
    for (int e = 0; e < VW; ++e) sa[e] = sb[e] = 0.f;
    rows.consume(r, rows.mine(r, t), [&](int row, const auto& raw) {
#pragma unroll
      for (const auto& one : raw) {
        float v[VW], w[VW];
        dev::Conv<T>::unpack(one[0], v);
        dev::Conv<T>::unpack(one[1], w);
        if (ODD && ends.has(row)) {  // 0 outside the sample: adds nothing
          const int64_t e0 = ends.e0 + row * ends.pitch;
          dev::load_frag<T, false>(x + r.n * d.L, e0, d.L, v);
          dev::load_frag<T, false>(dy + r.n * d.L, e0, d.L, w);
        }
        ++row;
        val(v, w);
        dev::add_pairs(sa, w);
        fma_pairs(w, v, sb);
      }
    });
    if (t.mine) {
      for_channels<VW>(c0, d.C, d.D, [&](int e, int, int g) { sb[e] *= inv[r.n * d.G + g]; });  // du t r = du h
      put(s_a, sa);
      put(s_b, sb);
    }
    consumer_sync();
    // by channel: to the totals, and times gamma to the first repeat's place, which only the
    // threads of that channel read (ODD: to memory of its own)
    sum_sets(consumers, cols.cols, cols.reps,
             [&](int i, int k, float& a, float& b) {
               const int pos = cols.at<ODD>(i, k, off);
               a += s_a[pos];
               b += s_b[pos];
             },
             [&](int i, float a, float b) {
               tot_a[i] = once ? a : tot_a[i] + a;
               tot_b[i] = once ? b : tot_b[i] + b;
               const float ga = dev::ld1_keep(gamma + cols.g0 * d.D + cols.in0 + i);
               t_a[i] = a * ga;
               t_b[i] = b * ga;
             });
    once = false;
    consumer_sync();
    float* out = gpart + (it.item() * p.tiles + t.tile) * d.slots * 2;
    sum_sets(consumers, cols.n_groups, cols.D,
             [&](int g, int k, float& a, float& b) {
               const int i = cols.lo(g) + k;
               if (i < cols.hi(g)) {
                 a += t_a[i];
                 b += t_b[i];
               }
             },
             [&](int g, float a, float b) {
               out[g * 2] = a;
               out[g * 2 + 1] = b;
             });
    consumer_sync();
  }
  if (cpart == nullptr) return;
  const int64_t cta_rows = gridDim.x / unsigned(p.tiles), cta_row = blockIdx.x / unsigned(p.tiles);
  float* oa = cpart + cta_row * d.C + cols.g0 * d.D + cols.in0;
  for (int i = threadIdx.x; i < cols.cols; i += consumers) {  // a thread's own or, after the barrier, any
    oa[i] = tot_a[i];
    oa[cta_rows * d.C + i] = tot_b[i];
  }
}

// Gradient, pass 2: dx, over the items in reverse.
template <typename T, bool GROUP, bool ODD, bool SILU>
__global__ void __launch_bounds__(kWalkThreads + 32, 2)
k_gn_grad_apply_staged(const T* dy, const T* x, const T* __restrict__ gamma, const T* __restrict__ beta,
                       const float* mean, const float* inv, const float* m1, const float* m2, T* dx, GnDims d) {
  constexpr int VW = dev::Vec16<T>::N;
  extern __shared__ __align__(128) unsigned char smem[];
  __shared__ __align__(8) StageBars bars;
  const WalkPlan& p = d.p;
  const Tile t(p);
  RowStream<T, 2, ODD> rows(&bars, smem, d, t);
  const int consumers = blockDim.x - 32;
  if (int(threadIdx.x) >= consumers) {  // (the inputs: before the join's end)
    const T* const base[2] = {x, dy};
    if (int(threadIdx.x) == consumers) rows.produce(base, d, t, true, dev::policy_evict_first());
    return;
  }
  int c0 = first_channel(t.j, VW, 0, d.C);
  bool waited = false;
  for (Items it(d, true); it.more(); it.next()) {  // (every CTA has an item)
    const Range r = rows.range(p, it.item());
    const int off = ODD ? rows.sample(r.n).off : 0;
    const Ends ends = rows.ends(r, t);
    if constexpr (ODD) c0 = first_channel(t.j, VW, off, d.C);
    GradApplyValues<T, GROUP ? 1 : VW, SILU> val;
    if (t.mine) val.load(c0, r.n * d.G, d, gamma, beta, mean, inv);
    if (!waited) {
      waited = true;
      dev::pdl_wait();
      dev::pdl_trigger();
    }
    if (t.mine) val.load_means(c0, r.n * d.G, d, inv, m1, m2);
    const int64_t pitch = p.row_frags * VW;
    T* po = dx + r.n * d.L - off + r.ra * pitch + t.j * VW;
    rows.consume(r, rows.mine(r, t), [&](int row, const auto& raw) {
#pragma unroll
      for (const auto& one : raw) {
        float v[VW], w[VW];
        dev::Conv<T>::unpack(one[0], v);
        dev::Conv<T>::unpack(one[1], w);
        if (ODD && ends.has(row)) {
          const int64_t e0 = ends.e0 + row * ends.pitch;
          dev::load_frag<T, false>(x + r.n * d.L, e0, d.L, v);
          dev::load_frag<T, false>(dy + r.n * d.L, e0, d.L, w);
          val.dx(v, w);
          dev::store_frag<T, false>(dx + r.n * d.L, e0, d.L, v);
        } else {
          val.dx(v, w);
          dev::st16_stream(po + row * pitch, dev::Conv<T>::pack(v));
        }
        ++row;
      }
    });
  }
}

// ---------------------------------------------------------------------------
// One position a sample (S = 1), D / VW a power of two up to 32: the norm over
// each token's groups.  A group's fragments are neighbouring lanes, so its sums
// are shuffles; the tensor is one walk over all the tokens (N = 1, S = tokens in
// `d`), in the staged rows above, and a thread's channels stay the same.  This
// form is for many tokens; k_gn_token (group_norm_fused.cu) takes few.
// ---------------------------------------------------------------------------

struct TokenSet {
  int lanes;       // of a group
  int tokens_a_row, token0;  // tokens of a walk row, this thread's among them
  int group;       // of the token
  __device__ __forceinline__ TokenSet(const GnDims& d, const Tile& t, int vw, int set) : lanes(set) {
    const unsigned frags = unsigned(d.C / vw);  // of a token
    tokens_a_row = static_cast<int>(unsigned(d.p.row_frags) / frags);
    token0 = static_cast<int>(unsigned(t.j) / frags);
    group = static_cast<int>(unsigned(t.j) - token0 * frags) / set;
  }
  // Sums over the set's lanes.  Every lane of the warp takes part (the shuffles
  // are whole warps': with a set's own mask the warp ran once for each set).
  template <int R>
  __device__ __forceinline__ void sum(float (&x)[R]) const {
    for (int o = lanes >> 1; o > 0; o >>= 1) {
      float y[R];
#pragma unroll
      for (int u = 0; u < R; ++u) y[u] = __shfl_xor_sync(0xffffffffu, x[u], o);
#pragma unroll
      for (int u = 0; u < R; ++u) x[u] += y[u];
    }
  }
};

template <typename T, bool SILU>
__global__ void __launch_bounds__(kWalkThreads + 32, 2)
k_gn_token_staged(const T* x, const T* __restrict__ gamma, const T* __restrict__ beta, T* y, float* mean_out,
                  float* inv_out, GnDims d, int set) {
  constexpr int VW = dev::Vec16<T>::N;
  extern __shared__ __align__(128) unsigned char smem[];
  __shared__ __align__(8) StageBars bars;
  const WalkPlan& p = d.p;
  const Tile t(p);
  RowStream<T, 1> rows(&bars, smem, d, t);
  dev::pdl_wait();
  dev::pdl_trigger();
  const int consumers = blockDim.x - 32;
  if (int(threadIdx.x) >= consumers) {
    const T* const base[1] = {x};
    if (int(threadIdx.x) == consumers) rows.produce(base, d, t, false, dev::policy_evict_first());
    return;
  }
  const TokenSet ts(d, t, VW, set);
  const float scale = 1.0f / float(d.D);
  const int lane = threadIdx.x & 31, lead = lane & ~(set - 1);
  float a[VW], b[VW];
#pragma unroll
  for (int e = 0; e < VW; ++e) a[e] = b[e] = 0.f;
  if (t.mine) {
    const int c0 = first_channel(t.j, VW, 0, d.C);
    load_param(gamma, c0, d.C, d.pvec, a);
    if (beta != nullptr) load_param(beta, c0, d.C, d.pvec, b);
  }
  for (Items it(d, false); it.more(); it.next()) {
    const Range r = rows.range(p, it.item());
    const int64_t pitch = p.row_frags * VW, gpitch = int64_t(ts.tokens_a_row) * d.G;
    const int mine = rows.mine(r, t);  // lanes without the last row go round with the others
    T* py = y + r.ra * pitch + t.j * VW;
    const int64_t g0 = (r.ra * ts.tokens_a_row + ts.token0) * d.G + ts.group;
    float* pm = mean_out != nullptr && lane == lead ? mean_out + g0 : nullptr;
    float* pi = inv_out != nullptr && lane == lead ? inv_out + g0 : nullptr;
    rows.template consume<2>(r, static_cast<int>(r.rb - r.ra), [&](int row, const auto& raw) {
      constexpr int R = sizeof(raw) / sizeof(raw[0]);
      // sums and sums of squares relative to a centre, the median of three of the
      // group's values; where that is more than 4 standard deviations off the mean of one
      // of the warp's groups (see far_off), again, with that group's mean as its centre
      float v[R][VW], c[R], s[2 * R], m[R], var[R];
#pragma unroll
      for (int u = 0; u < R; ++u) {
        dev::Conv<T>::unpack(raw[u][0], v[u]);
        c[u] = median3(__shfl_sync(0xffffffffu, v[u][0], lead), __shfl_sync(0xffffffffu, v[u][VW / 2], lead + set / 2),
                       __shfl_sync(0xffffffffu, v[u][VW - 1], lead + set - 1));
      }
      auto sums = [&] {
#pragma unroll
        for (int u = 0; u < R; ++u) {
          float2 p = make_float2(0.f, 0.f), q = p;
#pragma unroll
          for (int e = 0; e < VW; e += 2) {
            const float2 w = __fadd2_rn(make_float2(v[u][e], v[u][e + 1]), make_float2(-c[u], -c[u]));
            p = __fadd2_rn(p, w);
            q = __ffma2_rn(w, w, q);
          }
          s[2 * u] = p.x + p.y;
          s[2 * u + 1] = q.x + q.y;
        }
        ts.sum(s);
#pragma unroll
        for (int u = 0; u < R; ++u) {
          m[u] = s[2 * u] * scale;
          var[u] = not_negative(fmaf(s[2 * u + 1], scale, -m[u] * m[u]));
        }
      };
      sums();
      bool far = false;
#pragma unroll
      for (int u = 0; u < R; ++u) far |= m[u] * m[u] > 16.f * var[u];
      if (__any_sync(0xffffffffu, far)) {
#pragma unroll
        for (int u = 0; u < R; ++u)
          if (far_off(m[u] * m[u], var[u])) c[u] += m[u];
        sums();
      }
#pragma unroll
      for (int u = 0; u < R; ++u) {
        // (rsqrtf, within 2 ulp: the other forms divide and take a root)
        const float mu[1] = {c[u] + m[u]}, k = rsqrtf(var[u] + d.eps);
        float f[VW];
#pragma unroll
        for (int e = 0; e < VW; ++e) f[e] = a[e] * k;
        centre_scale_add(v[u], mu, f, b);
        if constexpr (SILU) activate<T>(v[u]);
        if (row + u < mine) {
          dev::st16_stream(py, dev::Conv<T>::pack(v[u]));
          if (pm != nullptr) *pm = mu[0];
          if (pi != nullptr) *pi = k;
        }
        py += pitch;
        if (pm != nullptr) pm += gpitch;
        if (pi != nullptr) pi += gpitch;
      }
    });
  }
}

// Its gradient.  The statistics of an item's tokens are fetched into shared memory
// first (the plan keeps an item that short): loaded row by row they cost 6 of 30
// us for bf16 8192 x 2048.  The parameters' sums run on in registers and leave as
// row blockIdx / tiles of cpart, 2 x [row][C].
template <typename T, bool SILU>
__global__ void __launch_bounds__(kWalkThreads + 32, 2)
k_gn_grad_token_staged(const T* dy, const T* x, const T* __restrict__ gamma, const T* __restrict__ beta,
                       const float* mean, const float* inv, T* dx, float* cpart, GnDims d, int set) {
  constexpr int VW = dev::Vec16<T>::N;
  extern __shared__ __align__(128) unsigned char smem[];
  __shared__ __align__(8) StageBars bars;
  // after the stages: an item's statistics, in the end the sums by position
  float* s_a = reinterpret_cast<float*>(smem + kStageSmem);
  float* s_b = s_a + kWalkThreads * VW;
  const WalkPlan& p = d.p;
  const Tile t(p);
  RowStream<T, 2> rows(&bars, smem, d, t);
  dev::pdl_wait();
  dev::pdl_trigger();
  const int consumers = blockDim.x - 32;
  if (int(threadIdx.x) >= consumers) {
    const T* const base[2] = {x, dy};
    if (int(threadIdx.x) == consumers) rows.produce(base, d, t, false, dev::policy_evict_first());
    return;
  }
  const TokenSet ts(d, t, VW, set);
  const float scale = 1.0f / float(d.D);
  float ga[VW], be[VW], tot_a[VW], tot_b[VW];
#pragma unroll
  for (int e = 0; e < VW; ++e) ga[e] = be[e] = tot_a[e] = tot_b[e] = 0.f;
  if (t.mine) {
    const int c0 = first_channel(t.j, VW, 0, d.C);
    load_param(gamma, c0, d.C, d.pvec, ga);
    if (SILU && beta != nullptr) load_param(beta, c0, d.C, d.pvec, be);
  }
  for (Items it(d, false); it.more(); it.next()) {
    const Range r = rows.range(p, it.item());
    const int64_t pitch = p.row_frags * VW;
    const int mine = rows.mine(r, t), all = static_cast<int>(r.rb - r.ra);
    T* po = dx + r.ra * pitch + t.j * VW;
    {
      // groups of the tile in a walk row (they are flat over a row's tokens), and of the tensor in all
      const int in_row = t.frags / set, count = all * in_row;
      const int64_t row_groups = int64_t(ts.tokens_a_row) * d.G, total = d.S * d.G;
      const int64_t g0 = r.ra * row_groups + t.tile * p.tile_frags / set;
      for (int i = threadIdx.x; i < count; i += consumers) {
        const int row = static_cast<int>(unsigned(i) / unsigned(in_row));
        const int64_t g = g0 + row * row_groups + (i - row * in_row);
        s_a[i] = g < total ? mean[g] : 0.f;
        s_b[i] = g < total ? inv[g] : 0.f;
      }
    }
    consumer_sync();
    const int in_row = t.frags / set, own_group = min(int(threadIdx.x) / set, in_row - 1);
    rows.stages(r, [&](int row, const unsigned char* src) {
      const int n = min(rows.rows, all - row);  // lanes without the last row go round too
      const int own = min(rows.rows, mine - row);
      const int warp_own = __reduce_min_sync(0xffffffffu, own);  // rows that all lanes have
      auto two = [&](int i) {
        uint4 raw[2][2];
        rows.load(src, i, raw);
        float h[2][VW], w[2][VW], s[4], kk[2];
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          dev::Conv<T>::unpack(raw[u][0], h[u]);
          dev::Conv<T>::unpack(raw[u][1], w[u]);
          if (i + u >= warp_own && i + u >= own) {
#pragma unroll
            for (int e = 0; e < VW; ++e) h[u][e] = w[u][e] = 0.f;
          }
          const int at = min(row + i + u, all - 1) * in_row + own_group;
          const float one_m[1] = {s_a[at]}, one_k[1] = {s_b[at]};
          kk[u] = one_k[0];
          centre_scale(h[u], one_m, one_k);
          if constexpr (SILU) {
            float a[VW];
#pragma unroll
            for (int e = 0; e < VW; ++e) a[e] = be[e];
            fma_pairs(h[u], ga, a);
            activate_grad<T>(w[u], a);
          }
          dev::add_pairs(tot_a, w[u]);
          fma_pairs(w[u], h[u], tot_b);
          float2 sa = make_float2(0.f, 0.f), sb = sa;
#pragma unroll
          for (int e = 0; e < VW; e += 2) {
            const float2 g = __fmul2_rn(make_float2(w[u][e], w[u][e + 1]), make_float2(ga[e], ga[e + 1]));
            sa = __fadd2_rn(sa, g);
            sb = __ffma2_rn(g, make_float2(h[u][e], h[u][e + 1]), sb);
            w[u][e] = g.x;
            w[u][e + 1] = g.y;
          }
          s[2 * u] = sa.x + sa.y;
          s[2 * u + 1] = sb.x + sb.y;
        }
        ts.sum(s);
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          // r (w - m1 - h m2) = w r + (h (-r m2) - r m1)
          const float p1 = -kk[u] * (s[2 * u] * scale), p2 = -kk[u] * (s[2 * u + 1] * scale);
#pragma unroll
          for (int e = 0; e < VW; e += 2) {
            const float2 q = __ffma2_rn(make_float2(h[u][e], h[u][e + 1]), make_float2(p2, p2), make_float2(p1, p1));
            const float2 z = __ffma2_rn(make_float2(w[u][e], w[u][e + 1]), make_float2(kk[u], kk[u]), q);
            w[u][e] = z.x;
            w[u][e + 1] = z.y;
          }
          if (i + u < own) dev::st16_stream(po + (row + i + u) * pitch, dev::Conv<T>::pack(w[u]));
        }
      };
      // (a second row beyond the last is read from within the block's memory, and not used)
      for (int i = 0; i < n; i += 2) two(i);
    });
    consumer_sync();
  }
  if (cpart == nullptr) return;
  if (t.mine) {
    put(s_a, tot_a);
    put(s_b, tot_b);
  }
  consumer_sync();
  const Columns cols(d, t, VW, 1);
  const int64_t cta_rows = gridDim.x / unsigned(p.tiles), cta_row = blockIdx.x / unsigned(p.tiles);
  float* oa = cpart + cta_row * d.C + int64_t(t.tile) * p.tile_frags * VW;
  sum_sets(consumers, cols.cols, cols.reps,
           [&](int i, int k, float& a, float& b) {
             a += s_a[i + k * cols.cols];
             b += s_b[i + k * cols.cols];
           },
           [&](int i, float a, float b) {
             oa[i] = a;
             oa[cta_rows * d.C + i] = b;
           });
}

// ---------------------------------------------------------------------------
// The same four passes for any C and alignment: fragments are checked against
// the sample's ends, and a sample may start off a 16-byte boundary (VEC: whole
// fragments are loaded as 16 bytes; else value by value).
// ---------------------------------------------------------------------------

// Blocks an SM of the general kernels' first passes, for the compiler (two, not three, of
// float32: f32 2x1000x1001 16.5 us, not 15.8, its gradient 22.3, not 19.1).
template <typename T> constexpr int kGeneralBlocks = sizeof(T) == 4 ? 3 : 2;

// Pass 1.  A thread takes its channels' values relative to their first in the item
// (`ref`), and sums their distances from a running mean `c` of those: after 4 rows,
// 8, 16 ... and then every kFoldRows the mean moves on by s / n, and the squares to it
// (q - s (s / n), at most half of q where no more rows are new than are old: nothing
// cancels, whatever the values).
constexpr int kFoldRows = 64;

template <typename T>
__global__ void __launch_bounds__(kWalkThreads, kGeneralBlocks<T>)
k_gn_stats(const T* x, GnDims d, float4* partial, float* mean_out, float* inv_out) {
  constexpr int VW = dev::Vec16<T>::N;
  constexpr int U = 4;
  __shared__ float s_cnt[kWalkThreads * VW], s_ref[kWalkThreads * VW], s_mean[kWalkThreads * VW],
      s_m2[kWalkThreads * VW];
  dev::pdl_wait();
  dev::pdl_trigger();
  const WalkPlan& p = d.p;
  const Tile t(p);
  for (Items it(d, false); it.more(); it.next()) {
    const Range r(p, it.item(), p.rows);
    const T* xs = x + r.n * d.L;
    const int off = walk_offset<T, true>(xs);
    if (t.mine) {
      float ref[VW], c[VW], m2[VW], s[VW], q[VW], cnt[VW];
#pragma unroll
      for (int e = 0; e < VW; ++e) ref[e] = c[e] = m2[e] = s[e] = q[e] = cnt[e] = 0.f;
      float whole = 0.f;  // rows since the last fold that count for every element
      auto fold = [&] {
#pragma unroll
        for (int e = 0; e < VW; ++e) {
          cnt[e] += whole;
          const float by = cnt[e] > 0.f ? s[e] / cnt[e] : 0.f;
          m2[e] += not_negative(q[e] - s[e] * by);
          c[e] += by;
          s[e] = q[e] = 0.f;
        }
        whole = 0.f;
      };
      int64_t folded = r.ra;
      int step = U;
      for (int64_t r0 = r.ra; r0 < r.rb; r0 += U) {
        float v[U][VW];
#pragma unroll
        for (int u = 0; u < U; ++u)
          if (r0 + u < r.rb) dev::load_frag<T, true>(xs, ((r0 + u) * p.row_frags + t.j) * VW - off, d.L, v[u]);
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const int64_t e0 = ((r0 + u) * p.row_frags + t.j) * VW - off;
          if (r0 > r.ra && r0 + u < r.rb && e0 >= 0 && e0 + VW <= d.L) {
#pragma unroll
            for (int e = 0; e < VW; ++e) {
              const float w = (v[u][e] - ref[e]) - c[e];
              s[e] += w;
              q[e] = fmaf(w, w, q[e]);
            }
            whole += 1.f;
            continue;
          }
#pragma unroll
          for (int e = 0; e < VW; ++e) {  // the item's first rows, and partial fragments
            if (r0 + u < r.rb && e0 + e >= 0 && e0 + e < d.L) {
              if (cnt[e] + whole == 0.f) ref[e] = v[u][e];
              const float w = (v[u][e] - ref[e]) - c[e];
              cnt[e] += 1.f;
              s[e] += w;
              q[e] = fmaf(w, w, q[e]);
            }
          }
        }
        if (r0 + U - folded >= step && r0 + U < r.rb) {
          step = folded == r.ra ? step : min(2 * step, kFoldRows);  // 4, 4, 8, 16 ...: no more than there were
          folded = r0 + U;
          fold();
        }
      }
      fold();
#pragma unroll
      for (int e = 0; e < VW; ++e) {
        s_cnt[threadIdx.x * VW + e] = cnt[e];
        s_ref[threadIdx.x * VW + e] = ref[e];
        s_mean[threadIdx.x * VW + e] = c[e];
        s_m2[threadIdx.x * VW + e] = m2[e];
      }
    }
    __syncthreads();
    join_statistics<T>(d, t, r, it.item(), off, blockDim.x / 32, s_cnt, s_ref, s_mean, s_m2, partial, mean_out,
                       inv_out);
    __syncthreads();
  }
}

template <typename T, bool VEC, bool SILU>
__global__ void __launch_bounds__(kWalkThreads)
k_gn_apply(const T* x, const T* __restrict__ gamma, const T* __restrict__ beta, const float* mean, const float* inv,
           T* y, GnDims d) {
  constexpr int VW = dev::Vec16<T>::N;
  constexpr int U = 4;
  dev::pdl_wait();
  dev::pdl_trigger();
  const WalkPlan& p = d.p;
  const Tile t(p);
  if (!t.mine) return;
  for (Items it(d, true); it.more(); it.next()) {
    const Range r(p, it.item(), p.rows);
    const T* xs = x + r.n * d.L;
    T* ys = y + r.n * d.L;
    const int off = walk_offset<T, VEC>(xs);
    ApplyValues<T, VW, SILU> val;
    const int c0 = first_channel(t.j, VW, off, d.C);
    val.load_params(c0, d, gamma, beta);
    val.scale(c0, r.n * d.G, d, mean, inv, CachedLoad{});
    for (int64_t r0 = r.ra; r0 < r.rb; r0 += U) {
      float v[U][VW];
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (r0 + u < r.rb) dev::load_frag<T, VEC>(xs, ((r0 + u) * p.row_frags + t.j) * VW - off, d.L, v[u]);
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (r0 + u < r.rb) {
          val(v[u]);
          dev::store_frag<T, VEC>(ys, ((r0 + u) * p.row_frags + t.j) * VW - off, d.L, v[u]);
        }
      }
    }
  }
}

// The sums over a thread's rows, of du (sa) and of du t (sb), to those of du and
// du h = r du t: for the parameters (added to tot) and, times gamma, for the groups.
template <typename T>
__device__ __forceinline__ void finish_sums(int c0, int64_t ng, const GnDims& d, const T* __restrict__ gamma,
                                            const float* inv, float (&sa)[dev::Vec16<T>::N],
                                            float (&sb)[dev::Vec16<T>::N], float* tot_a, float* tot_b, float* s_a,
                                            float* s_b, bool first) {
  constexpr int VW = dev::Vec16<T>::N;
  float ga[VW];
  for_channels<VW>(c0, d.C, d.D, [&](int e, int c, int g) {
    ga[e] = dev::ld1_keep(gamma + c);
    sb[e] *= inv[ng + g];
  });
#pragma unroll
  for (int e = 0; e < VW; e += 4) {  // a thread's own places
    float4* a = reinterpret_cast<float4*>(tot_a + threadIdx.x * VW + e);
    float4* b = reinterpret_cast<float4*>(tot_b + threadIdx.x * VW + e);
    const float4 pa = first ? make_float4(0.f, 0.f, 0.f, 0.f) : *a, pb = first ? make_float4(0.f, 0.f, 0.f, 0.f) : *b;
    *a = make_float4(pa.x + sa[e], pa.y + sa[e + 1], pa.z + sa[e + 2], pa.w + sa[e + 3]);
    *b = make_float4(pb.x + sb[e], pb.y + sb[e + 1], pb.z + sb[e + 2], pb.w + sb[e + 3]);
  }
#pragma unroll
  for (int e = 0; e < VW; ++e) {
    sa[e] *= ga[e];
    sb[e] *= ga[e];
  }
  put(s_a, sa);
  put(s_b, sb);
}

// A CTA's items share `off` (the launch sees to it), so a thread's channels stay
// the same and its sums run on over them.
template <typename T, bool VEC, bool SILU>
__global__ void __launch_bounds__(kWalkThreads, kGeneralBlocks<T>)
k_gn_grad_sums(const T* dy, const T* x, const T* __restrict__ gamma, const T* __restrict__ beta, const float* mean,
               const float* inv, GnDims d, float* gpart, float* cpart) {
  constexpr int VW = dev::Vec16<T>::N;
  constexpr int U = 2;
  __shared__ __align__(16) float s_a[kWalkThreads * VW], s_b[kWalkThreads * VW];
  extern __shared__ __align__(128) unsigned char smem[];
  float* tot_a = reinterpret_cast<float*>(smem);  // the totals over the CTA's items
  float* tot_b = tot_a + kWalkThreads * VW;
  dev::pdl_wait();
  dev::pdl_trigger();
  const WalkPlan& p = d.p;
  const Tile t(p);
  int off = 0;
  bool once = true;
  for (Items it(d, false); it.more(); it.next()) {
    const Range r(p, it.item(), p.rows);
    const T* xs = x + r.n * d.L;
    const T* ds = dy + r.n * d.L;
    off = walk_offset<T, VEC>(xs);
    if (t.mine) {
      const int c0 = first_channel(t.j, VW, off, d.C);
      GradValues<T, VW, SILU> val;
      val.load(c0, r.n * d.G, d, gamma, beta, mean, inv);
      float sa[VW], sb[VW];
#pragma unroll
      for (int e = 0; e < VW; ++e) sa[e] = sb[e] = 0.f;
      for (int64_t r0 = r.ra; r0 < r.rb; r0 += U) {
        float v[U][VW], w[U][VW];
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const int64_t e0 = ((r0 + u) * p.row_frags + t.j) * VW - off;
          if (r0 + u < r.rb) {
            dev::load_frag<T, VEC>(xs, e0, d.L, v[u]);
            dev::load_frag<T, VEC>(ds, e0, d.L, w[u]);  // 0 outside the sample: adds nothing
          }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
          if (r0 + u < r.rb) {
            val(v[u], w[u]);
            dev::add_pairs(sa, w[u]);
            fma_pairs(w[u], v[u], sb);
          }
        }
      }
      finish_sums<T>(c0, r.n * d.G, d, gamma, inv, sa, sb, tot_a, tot_b, s_a, s_b, once);
    }
    once = false;
    __syncthreads();
    join_group_sums<T>(d, t, it.item(), off, blockDim.x / 32, s_a, s_b, gpart);
    __syncthreads();
  }
  if (cpart != nullptr)
    leave_channel_sums<T>(d, t, off, int(blockDim.x), tot_a, tot_b, cpart, [] { __syncthreads(); });
}

template <typename T, bool VEC, bool SILU>
__global__ void __launch_bounds__(kWalkThreads)
k_gn_grad_apply(const T* dy, const T* x, const T* __restrict__ gamma, const T* __restrict__ beta, const float* mean,
                const float* inv, const float* m1, const float* m2, T* dx, GnDims d) {
  constexpr int VW = dev::Vec16<T>::N;
  constexpr int U = 2;
  dev::pdl_wait();
  dev::pdl_trigger();
  const WalkPlan& p = d.p;
  const Tile t(p);
  if (!t.mine) return;
  for (Items it(d, true); it.more(); it.next()) {
    const Range r(p, it.item(), p.rows);
    const T* xs = x + r.n * d.L;
    const T* ds = dy + r.n * d.L;
    T* os = dx + r.n * d.L;
    const int off = walk_offset<T, VEC>(xs);
    const int c0 = first_channel(t.j, VW, off, d.C);
    GradApplyValues<T, VW, SILU> val;
    val.load(c0, r.n * d.G, d, gamma, beta, mean, inv);
    val.load_means(c0, r.n * d.G, d, inv, m1, m2);
    for (int64_t r0 = r.ra; r0 < r.rb; r0 += U) {
      float v[U][VW], w[U][VW];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int64_t e0 = ((r0 + u) * p.row_frags + t.j) * VW - off;
        if (r0 + u < r.rb) {
          dev::load_frag<T, VEC>(xs, e0, d.L, v[u]);
          dev::load_frag<T, VEC>(ds, e0, d.L, w[u]);
        }
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (r0 + u < r.rb) {
          val.dx(v[u], w[u]);
          dev::store_frag<T, VEC>(os, ((r0 + u) * p.row_frags + t.j) * VW - off, d.L, v[u]);
        }
      }
    }
  }
}

// ---------------------------------------------------------------------------
// Joining a group's chunks and tiles: a warp takes one (n, g); bound by the latency
// of a few reads.
//
// The joins let pass 2 launch before they wait for pass 1: pass 1 has seen the
// call's predecessors end before a join starts, so the inputs are there for pass
// 2's producers, which fill their stages while pass 1 runs out.  Its consumers
// wait for the join's results (and through them for pass 1).
// ---------------------------------------------------------------------------

constexpr int kJoinThreads = 64;

// (count, centre, mean - centre, M2) of the parts -> the group's statistics, the means
// relative to that of the first lane whose first part is not empty (tiles of a walk row
// can lack the group; if all do, to the group's first value).  `lanes` of a warp (a power
// of two) take one (n, g), each keeping up to KEPT parts in registers for the second
// sum and reading others again; KEPT 1 where a warp's lanes hold all parts of a group (a
// warp for each group: f16 40x100x16384 in 4096 groups 271 us in all, 97 so).
constexpr int kJoinKept = 10;

template <typename T, int WAY, int KEPT>
__global__ void __launch_bounds__(kJoinThreads)
k_gn_join(const T* x, const float4* partial, GnDims d, float* mean_out, float* inv_out, int log_lanes) {
  dev::pdl_trigger();
  bool waited = false;  // where the first group's parts lie, and x: before pass 1 ends
  const int lanes = KEPT == 1 ? 1 << log_lanes : 32, lane = threadIdx.x & (lanes - 1);
  const int64_t of_sample = int64_t(d.p.chunks) * d.p.tiles * d.slots, all = d.N * d.G;
  auto sum = [&](float v) {
    for (int o = lanes >> 1; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
  };
  // (a warp's lanes go round together: lanes beyond the last group take part in its shuffles)
  const int per_warp = 32 / lanes, in_warp = (threadIdx.x & 31) / lanes;
  for (int64_t i0 = (int64_t(blockIdx.x) * (kJoinThreads / 32) + (threadIdx.x >> 5)) * per_warp; i0 < all;
       i0 += int64_t(gridDim.x) * (kJoinThreads / 32) * per_warp) {
    const int64_t i = i0 + in_warp;
    const bool live = KEPT > 1 || i < all;
    const int64_t n = live ? quotient(i, d.G) : 0;
    const int g = live ? static_cast<int>(i - n * d.G) : 0;
    const T* xs = x + n * d.L;
    const float4* src = partial + n * of_sample;
    const float first = dev::ld1_keep(xs + int64_t(g) * d.D);
    auto join = [&](const auto& parts) {
      if (!waited) dev::pdl_wait();
      waited = true;
      auto part = [&](unsigned k) { return live ? parts.load(src, k) : float4{}; };
      float4 kept[KEPT];
#pragma unroll
      for (int u = 0; u < KEPT; ++u) kept[u] = part(lane + u * 32);
      const int lead = (threadIdx.x & 31) - lane;
      const unsigned filled = __ballot_sync(0xffffffffu, kept[0].x > 0.f) >> lead & (0xffffffffu >> (32 - lanes));
      const float mean0 = __shfl_sync(0xffffffffu, kept[0].y + kept[0].z, lead + max(0, __ffs(filled) - 1));
      const float ref = filled != 0 ? mean0 : first;
      float c = 0.f, s = 0.f, q = 0.f, res = 0.f;
      auto add = [&](float4& v) {
        v.y = (v.y - ref) + v.z;
        c += v.x;
        s = fmaf(v.x, v.y, s);
      };
#pragma unroll
      for (int u = 0; u < KEPT; ++u) add(kept[u]);
      if constexpr (KEPT > 1) {
        for (unsigned k = lane + KEPT * 32; k < parts.count; k += 32) {
          float4 v = part(k);
          add(v);
        }
      }
      c = sum(c);
      const float mg = sum(s) / c;
      auto square = [&](const float4& v) {
        const float w = v.y - mg;
        res = fmaf(v.x, w, res);
        q += fmaf(v.x * w, w, v.w);
      };
#pragma unroll
      for (int u = 0; u < KEPT; ++u) square(kept[u]);
      if constexpr (KEPT > 1) {
        for (unsigned k = lane + KEPT * 32; k < parts.count; k += 32) {
          float4 v = part(k);
          v.y = (v.y - ref) + v.z;
          square(v);
        }
      }
      res = sum(res);
      q = sum(q);
      if (live && lane == 0) {
        const float fix = res / c;  // what rounding left out of the mean
        mean_out[i] = ref + (mg + fix);
        inv_out[i] = 1.0f / sqrtf(not_negative(q - res * fix) / c + d.eps);
      }
    };
    with_parts<T, WAY>(d, g, xs, join);
  }
}

// The gradient's sums of the parts -> m1, m2 of each (n, g), 2^log_lanes lanes to one;
// and, in the blocks after the first `join_blocks`, the channels' sums -> dbeta, dgamma.
template <typename T, int WAY>
__global__ void __launch_bounds__(kSumsThreads)
k_gn_grad_join(const T* x, const float* gpart, GnDims d, float* m1, float* m2, int join_blocks, const float* cpart, int64_t rows,
               int64_t reps, T* dbeta, T* dgamma, int log_lanes) {
  dev::pdl_trigger();
  dev::pdl_wait();
  if (int(blockIdx.x) >= join_blocks) {
    channel_sums<T>(cpart, rows, reps, d.C, 2, dbeta, dgamma, blockIdx.x - join_blocks, gridDim.x - join_blocks);
    return;
  }
  const int lanes = WAY == 1 ? 1 << log_lanes : 32, lane = threadIdx.x & (lanes - 1);
  const int per_warp = 32 / lanes, in_warp = (threadIdx.x & 31) / lanes;
  const int64_t of_sample = int64_t(d.p.chunks) * d.p.tiles * d.slots, all = d.N * d.G;
  const float scale = 1.0f / (float(d.S) * float(d.D));
  // (a warp's lanes go round together, as in k_gn_join)
  for (int64_t i0 = (int64_t(threadIdx.x / 32) * join_blocks + blockIdx.x) * per_warp; i0 < all;
       i0 += int64_t(join_blocks) * (kSumsThreads / 32) * per_warp) {
    const int64_t i = i0 + in_warp;
    const bool live = WAY != 1 || i < all;
    float a = 0.f, b = 0.f;
    if (live) {
      const int64_t n = quotient(i, d.G);
      const float2* src = reinterpret_cast<const float2*>(gpart) + n * of_sample;
      with_parts<T, WAY>(d, static_cast<int>(i - n * d.G), x + n * d.L, [&](const auto& parts) {
#pragma unroll 8
        for (unsigned k = lane; k < parts.count; k += lanes) {
          const float2 v = parts.load(src, k);
          a += v.x;
          b += v.y;
        }
      });
    }
    for (int o = lanes >> 1; o > 0; o >>= 1) {
      a += __shfl_xor_sync(0xffffffffu, a, o);
      b += __shfl_xor_sync(0xffffffffu, b, o);
    }
    if (live && lane == 0) {
      m1[i] = a * scale;
      m2[i] = b * scale;
    }
  }
}

// CTAs an SM that the general kernels' plan is made for (us, 2, 8 and 16 of them: f16
// 2x16070x1044 176, 127 and 146, its gradient 263, 217 and 236).
constexpr int kGeneralCtas = 8;

int64_t vec_width(DType t) { return t == DType::F32 ? 4 : 8; }

// The most groups of D channels that a tile's run of channels can meet.
int slots_of(const WalkPlan& p, int64_t vw, int64_t G, int64_t D) {
  return p.tiles == 1 ? int(G) : int(std::min(G, (p.tile_frags * vw + D - 2) / D + 1));
}

// `periods`: walk rows are whole periods of the channels, as the gradient's channel
// sums want them; else a sample shorter than a period is a walk row by itself.
GnDims dims_of(DType t, int64_t N, int64_t S, int64_t C, int64_t G, float eps, bool periods) {
  GnDims d{N, S, S * C, int(C), int(G), int(C / G), eps, 0, 0, 0, false, false, 0, false, false, 0, {}};
  d.p = make_walk(d.L, C, int(vec_width(t)), N, kPlanSms * 2, 4);
  d.ctas = kPlanSms * 2;
  if (d.p.tiles > 1 && C % vec_width(t) != 0) {  // the general kernels: no stages, so more blocks an SM
    d.ctas = kPlanSms * kGeneralCtas;
    d.p = make_walk(d.L, C, int(vec_width(t)), N, d.ctas, 4);
    const int64_t all = (d.L + 2 * (vec_width(t) - 1)) / vec_width(t);
    if (!periods && all < d.p.row_frags && all > kWalkThreads) {
      // (f16 5000x1x5001 in these kernels: 3267 us to 499)
      d.p.row_frags = all;
      d.p.tiles = int((all + kWalkThreads - 1) / kWalkThreads);
      d.p.tile_frags = int((all + d.p.tiles - 1) / d.p.tiles);
      d.p.threads = (d.p.tile_frags + 31) / 32 * 32;
      d.p.rows = d.p.rows_per_chunk = 1;
      d.p.chunks = 1;
    }
  }
  d.slots = slots_of(d.p, vec_width(t), G, d.D);
  d.frags = d.L / vec_width(t);
  d.full_rows = d.frags / d.p.row_frags;
  d.rest = int(d.frags % d.p.row_frags);
  return d;
}

// Parts of a group at most (staged rows), and the lanes that join them: a power of two.
int64_t most_parts(const GnDims& d, int64_t vw) {
  const int64_t tile = d.p.tile_frags * vw;
  return d.p.chunks * std::min<int64_t>(d.p.tiles, (d.D + tile - 2) / tile + 1);
}
int log_lanes_of(const GnDims& d, int64_t vw) {
  int log = 0;
  while (log < 5 && (1 << log) < most_parts(d, vw)) ++log;
  return log;
}

// CTA rows (of `tiles` CTAs) of a launch over N * chunks items.
int64_t cta_rows_of(const GnDims& d) {
  return std::max<int64_t>(1, std::min(d.N * d.p.chunks, d.ctas / d.p.tiles));
}

// Pass 2 joins the parts itself where a block reads them fast: 1024 of them, not
// more than 128 chunks.  With the join in pass 2 and as a launch of its own, us: f16
// 3x1331x189 (909 parts) 10.6 and 11.4, bf16 32x4096x320 (320) 45.8 and 47.5; but
// f16 8x1024x640 (1216) 13.3 and 12.6, 2x4096x320 (4864) 14.6 and 10.9, and one
// group in 304 chunks 12.2 and 11.6.  (The gradient, whose join adds up the channels
// too, lost by it: f16 8x1024x640 22.6 and 20.0.)
bool join_in_pass2(const GnDims& d) {
  return d.p.tiles == 1 && d.G <= d.p.threads && d.p.chunks <= 128 && int64_t(d.p.chunks) * d.G <= 1024;
}

bool split_parts(const GnDims& d) { return d.p.chunks > 1 || d.p.tiles > 1; }
int64_t grad_rows(const GnDims& d) { return cta_rows_of(d); }

// Offset in bytes of the next array in a workspace: each starts on 16 bytes.
size_t pad16(size_t b) { return (b + 15) / 16 * 16; }

struct GnWorkspace {
  size_t partial, mean, inv, total;
};
GnWorkspace gn_workspace(const GnDims& d) {
  GnWorkspace w;
  const size_t stats = pad16(size_t(d.N) * d.G * 4);
  w.partial = 0;
  w.mean = size_t(d.N) * d.p.chunks * d.p.tiles * d.slots * 16;
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
  w.m1 = pad16(size_t(d.N) * d.p.chunks * d.p.tiles * d.slots * 8);
  w.m2 = w.m1 + stats;
  w.cpart = w.m2 + stats;
  w.total = w.cpart + size_t(grad_rows(d)) * width * 8;
  return w;
}

inline unsigned misalign16(const void* p) { return unsigned(reinterpret_cast<uintptr_t>(p) & 15u); }

// Staged kernels: CTAs of consumers and a producer warp, two an SM.
template <typename... KArgs, typename... Args>
cudaError_t launch_staged(void (*fn)(KArgs...), int64_t rows, const GnDims& d, cudaStream_t stream, int* launches,
                          size_t extra, Args... args) {
  cudaError_t e = allow_smem(reinterpret_cast<const void*>(fn));
  if (e != cudaSuccess) return e;
  e = launch(fn, dim3(unsigned(rows * d.p.tiles)), dim3(d.p.threads + 32), kStageSmem + extra, stream, args...);
  if (e == cudaSuccess) *launches += 1;
  return e;
}
template <typename... KArgs, typename... Args>
cudaError_t launch_plain(void (*fn)(KArgs...), int64_t rows, const GnDims& d, cudaStream_t stream, int* launches,
                         size_t extra, Args... args) {
  const cudaError_t e = launch(fn, dim3(unsigned(rows * d.p.tiles)), dim3(d.p.threads), extra, stream, args...);
  if (e == cudaSuccess) *launches += 1;
  return e;
}

template <typename T>
cudaError_t group_norm_t(const GroupNormArgs& a, cudaStream_t stream, int* launches) {
  constexpr int VW = dev::Vec16<T>::N;
  GnDims d = dims_of(a.t, a.N, a.S, a.C, a.G, a.eps, false);
  d.pvec = a.C % VW == 0 && misalign16(a.x) == 0 && misalign16(a.gamma) == 0 && misalign16(a.beta) == 0;
  const GnWorkspace w = gn_workspace(d);
  char* ws = static_cast<char*>(a.workspace);
  float* mean = a.mean != nullptr ? a.mean : reinterpret_cast<float*>(ws + w.mean);
  float* inv = a.inv != nullptr ? a.inv : reinterpret_cast<float*>(ws + w.inv);
  // (the general statistics of a single part are final at once)
  const bool odd = a.C % VW != 0, group = !odd && d.D % VW == 0;
  const bool staged = misalign16(a.x) == 0 && (!odd || d.p.tiles == 1);
  float4* partial = staged || split_parts(d) ? reinterpret_cast<float4*>(ws + w.partial) : nullptr;
  const T* x = static_cast<const T*>(a.x);
  const T* gamma = static_cast<const T*>(a.gamma);
  const T* beta = static_cast<const T*>(a.beta);
  T* y = static_cast<T*>(a.y);
  const int64_t rows = cta_rows_of(d);
  // the staged passes want whole fragments; the statistics need no alignment of y
  const bool vec = misalign16(x) == misalign16(y);
  d.here = staged && vec && join_in_pass2(d);
  d.staged = staged;
  d.shifted = !staged;
  cudaError_t e;
  if (staged) {
    auto f = group ? k_gn_stats_staged<T, true, false>
             : odd ? k_gn_stats_staged<T, false, true>
                   : k_gn_stats_staged<T, false, false>;
    // two sums by position and the groups' centres (and two sums by column)
    const size_t extra = sizeof(float) * kWalkThreads * (odd ? 5 : 3) * (group ? 1 : VW);
    e = launch_staged(f, rows, d, stream, launches, extra, x, d, partial);
  } else {
    e = launch_plain(k_gn_stats<T>, rows, d, stream, launches, 0, x, d, partial, mean, inv);
  }
  if (e != cudaSuccess) return e;
  if (partial != nullptr && !d.here) {
    const int way = way_of(d);
    const bool many = way != 1 || most_parts(d, VW) > 32;
    const int log_lanes = many ? 5 : log_lanes_of(d, VW);
    auto f = way == 0   ? k_gn_join<T, 0, kJoinKept>
             : way == 2 ? k_gn_join<T, 2, kJoinKept>
             : many     ? k_gn_join<T, 1, 4>
                        : k_gn_join<T, 1, 1>;
    const int64_t groups = kJoinThreads >> log_lanes;  // of a block
    const int64_t joins = std::min<int64_t>((d.N * d.G + groups - 1) / groups, kPlanSms * 8);
    e = launch(f, dim3(unsigned(joins)), dim3(kJoinThreads), 0, stream, x, partial, d, mean, inv, log_lanes);
    if (e != cudaSuccess) return e;
    *launches += 1;
  }
  if (staged && vec) {
    auto pick = [&](auto silu) {
      constexpr bool kSilu = decltype(silu)::value;
      return group ? k_gn_apply_staged<T, true, false, kSilu>
             : odd ? k_gn_apply_staged<T, false, true, kSilu>
                   : k_gn_apply_staged<T, false, false, kSilu>;
    };
    auto f = a.silu ? pick(std::true_type{}) : pick(std::false_type{});
    return launch_staged(f, rows, d, stream, launches, 0, x, gamma, beta, partial, d.here ? a.mean : mean,
                         d.here ? a.inv : inv, y, d);
  }
  auto f = vec ? (a.silu ? k_gn_apply<T, true, true> : k_gn_apply<T, true, false>)
               : (a.silu ? k_gn_apply<T, false, true> : k_gn_apply<T, false, false>);
  return launch_plain(f, rows, d, stream, launches, 0, x, gamma, beta, mean, inv, y, d);
}

template <typename T>
cudaError_t group_norm_grad_t(const GroupNormGradArgs& a, cudaStream_t stream, int* launches) {
  constexpr int VW = dev::Vec16<T>::N;
  // shared memory of the sums: by position and by channel (staged), or the totals (general)
  constexpr size_t kStagedSums = size_t(kWalkThreads) * VW * 16, kTotals = size_t(kWalkThreads) * VW * 8;
  GnDims d = dims_of(a.t, a.N, a.S, a.C, a.G, 0.f, true);
  d.pvec = a.C % VW == 0 && misalign16(a.x) == 0 && misalign16(a.gamma) == 0 && misalign16(a.beta) == 0;
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
  const bool same = misalign16(x) == misalign16(dy);
  const bool odd = a.C % VW != 0, group = !odd && d.D % VW == 0;
  const bool staged = misalign16(x) == 0 && same && (!odd || d.p.tiles == 1);
  const bool vec1 = same && (d.L % VW == 0 || rows >= d.N * d.p.chunks);
  const bool vec2 = same && misalign16(x) == misalign16(dx);
  d.staged = staged;
  d.shifted = !staged && vec1;
  cudaError_t e;
  if (staged) {
    auto pick = [&](auto silu) {
      constexpr bool kSilu = decltype(silu)::value;
      return group ? k_gn_grad_sums_staged<T, true, false, kSilu>
             : odd ? k_gn_grad_sums_staged<T, false, true, kSilu>
                   : k_gn_grad_sums_staged<T, false, false, kSilu>;
    };
    auto f = a.silu ? pick(std::true_type{}) : pick(std::false_type{});
    e = launch_staged(f, rows, d, stream, launches, odd ? kStagedSums / 2 * 3 : kStagedSums, dy, x, gamma, beta, a.mean, a.inv, d, gpart, cpart);
  } else {
    auto f = vec1 ? (a.silu ? k_gn_grad_sums<T, true, true> : k_gn_grad_sums<T, true, false>)
                  : (a.silu ? k_gn_grad_sums<T, false, true> : k_gn_grad_sums<T, false, false>);
    e = launch_plain(f, rows, d, stream, launches, kTotals, dy, x, gamma, beta, a.mean, a.inv, d, gpart, cpart);
  }
  if (e != cudaSuccess) return e;
  // joining the groups' parts and adding up the channels in one launch
  const int way = way_of(d), log_lanes = way == 1 ? log_lanes_of(d, VW) : 5;
  const int64_t groups = int64_t(8) << (5 - log_lanes);  // of a block, where there are few
  const int64_t joins = std::min<int64_t>((d.N * d.G + groups - 1) / groups, kPlanSms);
  const int64_t sums = cpart != nullptr ? std::min<int64_t>((int64_t(d.C) + 31) / 32 * 2, kPlanSms * 4) : 0;
  // (the sums of du are dbeta, those of du * h are dgamma)
  auto join = way == 0 ? k_gn_grad_join<T, 0> : way == 1 ? k_gn_grad_join<T, 1> : k_gn_grad_join<T, 2>;
  e = launch(join, dim3(unsigned(joins + sums)), dim3(kSumsThreads), 0, stream, x, gpart, d, m1, m2, int(joins), cpart,
             rows, d.p.tiles > 1 && !staged ? d.p.reps : int64_t(1), static_cast<T*>(a.dbeta), static_cast<T*>(a.dgamma), log_lanes);
  if (e != cudaSuccess) return e;
  *launches += 1;
  if (staged && vec2) {
    auto pick = [&](auto silu) {
      constexpr bool kSilu = decltype(silu)::value;
      return group ? k_gn_grad_apply_staged<T, true, false, kSilu>
             : odd ? k_gn_grad_apply_staged<T, false, true, kSilu>
                   : k_gn_grad_apply_staged<T, false, false, kSilu>;
    };
    auto f = a.silu ? pick(std::true_type{}) : pick(std::false_type{});
    return launch_staged(f, rows, d, stream, launches, 0, dy, x, gamma, beta, a.mean, a.inv, m1, m2, dx, d);
  }
  auto f = vec2 ? (a.silu ? k_gn_grad_apply<T, true, true> : k_gn_grad_apply<T, true, false>)
                : (a.silu ? k_gn_grad_apply<T, false, true> : k_gn_grad_apply<T, false, false>);
  return launch_plain(f, rows, d, stream, launches, 0, dy, x, gamma, beta, a.mean, a.inv, m1, m2, dx, d);
}

// The token form: the tensor as one sample of N positions, tiles of whole groups.
GnDims token_dims(DType t, int64_t N, int64_t C, int64_t G, float eps) {
  GnDims d = dims_of(t, 1, N, C, G, eps, true);
  const int set = int(d.D / vec_width(t));
  d.p = make_walk(d.L, C, int(vec_width(t)), 1, kPlanSms * 2, 4);
  d.p.tile_frags = (d.p.tile_frags + set - 1) / set * set;
  d.p.threads = (d.p.tile_frags + 31) / 32 * 32;
  return d;
}
int64_t token_rows(const GnDims& d) { return cta_rows_of(d); }

// The gradient's items are short enough for their statistics to fit shared memory
// (a float each for kWalkThreads * vw groups).
GnDims token_grad_dims(DType t, int64_t N, int64_t C, int64_t G) {
  GnDims d = token_dims(t, N, C, G, 0.f);
  const int64_t in_row = d.p.tile_frags / (d.D / vec_width(t));
  d.p.rows_per_chunk = std::min<int64_t>(d.p.rows_per_chunk, kWalkThreads * vec_width(t) / in_row);
  d.p.chunks = int((d.p.rows + d.p.rows_per_chunk - 1) / d.p.rows_per_chunk);
  return d;
}

// The staged token form from this many bytes of x on; below, the direct form's
// shorter start wins.  Staged and direct, us, at 0.5, 1 and 2 MB:
//   bf16 C = 256   3.4 3.3, 3.4 3.8, 3.5 5.8   gradient  6.2 5.7, 6.5 6.5, 7.0 9.1
//   bf16 C = 4096  3.5 3.5, 3.5 4.0, 3.6 6.1             8.8 7.5, 9.7 8.0, 10.2 12.8
//   f32  C = 256   3.0 3.1, 3.0 3.4, 3.1 6.2             5.6 4.8, 5.8 5.9, 6.3 7.6
//   f32  C = 4096  3.3 3.3, 3.3 3.6, 3.3 6.6             6.9 7.6, 9.1 7.8, 9.3 8.3
// (f32's wide gradients are the same either way up to 4 MB: 9.9 and 9.4.)
constexpr int64_t kTokenStagedBytes = int64_t(1) << 20;
constexpr int64_t kTokenGradStagedBytes = int64_t(2) << 20;

bool token_staged(DType t, int64_t N, int64_t S, int64_t C, int64_t G, int64_t from) {
  const int64_t vw = vec_width(t), D = C / G;
  return S == 1 && D % vw == 0 && D / vw <= 32 && (D / vw & (D / vw - 1)) == 0 &&
         N * C * (t == DType::F32 ? 4 : 2) >= from;
}

template <typename T>
cudaError_t token_fwd_t(const GroupNormArgs& a, cudaStream_t stream, int* launches) {
  GnDims d = token_dims(a.t, a.N, a.C, a.G, a.eps);
  d.pvec = misalign16(a.gamma) == 0 && misalign16(a.beta) == 0;
  auto f = a.silu ? k_gn_token_staged<T, true> : k_gn_token_staged<T, false>;
  return launch_staged(f, token_rows(d), d, stream, launches, 0, static_cast<const T*>(a.x),
                       static_cast<const T*>(a.gamma), static_cast<const T*>(a.beta), static_cast<T*>(a.y), a.mean,
                       a.inv, d, int(d.D / dev::Vec16<T>::N));
}

template <typename T>
cudaError_t token_grad_t(const GroupNormGradArgs& a, cudaStream_t stream, int* launches) {
  constexpr int VW = dev::Vec16<T>::N;
  GnDims d = token_grad_dims(a.t, a.N, a.C, a.G);
  d.pvec = misalign16(a.gamma) == 0 && misalign16(a.beta) == 0;
  const int64_t rows = token_rows(d);
  float* cpart = a.dgamma != nullptr || a.dbeta != nullptr ? static_cast<float*>(a.workspace) : nullptr;
  auto f = a.silu ? k_gn_grad_token_staged<T, true> : k_gn_grad_token_staged<T, false>;
  cudaError_t e = launch_staged(f, rows, d, stream, launches, size_t(kWalkThreads) * VW * 8,
                                static_cast<const T*>(a.dy), static_cast<const T*>(a.x),
                                static_cast<const T*>(a.gamma), static_cast<const T*>(a.beta), a.mean, a.inv,
                                static_cast<T*>(a.dx), cpart, d, int(d.D / VW));
  if (e != cudaSuccess || cpart == nullptr) return e;
  e = launch(k_channel_sums<T>, dim3(unsigned((int64_t(d.C) + 31) / 32 * 2)), dim3(kSumsThreads), 0, stream, cpart,
             rows, int64_t(1), int64_t(d.C), 2, static_cast<T*>(a.dbeta), static_cast<T*>(a.dgamma));
  if (e == cudaSuccess) *launches += 1;
  return e;
}

}  // namespace

size_t group_norm_workspace_bytes(DType t, int64_t N, int64_t S, int64_t C, int64_t G, bool aligned) {
  if (aligned && (token_staged(t, N, S, C, G, kTokenStagedBytes) || group_norm_fused_applies(t, N, S, C, G))) return 0;
  return gn_workspace(dims_of(t, N, S, C, G, 0.f, false)).total;
}

size_t group_norm_grad_workspace_bytes(DType t, int64_t N, int64_t S, int64_t C, int64_t G, bool aligned) {
  const bool token = token_staged(t, N, S, C, G, kTokenGradStagedBytes);
  const size_t of_token = token ? size_t(token_rows(token_grad_dims(t, N, C, G))) * size_t(C) * 8 : 0;
  if (aligned && token) return of_token;
  bool fused = false;
  const size_t of_fused = group_norm_grad_fused_bytes(t, N, S, C, G, aligned, &fused);
  if (aligned && fused) return of_fused;
  return std::max({of_token, of_fused, gn_grad_workspace(dims_of(t, N, S, C, G, 0.f, true), t).total});
}

cudaError_t launch_group_norm(const GroupNormArgs& a, cudaStream_t stream, int* launches) {
  if (token_staged(a.t, a.N, a.S, a.C, a.G, kTokenStagedBytes) && misalign16(a.x) == 0 && misalign16(a.y) == 0) {
    switch (a.t) {
      case DType::F32: return token_fwd_t<float>(a, stream, launches);
      case DType::F16: return token_fwd_t<__half>(a, stream, launches);
      default: return token_fwd_t<__nv_bfloat16>(a, stream, launches);
    }
  }
  bool done = false;
  const cudaError_t e = launch_group_norm_fused(a, stream, launches, &done);
  if (done || e != cudaSuccess) return e;
  switch (a.t) {
    case DType::F32: return group_norm_t<float>(a, stream, launches);
    case DType::F16: return group_norm_t<__half>(a, stream, launches);
    default: return group_norm_t<__nv_bfloat16>(a, stream, launches);
  }
}

cudaError_t launch_group_norm_grad(const GroupNormGradArgs& a, cudaStream_t stream, int* launches) {
  if (token_staged(a.t, a.N, a.S, a.C, a.G, kTokenGradStagedBytes) && misalign16(a.x) == 0 &&
      misalign16(a.dy) == 0 && misalign16(a.dx) == 0) {
    switch (a.t) {
      case DType::F32: return token_grad_t<float>(a, stream, launches);
      case DType::F16: return token_grad_t<__half>(a, stream, launches);
      default: return token_grad_t<__nv_bfloat16>(a, stream, launches);
    }
  }
  bool done = false;
  const cudaError_t e = launch_group_norm_grad_fused(a, stream, launches, &done);
  if (done || e != cudaSuccess) return e;
  switch (a.t) {
    case DType::F32: return group_norm_grad_t<float>(a, stream, launches);
    case DType::F16: return group_norm_grad_t<__half>(a, stream, launches);
    default: return group_norm_grad_t<__nv_bfloat16>(a, stream, launches);
  }
}

cudaError_t group_norm_pipe_timeouts(unsigned int* count, bool clear) { return read_pipe_timeouts(count, clear); }

}  // namespace ep

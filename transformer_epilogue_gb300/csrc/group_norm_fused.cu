// GroupNorm and its gradient for small samples: a sample is held by one block,
// in registers, x (and dy) are read once and the result is written from there.  One
// launch for the forward pass, no scratch.  The definitions stand in group_norm.cu.
//
// A block holds walk rows of `cf` fragments, one thread to a fragment column, so
// a thread's channels stay the same:
//   MODE 0  C % VW == 0 and D % VW == 0: a walk row is a position's C channels, and
//           a fragment lies in one group;
//   MODE 1  C % VW == 0, any D: the same rows, sums for each channel;
//   MODE 2  any C and alignment: a walk row is the C / gcd(C, VW) fragments after
//           which channels repeat (column_walk.cuh), or the sample where that has
//           fewer; the first and the last fragment of a sample may be partial.
// `phases` walk rows lie side by side in a block, `per_sample` of them in one
// sample; each thread has up to NV rows.  Several samples share a block where
// there are many.  (Blocks that take several sets of samples in turn, parameters
// kept, lost: f16 300x48x256 7.7 us to 10.8.)
//
// Statistics: sums and sums of squares of the distances from a centre of the group,
// the median of three of its values (the first, a middle, the last; or 0, see centre3),
// so that no single outlier moves it: k standard deviations off the mean it multiplies the
// rounding of the sums by 1 + k^2.  Where far_off() shows k > 4 (two outliers of the
// three) the block sums again, from its registers, about the means so found, and the
// groups concerned take those sums.  All in float32, in an order that does not depend
// on timing.  (The squares about the mean in every block, as a second pass, took two
// more block sums: f16 1x64x256 5.7 us and 4.7, f32 9651x2x459 122 and 68.)
//
// What bounds it: the latency of load, two block reductions and store (f16 1x64x256
// 4.3 us, 76 such samples 4.5; as a split form 7.7 and 10.2).  Where there are
// thousands of samples, the instructions of MODE 1 and 2 (bf16 9668x1x2976
// in groups of 93 110 us, of which 18 are its bytes).  (Spreading
// a larger sample over a cluster of up to 16 blocks, with the groups' sums in
// distributed shared memory, was built and measured: 7.0 us against the split
// form's 8.6 for f16 2x256x1280, but 20.7 against 11.0 for 2x4096x320 and 156
// against 66 for bf16 8x16384x512, so larger samples take the split form.)
#include <algorithm>
#include <climits>
#include <numeric>
#include <type_traits>

#include "column_walk.cuh"
#include "device_common.cuh"
#include "group_norm.cuh"
#include "launch_util.h"
#include "smem_limit.h"
#include "training_internal.h"

namespace ep {
namespace {

constexpr int kMaxThreads = 512, kWideThreads = 1024;  // kWideThreads: samples of one walk row

struct FusedPlan {
  int W;              // channels: C
  int cf;             // fragments of a walk row
  int phases, per_sample, samples;  // walk rows side by side, of one sample, samples in a block
  int threads, nv;
  int rows;           // walk rows of a sample
  int reps;           // times each channel occurs in a thread's walk rows of a sample, side by side
  bool direct;        // entries are columns: one repeat (MODE 2: and one position a sample)
  int64_t items;      // blocks of samples
  int64_t grid_items; // the gradient: items that run at a time
};

struct FusedDims {
  int64_t N, S, L;  // (a sample that fits a block has less than 2^31 elements)
  int C, G, D;
  float eps, scale;   // scale: 1 / (S D)
  bool silu;
  bool pvec;          // gamma and beta 16-byte aligned
  FusedPlan p;
};

// Where a thread stands in an item.
template <typename T, int MODE>
struct Place {
  static constexpr int VW = dev::Vec16<T>::N;
  int64_t n;   // its sample
  int e0;      // its first fragment's first element, from the sample's start
  int stride;  // elements from one of its fragments to the next
  int lim;     // MODE 2: elements of the sample
  int off;
  int kn;      // its fragments

  __device__ __forceinline__ Place(const FusedDims& d, const T* x, unsigned item, int trow, int tcol, int ns) {
    const FusedPlan& p = d.p;
    const int ph = trow - ns * p.per_sample;
    n = int64_t(item) * p.samples + ns;
    const bool live = trow < p.phases && n < d.N;
    off = MODE == 2 && live ? dev::misalignment(x + n * d.L) : 0;
    const int row = p.cf * VW;  // (C where C % VW == 0)
    kn = !live || ph >= p.rows          ? 0
         : p.rows <= p.per_sample       ? 1
                                        : static_cast<int>(unsigned(p.rows - ph + p.per_sample - 1) / unsigned(p.per_sample));
    e0 = ph * row + tcol * VW - off;
    stride = p.per_sample * row;
    lim = static_cast<int>(d.L);
  }
  __device__ __forceinline__ bool whole(int k) const {
    return MODE != 2 || (e0 + k * stride >= 0 && e0 + k * stride + VW <= lim);
  }
  __device__ __forceinline__ bool inside(int k, int e) const {
    return MODE != 2 || unsigned(e0 + k * stride + e) < unsigned(lim);
  }
  // Fragment k, where it lies in the sample, on its way into L2.
  __device__ __forceinline__ void prefetch(const T* base, int k) const {
    const int at = e0 + k * stride;
    if (MODE != 2 || unsigned(at) < unsigned(lim)) asm volatile("prefetch.global.L2 [%0];" ::"l"(base + at));
  }
  __device__ __forceinline__ uint4 load(const T* base, int k) const {
    const T* at = base + (e0 + k * stride);
    if (whole(k)) return dev::ld16_stream(at);
    float v[VW];
#pragma unroll
    for (int e = 0; e < VW; ++e) v[e] = inside(k, e) ? dev::ld1_stream(at + e) : 0.f;
    return dev::Conv<T>::pack(v);  // exact: the values are T's
  }
  __device__ __forceinline__ void store(T* base, int k, const float (&v)[VW]) const {
    T* at = base + (e0 + k * stride);
    if (whole(k)) {
      dev::st16_stream(at, dev::Conv<T>::pack(v));
    } else {
#pragma unroll
      for (int e = 0; e < VW; ++e)
        if (inside(k, e)) dev::st1_stream(at + e, v[e]);
    }
  }
};

// The channel of the first element of a thread's fragments.
__device__ __forceinline__ int fused_channel(int tcol, int vw, int off, int W) {
  const unsigned c = unsigned(tcol * vw + W - (off < W ? off : off % W));
  return static_cast<int>(c < unsigned(W) ? c : c < 2u * unsigned(W) ? c - unsigned(W) : c % unsigned(W));
}

// Sums over the entries of each (sample, group) of a block, in two steps: over
// the repeats of each column (fragments in MODE 0, else channels), then over a
// group's columns.  Entries are floats by position; column c of sample ns is at
// start[ns] + c + k Cw, modulo the np positions of a sample (the positions before
// its start hold the channels that the last repeat misses; MODE 0, 1: no starts).
template <int MODE>
struct Entries {
  int De, Cw, np, reps, q, slots, cols;
  bool direct;
  const int* start;
  __device__ __forceinline__ Entries(const FusedPlan& p, int D, int VW, const int* start_) : start(start_) {
    De = MODE == 0 ? D / VW : D;
    Cw = MODE == 0 ? p.cf : p.W;
    np = p.per_sample * p.cf * (MODE == 0 ? 1 : VW);
    reps = p.reps;
    q = p.W / D;
    slots = p.samples * q;
    cols = p.samples * Cw;
    direct = p.direct;
  }
  __device__ __forceinline__ int sample_of(int slot) const {
    return slots == q ? 0 : static_cast<int>(unsigned(slot) / unsigned(q));
  }
  // The columns' sums, where entries are not columns already: add(position, a, b)
  // for each entry, into col_a (and col_b).
  template <typename ADD>
  __device__ __forceinline__ void columns(float* col_a, float* col_b, ADD add) const {
    if (direct) return;
    sum_sets(blockDim.x, cols, reps,
             [&](int i, int k, float& a, float& b) {
               const int ns = cols == Cw ? 0 : static_cast<int>(unsigned(i) / unsigned(Cw));
               int pos = (i - ns * Cw) + k * Cw;
               if constexpr (MODE == 2) {
                 pos += start[ns];
                 if (pos >= np) pos -= np;
               }
               add(ns * np + pos, a, b);
             },
             [&](int i, float a, float b) {
               col_a[i] = a;
               col_b[i] = b;
             });
    __syncthreads();
  }
  // MODE 2: where sample ns's columns stand, in the entries (direct) or the columns' sums.
  __device__ __forceinline__ int base(int ns) const { return direct ? ns * np + start[ns] : ns * Cw; }
  // The groups' sums: add(column's place, channel (MODE 2), a, b), then done(slot,
  // sample, a, b) by one lane.
  template <typename ADD, typename DONE>
  __device__ __forceinline__ void groups(ADD add, DONE done) const {
    sum_sets(blockDim.x, slots, De,
             [&](int s, int k, float& a, float& b) {
               if constexpr (MODE == 2) {
                 const int ns = sample_of(s), c = (s - ns * q) * De + k;
                 add(base(ns) + c, c, a, b);
               } else {
                 add(s * De + k, 0, a, b);  // (at ns Cw + g De + k, direct or not)
               }
             },
             [&](int s, float a, float b) { done(s, sample_of(s), a, b); });
  }
  // Both.
  template <typename ADD, typename DONE>
  __device__ __forceinline__ void run(const float* ent_a, const float* ent_b, float* col_a, float* col_b, ADD add,
                                      DONE done) const {
    columns(col_a, col_b, add);
    const float* ca = direct ? ent_a : col_a;
    const float* cb = direct ? ent_b : col_b;
    groups(
        [&](int i, int, float& a, float& b) {
          a += ca[i];
          b += cb[i];
        },
        done);
  }
};

// Where each sample of an item starts in its first fragment, by the first threads.
template <typename T>
__device__ __forceinline__ void put_starts(int* start, const FusedDims& d, const T* x, unsigned item) {
  if (int(threadIdx.x) < d.p.samples) {
    const int64_t n = int64_t(item) * d.p.samples + threadIdx.x;
    start[threadIdx.x] = n < d.N ? dev::misalignment(x + n * d.L) : 0;
  }
}

// gamma and beta of VW channels from c on (modulo W).
template <typename T, bool WRAP>
__device__ __forceinline__ void load_params(const T* __restrict__ gamma, const T* __restrict__ beta, int c, int W,
                                            bool vec, float (&a)[dev::Vec16<T>::N],
                                            float (&b)[dev::Vec16<T>::N]) {
  constexpr int VW = dev::Vec16<T>::N;
#pragma unroll
  for (int e = 0; e < VW; ++e) b[e] = 0.f;
  if (!WRAP && vec) {
    dev::Conv<T>::unpack(dev::ld16_keep(gamma + c), a);
    if (beta != nullptr) dev::Conv<T>::unpack(dev::ld16_keep(beta + c), b);
  } else {
#pragma unroll
    for (int e = 0; e < VW; ++e) {
      a[e] = dev::ld1_keep(gamma + c);
      if (beta != nullptr) b[e] = dev::ld1_keep(beta + c);
      if (++c == W) c = 0;
    }
  }
}

// Sums over `set` neighbouring lanes (a power of two).
__device__ __forceinline__ float set_sum(float x, int set) {
  for (int o = set >> 1; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}

// A thread's entries to their positions, 16 bytes at a time where there are several.
template <int EV>
__device__ __forceinline__ void put_entries(float* ent, const float (&v)[EV]) {
  if constexpr (EV == 1) {
    ent[threadIdx.x] = v[0];
  } else {
#pragma unroll
    for (int e = 0; e < EV; e += 4)
      *reinterpret_cast<float4*>(ent + threadIdx.x * EV + e) = make_float4(v[e], v[e + 1], v[e + 2], v[e + 3]);
  }
}

// A thread's sums of its values' distances from a centre, and of their squares.
template <typename T, int NV, int MODE>
__device__ __forceinline__ void centred_sums(const uint4 (&raw)[NV], const Place<T, MODE>& at,
                                             const float (&c)[MODE == 0 ? 1 : dev::Vec16<T>::N],
                                             float (&s)[MODE == 0 ? 1 : dev::Vec16<T>::N],
                                             float (&q)[MODE == 0 ? 1 : dev::Vec16<T>::N]) {
  constexpr int VW = dev::Vec16<T>::N;
  float ts[VW], tq[VW];
#pragma unroll
  for (int e = 0; e < VW; ++e) ts[e] = tq[e] = 0.f;
#pragma unroll
  for (int k = 0; k < NV; ++k) {
    if (k < at.kn) {
      float v[VW];
      dev::Conv<T>::unpack(raw[k], v);
#pragma unroll
      for (int e = 0; e < VW; ++e) v[e] -= c[MODE == 0 ? 0 : e];
      if (MODE == 2 && !at.whole(k)) {
#pragma unroll
        for (int e = 0; e < VW; ++e) v[e] = at.inside(k, e) ? v[e] : 0.f;
      }
      dev::add_pairs(ts, v);
      fma_pairs(v, v, tq);
    }
  }
  if constexpr (MODE == 0) {
    s[0] = q[0] = 0.f;
#pragma unroll
    for (int e = 0; e < VW; ++e) {
      s[0] += ts[e];
      q[0] += tq[e];
    }
  } else {
#pragma unroll
    for (int e = 0; e < VW; ++e) {
      s[e] = ts[e];
      q[e] = tq[e];
    }
  }
}

template <typename T, int NV, int MODE, int THREADS>
__global__ void __launch_bounds__(THREADS)
k_gn_fused(const T* x, const T* __restrict__ gamma, const T* __restrict__ beta, T* y, float* mean_out,
           float* inv_out, FusedDims d) {
  constexpr int VW = dev::Vec16<T>::N;
  constexpr int EV = MODE == 0 ? 1 : VW;  // entries of a thread
  extern __shared__ __align__(16) float smem[];
  const FusedPlan& p = d.p;
  const int slots = p.samples * d.G, ents = p.phases * p.cf * EV;
  float* ent_a = smem;             // sums and sums of squares by position
  float* ent_b = ent_a + ents;
  const int cols = p.direct ? 0 : p.samples * (MODE == 0 ? p.cf : p.W);
  float* col_a = ent_b + ents;     // by column
  float* col_b = col_a + cols;
  float* gm = col_b + cols;        // the groups' centres, then means
  float* gr = gm + slots;
  int* start = reinterpret_cast<int*>(gr + slots);  // MODE 2: the samples' starts
  const unsigned item = blockIdx.x;
  const int trow = p.phases == 1 ? (int(threadIdx.x) < p.cf ? 0 : 1) : int(threadIdx.x / unsigned(p.cf));
  const int tcol = threadIdx.x - trow * p.cf;
  const int ns = p.samples == 1 ? 0 : int(unsigned(trow) / unsigned(p.per_sample));
  dev::pdl_wait();
  dev::pdl_trigger();

  const Place<T, MODE> at(d, x, item, trow, tcol, ns);
  const T* xs = x + (at.kn > 0 ? at.n * d.L : 0);
  uint4 raw[NV];
#pragma unroll
  for (int k = 0; k < NV; ++k)
    if (k < at.kn) raw[k] = at.load(xs, k);

  if constexpr (MODE == 2) put_starts(start, d, x, item);
  const int64_t n0 = int64_t(item) * p.samples;
  const int mid = static_cast<int>(d.S / 2) * d.C + d.D / 2, end = static_cast<int>(d.L) - d.C + d.D - 1;
  for (int s = threadIdx.x; s < slots; s += blockDim.x) {
    const int sn = p.samples == 1 ? 0 : int(unsigned(s) / unsigned(d.G));
    if (n0 + sn < d.N) {
      const T* first = x + (n0 + sn) * d.L + (s - sn * d.G) * d.D;
      gm[s] = centre3(dev::ld1_stream(first), dev::ld1_stream(first + mid), dev::ld1_stream(first + end));
    }
  }
  // this thread's channels and groups
  const int c0 = fused_channel(tcol, VW, at.off, p.W);
  int grp[EV];
  for_channels<VW>(c0, p.W, d.D, [&](int e, int, int g) {
    if (e < EV) grp[e] = ns * d.G + g;
  });
  const bool mine = trow < p.phases;
  const Entries<MODE> entries(p, d.D, VW, start);
  __syncthreads();

  bool far = false;
  auto statistics = [&](auto second) {
    constexpr bool again = decltype(second)::value;
    float m[EV], s[EV], q[EV];
#pragma unroll
    for (int e = 0; e < EV; ++e) m[e] = at.kn > 0 ? gm[grp[e]] : 0.f;
    centred_sums<T, NV, MODE>(raw, at, m, s, q);
    if (mine) {
      put_entries(ent_a, s);
      put_entries(ent_b, q);
    }
    __syncthreads();
    entries.run(
        ent_a, ent_b, col_a, col_b,
        [&](int i, float& a, float& b) {
          a += ent_a[i];
          b += ent_b[i];
        },
        [&](int s, int ns, float a, float b) {
          if (again && !(gr[s] < 0.f)) return;  // this group's centre was near
          const float m = a * d.scale;  // from the centre
          const float m2 = not_negative(b - a * m);
          const float mean = gm[s] + m, r = 1.0f / sqrtf(m2 * d.scale + d.eps);
          const bool redo = !again && far_off(a * m, m2);
          far |= redo;
          gm[s] = mean;
          gr[s] = redo ? -r : r;
          if (n0 + ns < d.N) {
            const int64_t i = n0 * d.G + s;  // (slots are samples' groups in order)
            if (mean_out != nullptr) mean_out[i] = mean;
            if (inv_out != nullptr) inv_out[i] = r;
          }
        });
  };
  statistics(std::false_type{});
  if (__syncthreads_or(far)) {
    statistics(std::true_type{});
    __syncthreads();
  }

  // y
  if (at.kn > 0) {
    float mu[EV], a[VW], b[VW];
    load_params<T, MODE == 2>(gamma, beta, c0, p.W, d.pvec, a, b);
#pragma unroll
    for (int e = 0; e < EV; ++e) mu[e] = gm[grp[e]];
#pragma unroll
    for (int e = 0; e < VW; ++e) a[e] *= gr[grp[MODE == 0 ? 0 : e]];
    T* ys = y + at.n * d.L;
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      if (k < at.kn) {
        float v[VW];
        dev::Conv<T>::unpack(raw[k], v);
        centre_scale_add(v, mu, a, b);
        if (d.silu) activate<T>(v);
        at.store(ys, k, v);
      }
    }
  }
}

// The gradient.  A CTA takes items in turn (grid_items apart) and keeps the sums
// of du and du * h of its channels over them, in registers or (MODE 2, where a
// thread's channels change with the sample's start) in shared memory; they leave
// once, as row blockIdx of cpart: 2 x [row][C].
template <typename T, int NV, int MODE, int THREADS>
__global__ void __launch_bounds__(THREADS)
k_gn_grad_fused(const T* dy, const T* x, const T* __restrict__ gamma, const T* __restrict__ beta, const float* mean,
                const float* inv, T* dx, float* cpart, FusedDims d) {
  constexpr int VW = dev::Vec16<T>::N;
  constexpr int EV = MODE == 0 ? 1 : VW;
  extern __shared__ __align__(16) float smem[];
  const FusedPlan& p = d.p;
  const int slots = p.samples * d.G, ents = p.phases * p.cf * VW;
  float* ent_a = smem;
  float* ent_b = ent_a + ents;
  const int cols = p.direct ? 0 : p.samples * (MODE == 0 ? p.cf : p.W);
  float* col_a = ent_b + ents;
  float* col_b = col_a + cols;
  float* g1 = col_b + cols;
  float* g2 = g1 + slots;
  float* ch_a = g2 + slots;  // MODE 2: the channels' sums, and gamma
  float* ch_b = ch_a + p.W;
  float* ch_g = ch_b + p.W;
  int* start = reinterpret_cast<int*>(ch_g + p.W);
  const unsigned first = blockIdx.x;
  const int trow = p.phases == 1 ? (int(threadIdx.x) < p.cf ? 0 : 1) : int(threadIdx.x / unsigned(p.cf));
  const int tcol = threadIdx.x - trow * p.cf;
  const int ns = p.samples == 1 ? 0 : int(unsigned(trow) / unsigned(p.per_sample));
  const bool mine = trow < p.phases;
  const float scale = d.scale;
  const Entries<MODE> entries(p, d.D, VW, start);
  dev::pdl_wait();
  dev::pdl_trigger();

  float tot_a[VW], tot_b[VW], ga[VW], be[VW];
  int grp[EV];
#pragma unroll
  for (int e = 0; e < VW; ++e) tot_a[e] = tot_b[e] = ga[e] = be[e] = 0.f;
  int off = -1;
  const int64_t ahead = p.grid_items * p.samples;  // samples to the next item
  if constexpr (MODE == 2) {
    for (int c = threadIdx.x; c < p.W; c += blockDim.x) {  // (used after the first item's first barrier)
      ch_a[c] = ch_b[c] = 0.f;
      ch_g[c] = dev::ld1_keep(gamma + c);
    }
  }

  for (unsigned item = first; item < unsigned(p.items); item += unsigned(p.grid_items)) {
    if constexpr (MODE == 2) put_starts(start, d, x, item);
    const Place<T, MODE> at(d, x, item, trow, tcol, ns);
    const int64_t base = at.kn > 0 ? at.n * d.L : 0;
    uint4 raw[NV], rdy[NV];
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      if (k < at.kn) {
        raw[k] = at.load(x + base, k);
        rdy[k] = at.load(dy + base, k);
      }
    }
    if (at.n + ahead < d.N) {
#pragma unroll
      for (int k = 0; k < NV; ++k) {
        if (k < at.kn) {
          at.prefetch(x + base + ahead * d.L, k);
          at.prefetch(dy + base + ahead * d.L, k);
        }
      }
    }
    if (off != at.off && mine) {
      off = at.off;
      const int c0 = fused_channel(tcol, VW, off, p.W);
      load_params<T, MODE == 2>(gamma, beta, c0, p.W, d.pvec, ga, be);
      for_channels<VW>(c0, p.W, d.D, [&](int e, int, int g) {
        if (e < EV) grp[e] = g;
      });
    }
    float mu[EV], rs[EV];
    const int64_t ng = at.n * d.G;
#pragma unroll
    for (int e = 0; e < EV; ++e) {
      mu[e] = at.kn > 0 ? mean[ng + grp[e]] : 0.f;
      rs[e] = at.kn > 0 ? inv[ng + grp[e]] : 0.f;
    }
    float sa[VW], sb[VW];
#pragma unroll
    for (int e = 0; e < VW; ++e) sa[e] = sb[e] = 0.f;
    // h and du of fragment k (0 outside the sample: adds nothing)
    auto values = [&](int k, float (&h)[VW], float (&du)[VW]) {
      dev::Conv<T>::unpack(raw[k], h);
      dev::Conv<T>::unpack(rdy[k], du);
      centre_scale(h, mu, rs);
      if (d.silu) {
        float u[VW];
#pragma unroll
        for (int e = 0; e < VW; ++e) u[e] = be[e];
        fma_pairs(h, ga, u);
        activate_grad<T>(du, u);
      }
    };
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      if (k < at.kn) {
        float h[VW], du[VW];
        values(k, h, du);
        dev::add_pairs(sa, du);
        fma_pairs(du, h, sb);
      }
    }
    if (mine) {
      if constexpr (MODE == 0) {
        float a = 0.f, b = 0.f;
#pragma unroll
        for (int e = 0; e < VW; ++e) {
          a = fmaf(sa[e], ga[e], a);
          b = fmaf(sb[e], ga[e], b);
        }
        ent_a[threadIdx.x] = a;
        ent_b[threadIdx.x] = b;
      } else if constexpr (MODE == 1) {
        float a[VW], b[VW];
#pragma unroll
        for (int e = 0; e < VW; ++e) {
          a[e] = sa[e] * ga[e];
          b[e] = sb[e] * ga[e];
        }
        put_entries(ent_a, a);
        put_entries(ent_b, b);
      } else {
        put_entries(ent_a, sa);
        put_entries(ent_b, sb);
      }
      if constexpr (MODE != 2) {
        dev::add_pairs(tot_a, sa);
        dev::add_pairs(tot_b, sb);
      }
    }
    __syncthreads();
    auto means = [&](int s, int, float a, float b) {
      g1[s] = a * scale;
      g2[s] = b * scale;
    };
    auto entry = [&](int i, float& a, float& b) {
      a += ent_a[i];
      b += ent_b[i];
    };
    if constexpr (MODE != 2) {
      entries.run(ent_a, ent_b, col_a, col_b, entry, means);
    } else {
      entries.columns(col_a, col_b, entry);
      const float* ca = entries.direct ? ent_a : col_a;
      const float* cb = entries.direct ? ent_b : col_b;
      for (int c = threadIdx.x; c < p.W; c += blockDim.x) {
        float a = ch_a[c], b = ch_b[c];
        for (int s = 0; s < p.samples; ++s) {
          a += ca[entries.base(s) + c];
          b += cb[entries.base(s) + c];
        }
        ch_a[c] = a;
        ch_b[c] = b;
      }
      entries.groups(
          [&](int i, int c, float& a, float& b) {
            a = fmaf(ca[i], ch_g[c], a);
            b = fmaf(cb[i], ch_g[c], b);
          },
          means);
    }
    __syncthreads();
    if (at.kn > 0) {
      float a1[EV], a2[EV];
#pragma unroll
      for (int e = 0; e < EV; ++e) {
        a1[e] = g1[ns * d.G + grp[e]];
        a2[e] = g2[ns * d.G + grp[e]];
      }
#pragma unroll
      for (int k = 0; k < NV; ++k) {
        if (k < at.kn) {
          float h[VW], v[VW];
          values(k, h, v);  // again: keeping du would cost more registers than the block has
#pragma unroll
          for (int e = 0; e < VW; ++e) {
            const int i = MODE == 0 ? 0 : e;
            v[e] = rs[i] * (fmaf(v[e], ga[e], -a1[i]) - h[e] * a2[i]);
          }
          at.store(dx + base, k, v);
        }
      }
    }
    // (g1, g2 are written again only after the next item's first barrier)
  }

  if (cpart == nullptr) return;
  __syncthreads();
  if constexpr (MODE == 2) {
    for (int c = threadIdx.x; c < p.W; c += blockDim.x) {
      float* out = cpart + int64_t(first) * d.C + c;
      out[0] = ch_a[c];
      out[p.grid_items * d.C] = ch_b[c];
    }
    return;
  }
  if (mine) {
    put_entries(ent_a, tot_a);
    put_entries(ent_b, tot_b);
  }
  __syncthreads();
  // channel c is at c + k W in every sample
  const int np = p.per_sample * p.cf * VW, reps = p.per_sample;
  const int many = reps * p.samples;
  const int set = many >= 32 ? 32 : 1;  // lanes to a channel
  for (int c = threadIdx.x / set; c < p.W; c += blockDim.x / set) {
    float a = 0.f, b = 0.f;
    for (int i = threadIdx.x & (set - 1); i < many; i += set) {
      const int pos = c + i % reps * p.W + i / reps * np;
      a += ent_a[pos];
      b += ent_b[pos];
    }
    if (set == 32) {  // (a warp's lanes share c)
      a = dev::warp_sum(a);
      b = dev::warp_sum(b);
    }
    if ((threadIdx.x & (set - 1)) == 0) {
      float* out = cpart + int64_t(first) * d.C + c;
      out[0] = a;
      out[p.grid_items * d.C] = b;
    }
  }
}

// ---------------------------------------------------------------------------
// One position a sample (S = 1), D % VW == 0: the norm over each token's groups.  A
// group's fragments are on neighbouring lanes (`set`, a power of two up to 32, where
// lanes beyond the group's fragments idle), NV on each, so its sums are shuffles and
// there is no shared memory and no barrier.  A block has `cols` lanes, of whole
// groups, and `rows` tokens side by side; it takes every grid-th set of tokens, so
// its channels stay the same.  U tokens are loaded before the first is used.
// ---------------------------------------------------------------------------

struct TokenPlan {
  int cols, rows, tiles, ctas;  // ctas: of each tile
  int set, log_set, nv;
};

struct TokenDims {
  int64_t N, C;
  int G, frags, tile_groups;    // fragments of a group, groups of a tile
  float eps, scale;             // scale: 1 / D
  bool silu, pvec;
  TokenPlan p;
};

// A thread's place: its token row, group and first fragment in the group.
struct TokenPlace {
  int trow, g, li, row;
  bool mine;  // uniform in a set
  __device__ __forceinline__ explicit TokenPlace(const TokenDims& d) {
    trow = threadIdx.x / unsigned(d.p.cols);
    const int lane = threadIdx.x - trow * d.p.cols, tile = blockIdx.x % unsigned(d.p.tiles);
    row = static_cast<int>(blockIdx.x / unsigned(d.p.tiles));
    g = tile * d.tile_groups + (lane >> d.p.log_set);
    li = lane & (d.p.set - 1);
    mine = trow < d.p.rows && g < d.G;
  }
  // Whether the thread has fragment k of its group, and its first channel.
  __device__ __forceinline__ bool has(const TokenDims& d, int k) const { return li + k * d.p.set < d.frags; }
  template <int VW>
  __device__ __forceinline__ int channel(const TokenDims& d, int k) const {
    return (g * d.frags + li + k * d.p.set) * VW;
  }
};

template <typename T, int NV>
__global__ void __launch_bounds__(kWalkThreads)
k_gn_token(const T* x, const T* __restrict__ gamma, const T* __restrict__ beta, T* y, float* mean_out,
           float* inv_out, TokenDims d) {
  constexpr int VW = dev::Vec16<T>::N;
  constexpr int U = NV >= 4 ? 1 : 4 / NV;
  dev::pdl_wait();
  dev::pdl_trigger();
  const TokenPlace at(d);
  const int64_t step = int64_t(d.p.ctas) * d.p.rows, n1 = d.N, first_row = int64_t(at.row) * d.p.rows;
  int64_t n = first_row + at.trow;
  const int lead = (threadIdx.x & 31) & ~(d.p.set - 1);
  // one fragment: the parameters stay in registers
  float a[VW], b[VW];
  if (NV == 1 && at.mine && at.has(d, 0))
    load_params<T, false>(gamma, beta, at.channel<VW>(d, 0), 0, d.pvec, a, b);
  // every lane of a warp goes round as often as its first (the shuffles are whole warps')
  const int rounds = static_cast<int>((n1 - first_row + step * U - 1) / (step * U));
  for (int i = 0; i < rounds; ++i, n += step * U) {
    uint4 raw[U][NV];
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int k = 0; k < NV; ++k)
        if (at.mine && n + u * step < n1 && at.has(d, k))
          raw[u][k] = dev::ld16_stream(x + (n + u * step) * d.C + at.channel<VW>(d, k));
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const bool on = at.mine && n + u * step < n1;
      float v[NV][VW];
#pragma unroll
      for (int k = 0; k < NV; ++k) {
        if (on && at.has(d, k)) {
          dev::Conv<T>::unpack(raw[u][k], v[k]);
        } else {
#pragma unroll
          for (int e = 0; e < VW; ++e) v[k][e] = 0.f;
        }
      }
      // the first value, or 0 where the first fragment's ends are farther apart (see centre3)
      const float v0 = __shfl_sync(0xffffffffu, v[0][0], lead), v1 = __shfl_sync(0xffffffffu, v[0][VW - 1], lead);
      const float first = fabsf(v0) <= fabsf(v1 - v0) ? 0.f : v0;
      float s = 0.f, q = 0.f;
#pragma unroll
      for (int k = 0; k < NV; ++k)
        if (at.has(d, k))
#pragma unroll
          for (int e = 0; e < VW; ++e) s += v[k][e] - first;
      const float m = set_sum(s, d.p.set) * d.scale;
      float mu = first + m, by = m - (mu - first);
#pragma unroll
      for (int k = 0; k < NV; ++k) {
#pragma unroll
        for (int e = 0; e < VW; ++e) v[k][e] -= mu;
        if (at.has(d, k))
#pragma unroll
          for (int e = 0; e < VW; ++e) q = fmaf(v[k][e], v[k][e], q);
      }
      q = set_sum(q, d.p.set) * d.scale;  // relative to mu, which is rounded: `by` off the mean
      float var = not_negative(q - by * by);
      // `first` far off the mean: so is mu, by the rounding of so distant a sum
      if (__any_sync(0xffffffffu, m * m > 16.f * var)) {
        s = 0.f;
#pragma unroll
        for (int k = 0; k < NV; ++k)
          if (at.has(d, k))
#pragma unroll
            for (int e = 0; e < VW; ++e) s += v[k][e];
        const float res = set_sum(s, d.p.set) * d.scale;
        if (far_off(m * m, var)) {
          mu += res;
          var = not_negative(q - res * res);
#pragma unroll
          for (int k = 0; k < NV; ++k)
#pragma unroll
            for (int e = 0; e < VW; ++e) v[k][e] -= res;
        }
      }
      const float r = 1.0f / sqrtf(var + d.eps);
      const int64_t t = n + u * step;
#pragma unroll
      for (int k = 0; k < NV; ++k) {
        if (on && at.has(d, k)) {
          if constexpr (NV > 1) load_params<T, false>(gamma, beta, at.channel<VW>(d, k), 0, d.pvec, a, b);
#pragma unroll
          for (int e = 0; e < VW; ++e) {
            v[k][e] = fmaf(v[k][e], a[e] * r, b[e]);
            if (d.silu) v[k][e] = silu<T>(v[k][e]);
          }
          dev::st16_stream(y + t * d.C + at.channel<VW>(d, k), dev::Conv<T>::pack(v[k]));
        }
      }
      if (on && at.li == 0) {
        if (mean_out != nullptr) mean_out[t * d.G + at.g] = mu;
        if (inv_out != nullptr) inv_out[t * d.G + at.g] = r;
      }
    }
  }
}

// The gradient; the sums for dgamma and dbeta run on in registers and leave as
// row blockIdx / tiles of cpart: 2 x [ctas][C].
template <typename T, int NV>
__global__ void __launch_bounds__(kWalkThreads)
k_gn_grad_token(const T* dy, const T* x, const T* __restrict__ gamma, const T* __restrict__ beta, const float* mean,
                const float* inv, T* dx, float* cpart, TokenDims d) {
  constexpr int VW = dev::Vec16<T>::N;
  constexpr int U = NV == 1 ? 2 : 1;
  __shared__ __align__(16) float s_a[kWalkThreads * VW], s_b[kWalkThreads * VW];
  dev::pdl_wait();
  dev::pdl_trigger();
  const TokenPlace at(d);
  const int64_t step = int64_t(d.p.ctas) * d.p.rows, n1 = d.N, first_row = int64_t(at.row) * d.p.rows;
  int64_t n = first_row + at.trow;
  float ga[VW], be[VW], tot_a[NV][VW], tot_b[NV][VW];
#pragma unroll
  for (int e = 0; e < VW; ++e) {
    ga[e] = be[e] = 0.f;
#pragma unroll
    for (int k = 0; k < NV; ++k) tot_a[k][e] = tot_b[k][e] = 0.f;
  }
  if (NV == 1 && at.mine && at.has(d, 0))
    load_params<T, false>(gamma, beta, at.channel<VW>(d, 0), 0, d.pvec, ga, be);
  const int rounds = static_cast<int>((n1 - first_row + step * U - 1) / (step * U));
  for (int i = 0; i < rounds; ++i, n += step * U) {
    uint4 rx[U][NV], rd[U][NV];
    float mu[U], rs[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t t = n + u * step;
      if (at.mine && t < n1) {
#pragma unroll
        for (int k = 0; k < NV; ++k) {
          if (at.has(d, k)) {
            rx[u][k] = dev::ld16_stream(x + t * d.C + at.channel<VW>(d, k));
            rd[u][k] = dev::ld16_stream(dy + t * d.C + at.channel<VW>(d, k));
          }
        }
        mu[u] = mean[t * d.G + at.g];
        rs[u] = inv[t * d.G + at.g];
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t t = n + u * step;
      const bool on = at.mine && t < n1;
      float h[NV][VW], w[NV][VW], p = 0.f, q = 0.f;
#pragma unroll
      for (int k = 0; k < NV; ++k) {
        if (on && at.has(d, k)) {
          if constexpr (NV > 1) load_params<T, false>(gamma, beta, at.channel<VW>(d, k), 0, d.pvec, ga, be);
          dev::Conv<T>::unpack(rx[u][k], h[k]);
          dev::Conv<T>::unpack(rd[u][k], w[k]);
#pragma unroll
          for (int e = 0; e < VW; ++e) {
            h[k][e] = (h[k][e] - mu[u]) * rs[u];
            if (d.silu) w[k][e] = silu_grad<T>(w[k][e], fmaf(h[k][e], ga[e], be[e]));
            tot_a[k][e] += w[k][e];
            tot_b[k][e] = fmaf(w[k][e], h[k][e], tot_b[k][e]);
            w[k][e] *= ga[e];
            p += w[k][e];
            q = fmaf(w[k][e], h[k][e], q);
          }
        }
      }
      p = set_sum(p, d.p.set) * d.scale;
      q = set_sum(q, d.p.set) * d.scale;
#pragma unroll
      for (int k = 0; k < NV; ++k) {
        if (on && at.has(d, k)) {
#pragma unroll
          for (int e = 0; e < VW; ++e) w[k][e] = rs[u] * ((w[k][e] - p) - h[k][e] * q);
          dev::st16_stream(dx + t * d.C + at.channel<VW>(d, k), dev::Conv<T>::pack(w[k]));
        }
      }
    }
  }
  if (cpart == nullptr) return;
#pragma unroll
  for (int k = 0; k < NV; ++k) {
    if (k > 0) __syncthreads();
    put_entries(s_a, tot_a[k]);
    put_entries(s_b, tot_b[k]);
    __syncthreads();
    const int W = d.p.cols * VW, tile0 = static_cast<int>(blockIdx.x % unsigned(d.p.tiles)) * d.tile_groups;
    for (int i = threadIdx.x; i < W; i += blockDim.x) {
      const int lane = i / VW, g = tile0 + (lane >> d.p.log_set), f = (lane & (d.p.set - 1)) + k * d.p.set;
      if (g >= d.G || f >= d.frags) continue;
      float sa = 0.f, sb = 0.f;
      for (int r = 0; r < d.p.rows; ++r) {
        sa += s_a[r * W + i];
        sb += s_b[r * W + i];
      }
      float* out = cpart + int64_t(at.row) * d.C + (g * d.frags + f) * VW + i % VW;
      out[0] = sa;
      out[int64_t(d.p.ctas) * d.C] = sb;
    }
  }
}

// ---------------------------------------------------------------------------
// plans
// ---------------------------------------------------------------------------

int pow2_at_least(int64_t v) {
  int p = 1;
  while (p < v) p *= 2;
  return p;
}

// Up to this many fragments a sample has a block of 256 threads, beyond that one of 512.
constexpr int64_t kSmallFrags = 4 * kWalkThreads;

// slab: C % vw == 0 and 16-byte-aligned operands; else the walk over whole
// samples.  False where a sample is too large for a block of nv_max fragments a thread.
bool fused_plan(int vw, int64_t N, int64_t S, int64_t C, bool slab, int nv_max, FusedPlan* p) {
  if (slab && C % vw != 0) return false;
  const int64_t all = (S * C + 2 * (vw - 1)) / vw;  // of a sample, wherever it starts
  const int64_t period = slab ? C / vw : std::min(C / std::gcd(C, int64_t(vw)), all);
  const int64_t rows = slab ? S : (all + period - 1) / period;
  if (period > (rows == 1 ? kWideThreads : kMaxThreads)) return false;
  p->W = int(C);
  p->cf = int(period);
  const int64_t frags = rows * period;
  if (frags > int64_t(kMaxThreads) * nv_max) return false;
  p->rows = int(rows);
  const int threads = frags > kSmallFrags ? kMaxThreads : kWalkThreads;
  const int phases = std::max(1, threads / p->cf);
  p->per_sample = int(std::min<int64_t>(rows, phases));
  while ((rows + p->per_sample - 1) / p->per_sample > nv_max && p->cf * (p->per_sample + 1) <= kMaxThreads)
    p->per_sample += 1;
  if ((rows + p->per_sample - 1) / p->per_sample > nv_max) return false;
  // other samples beside it, where there are enough of them
  const int64_t fit = std::max(1, phases / p->per_sample);
  p->samples = int(std::max<int64_t>(1, std::min(fit, N / (2 * kPlanSms))));
  p->phases = p->samples * p->per_sample;
  p->direct = slab ? p->per_sample == 1 : S == 1 && period == all;
  // (a walk row that is the sample has its S positions, one that is a period as many as fit)
  p->reps = slab ? p->per_sample : rows == 1 && period == all ? int(S) : int(p->per_sample * period * vw / C);
  p->threads = (p->phases * p->cf + 31) / 32 * 32;
  p->nv = pow2_at_least((rows + p->per_sample - 1) / p->per_sample);
  p->items = (N + p->samples - 1) / p->samples;
  p->grid_items = p->items;
  return p->items <= INT_MAX;
}

// The token form applies: S = 1, aligned, and a group is up to nv_max fragments on each of 32 lanes.
bool token_plan(int vw, int64_t N, int64_t S, int64_t C, int64_t G, int nv_max, TokenPlan* p) {
  const int64_t D = C / G, frags = D / vw;
  if (S != 1 || D % vw != 0 || frags > 32 * nv_max) return false;
  p->set = int(std::min<int64_t>(32, pow2_at_least(frags)));
  p->log_set = __builtin_ctz(unsigned(p->set));
  p->nv = pow2_at_least((frags + 31) / 32);
  const int64_t most_groups = kWalkThreads / p->set;
  p->tiles = int((G + most_groups - 1) / most_groups);
  p->cols = int((G + p->tiles - 1) / p->tiles) * p->set;
  p->rows = int(std::max<int64_t>(1, std::min<int64_t>(kWalkThreads / p->cols, (N + kPlanSms - 1) / kPlanSms)));
  // about 1024 threads an SM
  const int threads = (p->cols * p->rows + 31) / 32 * 32;
  const int64_t most = std::max<int64_t>(1, int64_t(kPlanSms) * (1024 / threads) / p->tiles);
  p->ctas = int(std::min((N + p->rows - 1) / p->rows, most));
  return true;
}

TokenDims token_dims(int64_t N, int64_t C, int64_t G, float eps, bool silu, bool pvec, const TokenPlan& p, int vw) {
  return TokenDims{N,   C,   int(G), int(C / G / vw), p.cols / p.set, eps, 1.0f / float(C / G), silu, pvec, p};
}

inline int token_threads(const TokenPlan& p) { return (p.cols * p.rows + 31) / 32 * 32; }

template <typename T>
cudaError_t token_fwd(const GroupNormArgs& a, const TokenDims& d, cudaStream_t stream, int* launches) {
  auto fn = d.p.nv == 1 ? k_gn_token<T, 1> : d.p.nv == 2 ? k_gn_token<T, 2> : d.p.nv == 4 ? k_gn_token<T, 4>
                                                                                          : k_gn_token<T, 8>;
  const cudaError_t e = launch(fn, dim3(unsigned(d.p.tiles * d.p.ctas)), dim3(token_threads(d.p)), 0, stream,
                               static_cast<const T*>(a.x), static_cast<const T*>(a.gamma),
                               static_cast<const T*>(a.beta), static_cast<T*>(a.y), a.mean, a.inv, d);
  if (e == cudaSuccess) *launches += 1;
  return e;
}

template <typename T>
cudaError_t token_grad(const GroupNormGradArgs& a, const TokenDims& d, float* cpart, cudaStream_t stream,
                       int* launches) {
  auto fn = d.p.nv == 1 ? k_gn_grad_token<T, 1> : d.p.nv == 2 ? k_gn_grad_token<T, 2> : k_gn_grad_token<T, 4>;
  cudaError_t e = launch(fn, dim3(unsigned(d.p.tiles * d.p.ctas)), dim3(token_threads(d.p)), 0, stream,
                         static_cast<const T*>(a.dy), static_cast<const T*>(a.x), static_cast<const T*>(a.gamma),
                         static_cast<const T*>(a.beta), a.mean, a.inv, static_cast<T*>(a.dx), cpart, d);
  if (e != cudaSuccess) return e;
  *launches += 1;
  if (cpart != nullptr) {
    const int64_t jobs = (d.C + 31) / 32 * 2;
    e = launch(k_channel_sums<T>, dim3(unsigned(jobs)), dim3(kSumsThreads), 0, stream, cpart, int64_t(d.p.ctas),
               int64_t(1), d.C, 2, static_cast<T*>(a.dbeta), static_cast<T*>(a.dgamma));
    if (e == cudaSuccess) *launches += 1;
  }
  return e;
}

// Shared memory: two sums for each entry, each column and each group (the gradient:
// an entry for every channel; MODE 2: and the channels' sums and gamma).
size_t fused_smem(const FusedPlan& p, int mode, int vw, int64_t G, bool grad) {
  const size_t slots = size_t(p.samples) * G, frags = size_t(p.phases) * p.cf;
  const size_t ents = 2 * frags * (grad || mode != 0 ? vw : 1);
  const size_t cols =
      p.direct ? 0 : 2 * size_t(p.samples) * (mode == 0 ? p.cf : p.W);
  const size_t channels = grad && mode == 2 ? 3 * size_t(p.W) : 0;
  return 4 * (ents + cols + 2 * slots + channels + (mode == 2 ? p.samples : 0));
}
// Two blocks an SM, or one where a block has more threads.
constexpr size_t smem_most(const FusedPlan& p) { return (p.threads > kMaxThreads ? 200 : 96) * 1024; }

// Blocks of more than 48 KB ask for it first.
template <typename... KArgs, typename... Args>
cudaError_t launch_fused(void (*fn)(KArgs...), unsigned blocks, int threads, size_t smem, cudaStream_t stream,
                         Args... args) {
  if (smem > 48 * 1024) {
    const cudaError_t e = allow_smem(reinterpret_cast<const void*>(fn));
    if (e != cudaSuccess) return e;
  }
  return launch(fn, dim3(blocks), dim3(threads), smem, stream, args...);
}

template <typename T, int MODE>
cudaError_t fused_fwd(const GroupNormArgs& a, const FusedDims& d, cudaStream_t stream, int* launches) {
  const FusedPlan& p = d.p;
  auto fn = p.threads > kMaxThreads ? k_gn_fused<T, 1, MODE, kWideThreads>
            : p.nv == 1             ? k_gn_fused<T, 1, MODE, kMaxThreads>
            : p.nv == 2             ? k_gn_fused<T, 2, MODE, kMaxThreads>
            : p.nv == 4             ? k_gn_fused<T, 4, MODE, kMaxThreads>
                                    : k_gn_fused<T, 8, MODE, kMaxThreads>;
  const cudaError_t e = launch_fused(fn, unsigned(p.items), p.threads,
                                     fused_smem(p, MODE, dev::Vec16<T>::N, a.G, false), stream,
                               static_cast<const T*>(a.x), static_cast<const T*>(a.gamma),
                               static_cast<const T*>(a.beta), static_cast<T*>(a.y), a.mean, a.inv, d);
  if (e == cudaSuccess) *launches += 1;
  return e;
}

template <typename T, int MODE>
cudaError_t fused_grad(const GroupNormGradArgs& a, const FusedDims& d, float* cpart, cudaStream_t stream,
                       int* launches) {
  const FusedPlan& p = d.p;
  auto fn = p.nv == 1   ? k_gn_grad_fused<T, 1, MODE, kMaxThreads>
            : p.nv == 2 ? k_gn_grad_fused<T, 2, MODE, kMaxThreads>
                        : k_gn_grad_fused<T, 4, MODE, kMaxThreads>;
  if constexpr (sizeof(T) == 4)
    if (p.threads > kMaxThreads) fn = k_gn_grad_fused<T, 1, MODE, kWideThreads>;
  cudaError_t e = launch_fused(fn, unsigned(p.grid_items), p.threads,
                               fused_smem(p, MODE, dev::Vec16<T>::N, a.G, true), stream, static_cast<const T*>(a.dy),
                         static_cast<const T*>(a.x), static_cast<const T*>(a.gamma), static_cast<const T*>(a.beta),
                         a.mean, a.inv, static_cast<T*>(a.dx), cpart, d);
  if (e != cudaSuccess) return e;
  *launches += 1;
  if (cpart != nullptr) {
    const int64_t jobs = (int64_t(d.C) + 31) / 32 * 2;
    // the sums of du are dbeta, those of du * h are dgamma
    e = launch(k_channel_sums<T>, dim3(unsigned(jobs)), dim3(kSumsThreads), 0, stream, cpart, p.grid_items,
               int64_t(1), int64_t(d.C), 2, static_cast<T*>(a.dbeta), static_cast<T*>(a.dgamma));
    if (e == cudaSuccess) *launches += 1;
  }
  return e;
}

inline unsigned misalign16(const void* p) { return unsigned(reinterpret_cast<uintptr_t>(p) & 15u); }

constexpr int kFwdNv = 8, kGradNv = 4;

// How fragments, channels and groups meet: see MODE above.
int mode_of(int vw, int64_t C, int64_t G, bool slab) { return !slab ? 2 : C / G % vw == 0 ? 0 : 1; }

bool fwd_plan(int vw, int64_t N, int64_t S, int64_t C, int64_t G, bool slab, FusedPlan* p) {
  return fused_plan(vw, N, S, C, slab, kFwdNv, p) &&
         fused_smem(*p, mode_of(vw, C, G, slab), vw, G, false) <= smem_most(*p);
}

bool grad_plan(int vw, int64_t N, int64_t S, int64_t C, int64_t G, bool slab, FusedPlan* p) {
  if (!fused_plan(vw, N, S, C, slab, kGradNv, p)) return false;
  // (8 values a thread do not fit the 64 registers of a wide block's threads: f16 3000x1x8160
  // 531 us, and 339 in the split form; f32 3000x1x2295 82, and 338)
  if (p->threads > kMaxThreads && vw != 4) return false;
  // items that run at a time: about 1024 threads an SM
  p->grid_items = std::min<int64_t>(p->items, kPlanSms * std::max(1, 1024 / p->threads));
  return fused_smem(*p, slab ? 1 : 2, vw, G, true) <= smem_most(*p);  // (mode 0 needs less)
}

}  // namespace

bool group_norm_fused_applies(DType t, int64_t N, int64_t S, int64_t C, int64_t G) {
  const int vw = t == DType::F32 ? 4 : 8;
  const bool slab = C % vw == 0;
  TokenPlan tp;
  FusedPlan p;
  return (slab && token_plan(vw, N, S, C, G, kFwdNv, &tp)) || fwd_plan(vw, N, S, C, G, slab, &p);
}

size_t group_norm_grad_fused_bytes(DType t, int64_t N, int64_t S, int64_t C, int64_t G, bool aligned, bool* applies) {
  const int vw = t == DType::F32 ? 4 : 8;
  const bool whole = C % vw == 0;
  size_t most = 0;
  *applies = false;
  TokenPlan tp;
  if (whole && token_plan(vw, N, S, C, G, kGradNv, &tp)) {
    *applies = true;
    most = size_t(tp.ctas) * size_t(C) * 8;
    if (aligned) return most;
  }
  for (int slab = 0; slab < 2; ++slab) {
    FusedPlan p;
    if ((!aligned || (slab != 0) == whole) && grad_plan(vw, N, S, C, G, slab != 0, &p)) {
      *applies = *applies || (slab != 0) == whole;
      most = std::max(most, size_t(p.grid_items) * size_t(C) * 8);
    }
  }
  return most;
}

cudaError_t launch_group_norm_fused(const GroupNormArgs& a, cudaStream_t stream, int* launches, bool* done) {
  const int vw = a.t == DType::F32 ? 4 : 8;
  const bool pvec = misalign16(a.gamma) == 0 && misalign16(a.beta) == 0;
  FusedDims d{a.N, a.S, a.S * a.C, int(a.C), int(a.G), int(a.C / a.G), a.eps, float(1.0 / (double(a.S) * double(a.C / a.G))), a.silu, pvec, {}};
  *done = false;
  if (misalign16(a.x) != misalign16(a.y)) return cudaSuccess;
  const bool slab = a.C % vw == 0 && misalign16(a.x) == 0;
  TokenPlan tp;
  if (slab && token_plan(vw, a.N, a.S, a.C, a.G, kFwdNv, &tp)) {
    *done = true;
    const TokenDims t = token_dims(a.N, a.C, a.G, a.eps, a.silu, pvec, tp, vw);
    switch (a.t) {
      case DType::F32: return token_fwd<float>(a, t, stream, launches);
      case DType::F16: return token_fwd<__half>(a, t, stream, launches);
      default: return token_fwd<__nv_bfloat16>(a, t, stream, launches);
    }
  }
  if (!fwd_plan(vw, a.N, a.S, a.C, a.G, slab, &d.p)) return cudaSuccess;
  const int mode = mode_of(vw, a.C, a.G, slab);
  *done = true;
#define EP_GN_FUSED(T)                                                          \
  (mode == 0   ? fused_fwd<T, 0>(a, d, stream, launches)                        \
   : mode == 1 ? fused_fwd<T, 1>(a, d, stream, launches)                        \
               : fused_fwd<T, 2>(a, d, stream, launches))
  switch (a.t) {
    case DType::F32: return EP_GN_FUSED(float);
    case DType::F16: return EP_GN_FUSED(__half);
    default: return EP_GN_FUSED(__nv_bfloat16);
  }
#undef EP_GN_FUSED
}

cudaError_t launch_group_norm_grad_fused(const GroupNormGradArgs& a, cudaStream_t stream, int* launches, bool* done) {
  const int vw = a.t == DType::F32 ? 4 : 8;
  const bool pvec = misalign16(a.gamma) == 0 && misalign16(a.beta) == 0;
  FusedDims d{a.N, a.S, a.S * a.C, int(a.C), int(a.G), int(a.C / a.G), 0.f, float(1.0 / (double(a.S) * double(a.C / a.G))), a.silu, pvec, {}};
  *done = false;
  if (misalign16(a.x) != misalign16(a.dy) || misalign16(a.x) != misalign16(a.dx)) return cudaSuccess;
  const bool slab = a.C % vw == 0 && misalign16(a.x) == 0;
  float* cpart = a.dgamma != nullptr || a.dbeta != nullptr ? static_cast<float*>(a.workspace) : nullptr;
  TokenPlan tp;
  if (slab && token_plan(vw, a.N, a.S, a.C, a.G, kGradNv, &tp)) {
    *done = true;
    const TokenDims t = token_dims(a.N, a.C, a.G, 0.f, a.silu, pvec, tp, vw);
    switch (a.t) {
      case DType::F32: return token_grad<float>(a, t, cpart, stream, launches);
      case DType::F16: return token_grad<__half>(a, t, cpart, stream, launches);
      default: return token_grad<__nv_bfloat16>(a, t, cpart, stream, launches);
    }
  }
  if (!grad_plan(vw, a.N, a.S, a.C, a.G, slab, &d.p)) return cudaSuccess;
  *done = true;
  const int mode = mode_of(vw, a.C, a.G, slab);
#define EP_GN_GRAD_FUSED(T)                                                     \
  (mode == 0   ? fused_grad<T, 0>(a, d, cpart, stream, launches)                \
   : mode == 1 ? fused_grad<T, 1>(a, d, cpart, stream, launches)                \
               : fused_grad<T, 2>(a, d, cpart, stream, launches))
  switch (a.t) {
    case DType::F32: return EP_GN_GRAD_FUSED(float);
    case DType::F16: return EP_GN_GRAD_FUSED(__half);
    default: return EP_GN_GRAD_FUSED(__nv_bfloat16);
  }
#undef EP_GN_GRAD_FUSED
}

}  // namespace ep

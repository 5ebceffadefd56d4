// GroupNorm and its gradient with the sample on chip: x (and dy) are read once,
// into registers, and the result is written from there.  One launch for the
// forward pass, no scratch.  The definitions stand in group_norm.cu.
//
// A block holds walk rows of `cf` fragments, one thread to a fragment column, so
// a thread's channels stay the same:
//   MODE 0  C % VW == 0 and D % VW == 0: a walk row is a row of a slab of W
//           channels (whole groups), and a fragment lies in one group;
//   MODE 1  C % VW == 0, any D: the same slabs, sums for each channel;
//   MODE 2  any C and alignment: a walk row is the C / gcd(C, VW) fragments after
//           which channels repeat (column_walk.cuh), over the whole sample; the
//           first and the last fragment of a sample may be partial.
// `phases` walk rows lie side by side in a block, `per_sample` of them in one
// sample; each thread has up to NV rows.  Small samples share a block; a large
// one is spread over the CTAs of a cluster, each with its range of rows, whose
// group sums meet in distributed shared memory.
//
// Statistics: values are taken relative to their group's first value, summed,
// and the squares of their distances from the block's mean of the group summed
// in a second pass over the registers; a cluster's blocks are joined with Chan's
// formula.  All in float32, in an order that does not depend on timing.
//
// What bounds it: small samples, the latency of load, two block reductions and
// store; large batches, DRAM.
#include <cstdlib>
#include <algorithm>
#include <climits>
#include <numeric>
#include <type_traits>

#include "column_walk.cuh"
#include "device_common.cuh"
#include "ep_internal.h"
#include "group_norm.cuh"
#include "launch_util.h"

namespace ep {
namespace {

constexpr int kMaxThreads = 512;
constexpr int kMaxCluster = 16;

struct FusedPlan {
  int W;              // channels after which a walk row repeats: a slab's, or C
  int cf;             // fragments of a walk row
  int slabs;          // C / W
  int q;              // groups in a slab
  int phases, per_sample, samples;  // walk rows side by side, of one sample, samples in a block
  int threads, nv, cluster;
  int rows, rows_per_cta;           // walk rows of a sample; of one CTA
  int64_t items;      // blocks of samples x slabs, each `cluster` CTAs
  int64_t grid_items; // items running at a time (the gradient; forward: all)
};

struct FusedDims {
  int64_t N, S, L;
  int C, G, D;
  float eps;
  bool silu;
  bool pvec;          // gamma and beta 16-byte aligned
  FusedPlan p;
};

// Where a thread stands in an item.
template <typename T, int MODE>
struct Place {
  static constexpr int VW = dev::Vec16<T>::N;
  int64_t n;       // its sample
  int64_t e0;      // its first fragment's first element, from the sample's (slab's) start
  int64_t stride;  // elements from one of its fragments to the next
  int64_t lim;     // MODE 2: elements of the sample
  int off;
  int kn;          // its fragments
  int slab;

  __device__ __forceinline__ Place(const FusedDims& d, const T* x, unsigned item, int rank, int trow, int tcol,
                                   int ns) {
    const FusedPlan& p = d.p;
    const unsigned block = p.slabs == 1 ? item : item / unsigned(p.slabs);
    slab = static_cast<int>(item - block * unsigned(p.slabs));
    const int ph = trow - ns * p.per_sample;
    n = int64_t(block) * p.samples + ns;
    const bool live = trow < p.phases && n < d.N;
    off = MODE == 2 && live ? dev::misalignment(x + n * d.L) : 0;
    const int64_t row = MODE == 2 ? int64_t(p.cf) * VW : d.C;
    const int r0 = rank * p.rows_per_cta + ph, r1 = min(p.rows, (rank + 1) * p.rows_per_cta);
    kn = live && r0 < r1 ? (r1 - r0 + p.per_sample - 1) / p.per_sample : 0;
    e0 = r0 * row + tcol * VW - off;
    stride = p.per_sample * row;
    lim = d.L;
  }
  __device__ __forceinline__ bool whole(int k) const {
    return MODE != 2 || (e0 + k * stride >= 0 && e0 + k * stride + VW <= lim);
  }
  __device__ __forceinline__ bool inside(int k, int e) const {
    return MODE != 2 || (e0 + k * stride + e >= 0 && e0 + k * stride + e < lim);
  }
  __device__ __forceinline__ uint4 load(const T* base, int k) const {
    const int64_t at = e0 + k * stride;
    if (whole(k)) return dev::ld16_stream(base + at);
    float v[VW];
    dev::load_frag<T, false>(base, at, lim, v);
    return dev::Conv<T>::pack(v);  // exact: the values are T's
  }
  __device__ __forceinline__ void store(T* base, int k, const float (&v)[VW]) const {
    const int64_t at = e0 + k * stride;
    if (whole(k)) dev::st16_stream(base + at, dev::Conv<T>::pack(v));
    else dev::store_frag<T, false>(base, at, lim, v);
  }
};

__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
}

// 16 bytes at this shared-memory address in the cluster's block `rank`.
__device__ __forceinline__ float4 ld_rank(const float4* p, int rank) {
  uint32_t a = static_cast<uint32_t>(__cvta_generic_to_shared(p));
  float4 v;
  asm volatile("mapa.shared::cluster.u32 %0, %0, %1;" : "+r"(a) : "r"(rank));
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(a) : "memory");
  return v;
}

// Sums over the entries of each (sample, group) of a block, in two steps: over
// the repeats of each column (fragments in MODE 0, else channels), then over a
// group's columns.  Entries are floats by position; column c of sample ns is at
// off + c + k Cw, modulo the np positions of a sample (the positions before
// `off` hold the channels that the last repeat misses).
struct Entries {
  int De, Cw, np, reps, q, slots, cols;
  __device__ __forceinline__ Entries(const FusedPlan& p, int D, int VW, bool frags) {
    De = frags ? D / VW : D;
    Cw = frags ? p.cf : p.W;
    np = p.per_sample * p.cf * (frags ? 1 : VW);
    reps = static_cast<int>(unsigned(np) / unsigned(Cw));
    q = p.q;
    slots = p.samples * p.q;
    cols = p.samples * Cw;
  }
  __device__ __forceinline__ int sample_of(int slot) const {
    return slots == q ? 0 : static_cast<int>(unsigned(slot) / unsigned(q));
  }
  // add(position, a, b) for each entry; col_a (and col_b): a float a column;
  // done(slot, sample, a, b) by one lane.  `plain`: one repeat and no offset, so
  // that entries are columns already.
  template <bool PAIR, typename OFF, typename ADD, typename DONE>
  __device__ __forceinline__ void run(const float* ent_a, const float* ent_b, float* col_a, float* col_b, bool plain,
                                      OFF off_of, ADD add, DONE done) const {
    const float* ca = ent_a;
    const float* cb = ent_b;
    if (!plain) {
      sum_sets(blockDim.x, cols, reps,
               [&](int i, int k, float& a, float& b) {
                 const int ns = cols == Cw ? 0 : static_cast<int>(unsigned(i) / unsigned(Cw));
                 int pos = off_of(ns) + (i - ns * Cw) + k * Cw;
                 if (pos >= np) pos -= np;
                 add(ns * np + pos, a, b);
               },
               [&](int i, float a, float b) {
                 col_a[i] = a;
                 if constexpr (PAIR) col_b[i] = b;
               });
      __syncthreads();
      ca = col_a;
      cb = col_b;
    }
    sum_sets(blockDim.x, slots, De,
             [&](int s, int k, float& a, float& b) {  // (sample ns, group g: columns ns Cw + g De + k)
               a += ca[s * De + k];
               if constexpr (PAIR) b += cb[s * De + k];
             },
             [&](int s, float a, float b) { done(s, sample_of(s), a, b); });
  }
};

// gamma and beta of VW channels from c on (modulo W), which start at `from`.
template <typename T, bool WRAP>
__device__ __forceinline__ void load_params(const T* __restrict__ gamma, const T* __restrict__ beta, int from, int c,
                                            int W, bool vec, float (&a)[dev::Vec16<T>::N],
                                            float (&b)[dev::Vec16<T>::N]) {
  constexpr int VW = dev::Vec16<T>::N;
#pragma unroll
  for (int e = 0; e < VW; ++e) b[e] = 0.f;
  if (!WRAP && vec) {
    dev::Conv<T>::unpack(dev::ld16_keep(gamma + from + c), a);
    if (beta != nullptr) dev::Conv<T>::unpack(dev::ld16_keep(beta + from + c), b);
  } else {
#pragma unroll
    for (int e = 0; e < VW; ++e) {
      a[e] = dev::ld1_keep(gamma + from + c);
      if (beta != nullptr) b[e] = dev::ld1_keep(beta + from + c);
      if (++c == W) c = 0;
    }
  }
}

// Joins the cluster's values of each slot: f(slot, lane's rank value or 0).
template <typename F>
__device__ __forceinline__ void for_slots_by_rank(int slots, int cluster, F f) {
  const int sets = blockDim.x / cluster;  // the cluster size is a power of two up to 16
  for (int s0 = 0; s0 < slots; s0 += sets) f(s0 + int(threadIdx.x) / cluster, int(threadIdx.x) & (cluster - 1));
}
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

// A thread's sums of its values' distances from a centre, or of their squares.
template <typename T, int NV, int MODE, bool SQUARE>
__device__ __forceinline__ void centred_sums(const uint4 (&raw)[NV], const Place<T, MODE>& at,
                                             const float (&c)[MODE == 0 ? 1 : dev::Vec16<T>::N],
                                             float (&s)[MODE == 0 ? 1 : dev::Vec16<T>::N]) {
  constexpr int VW = dev::Vec16<T>::N;
#pragma unroll
  for (int e = 0; e < (MODE == 0 ? 1 : VW); ++e) s[e] = 0.f;
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
      if constexpr (MODE == 0) {
        float a[2] = {0.f, 0.f};
#pragma unroll
        for (int e = 0; e < VW; ++e) a[e & 1] = SQUARE ? fmaf(v[e], v[e], a[e & 1]) : a[e & 1] + v[e];
        s[0] += a[0] + a[1];
      } else {
#pragma unroll
        for (int e = 0; e < VW; ++e) s[e] = SQUARE ? fmaf(v[e], v[e], s[e]) : s[e] + v[e];
      }
    }
  }
}

template <typename T, int NV, int MODE>
__global__ void __launch_bounds__(kMaxThreads)
k_gn_fused(const T* x, const T* __restrict__ gamma, const T* __restrict__ beta, T* y, float* mean_out,
           float* inv_out, FusedDims d) {
  constexpr int VW = dev::Vec16<T>::N;
  constexpr int EV = MODE == 0 ? 1 : VW;  // entries of a thread
  extern __shared__ __align__(16) float smem[];
  const FusedPlan& p = d.p;
  const int slots = p.samples * p.q, ents = p.phases * p.cf * EV;
  float4* xch = reinterpret_cast<float4*>(smem);                 // (count, mean, M2) for the cluster
  float* ent = smem + (p.cluster > 1 ? 4 * slots : 0);
  float* cnt = ent + ents;                                       // MODE 2: valid values behind each entry
  float* col = cnt + (MODE == 2 ? ents : 0);                     // sums by column, and their counts
  const int cols = p.samples * (MODE == 0 ? p.cf : p.W);
  float* col_n = col + cols;
  float* gk = col_n + (MODE == 2 ? cols : 0);                    // the group's first value
  float* gm = gk + slots;
  float* gr = gm + slots;
  const int rank = blockIdx.x & (p.cluster - 1);
  const unsigned item = blockIdx.x / unsigned(p.cluster);
  const int trow = threadIdx.x / unsigned(p.cf), tcol = threadIdx.x - trow * p.cf;
  const int ns = p.samples == 1 ? 0 : trow / unsigned(p.per_sample);
  dev::pdl_wait();
  dev::pdl_trigger();

  const Place<T, MODE> at(d, x, item, rank, trow, tcol, ns);
  const T* xs = x + (at.kn > 0 ? at.n * d.L + int64_t(at.slab) * p.W : 0);
  uint4 raw[NV];
#pragma unroll
  for (int k = 0; k < NV; ++k)
    if (k < at.kn) raw[k] = at.load(xs, k);

  // this thread's channels (within the slab), groups and shifts
  int c0 = MODE == 2 ? (tcol * VW + p.W - at.off % p.W) % p.W : tcol * VW;
  int grp[EV];
  float shift[EV];
  for_channels<VW>(c0, p.W, d.D, [&](int e, int, int g) {
    if (e < EV) {
      grp[e] = ns * p.q + g;
      shift[e] = at.kn > 0 ? dev::ld1_stream(xs + g * d.D) : 0.f;
    }
  });

  const bool mine = trow < p.phases;
  const Entries entries(p, d.D, VW, MODE == 0);
  const bool plain = MODE != 2 && entries.reps == 1;
  const int64_t n0 = int64_t(p.slabs == 1 ? item : item / unsigned(p.slabs)) * p.samples;
  auto off_of = [&](int s) {
    return MODE == 2 && n0 + s < d.N ? dev::misalignment(x + (n0 + s) * d.L) : 0;
  };
  // values of a group in this CTA
  const int my_rows = max(0, min(p.rows, (rank + 1) * p.rows_per_cta) - rank * p.rows_per_cta);
  const float count = MODE == 2 ? float(d.S) * float(d.D) : float(my_rows) * float(d.D);

  float m[EV], s[EV];
  centred_sums<T, NV, MODE, false>(raw, at, shift, s);
  if (mine) {
    put_entries(ent, s);
    if constexpr (MODE == 2) {
#pragma unroll
      for (int e = 0; e < EV; ++e) m[e] = 0.f;
#pragma unroll
      for (int k = 0; k < NV; ++k) {
        if (k < at.kn) {
#pragma unroll
          for (int e = 0; e < EV; ++e) m[e] += at.inside(k, e) ? 1.f : 0.f;
        }
      }
      put_entries(cnt, m);
    }
  }
  __syncthreads();
  entries.run<MODE == 2>(
             ent, cnt, col, col_n, plain, off_of,
             [&](int i, float& a, float& b) {
               a += ent[i];
               if constexpr (MODE == 2) b += cnt[i];
             },
             [&](int s, int ns, float a, float b) {
               const float n = MODE == 2 ? b : count;
               const int g = s - ns * p.q;
               const int64_t sample = n0 + ns;
               const float first =
                   sample < d.N ? dev::ld1_stream(x + sample * d.L + int64_t(at.slab) * p.W + g * d.D) : 0.f;
               const float mean = n > 0.f ? a / n : 0.f;
               const float centre = first + mean;
               // the centre is rounded: it lies by `by` off the mean, which adds n by^2 to the squares
               const float by = mean - (centre - first);
               gk[s] = first;
               gm[s] = centre;
               gr[s] = n * by * by;
               if (p.cluster > 1) xch[s] = make_float4(n, mean, 0.f, 0.f);
             });
  __syncthreads();
#pragma unroll
  for (int e = 0; e < EV; ++e) m[e] = mine ? gm[grp[e]] : 0.f;
  centred_sums<T, NV, MODE, true>(raw, at, m, s);
  if (mine) {
    put_entries(ent, s);
  }
  __syncthreads();
  const float total = float(d.S) * float(d.D);
  auto finish = [&](int s, int ns, float mu, float m2) {
    const float r = 1.0f / sqrtf(not_negative(m2) / total + d.eps);
    gm[s] = mu;
    gr[s] = r;
    const int64_t sample = n0 + ns;
    if (rank == 0 && sample < d.N) {
      const int64_t i = sample * d.G + int64_t(at.slab) * p.q + (s - ns * p.q);
      if (mean_out != nullptr) mean_out[i] = mu;
      if (inv_out != nullptr) inv_out[i] = r;
    }
  };
  entries.run<false>(
             ent, cnt, col, col_n, plain, off_of, [&](int i, float& a, float&) { a += ent[i]; },
             [&](int s, int ns, float a, float) {
               if (p.cluster == 1) finish(s, ns, gm[s], a - gr[s]);
               else xch[s].z = not_negative(a - gr[s]);
             });
  if (p.cluster > 1) {
    cluster_sync();
    for_slots_by_rank(slots, p.cluster, [&](int s, int r) {
      const float4 v = s < slots ? ld_rank(xch + s, r) : make_float4(0.f, 0.f, 0.f, 0.f);
      const float mean = set_sum(v.x * v.y, p.cluster) / total;
      const float t = v.y - mean;
      const float m2 = set_sum(v.z + v.x * t * t, p.cluster);
      if (s < slots && r == 0) finish(s, 0, gk[s] + mean, m2);
    });
    cluster_sync();  // no block leaves (or overwrites x) while another reads its sums
  } else {
    __syncthreads();
  }

  // y
  float mu[EV], rs[EV], a[VW], b[VW];
#pragma unroll
  for (int e = 0; e < EV; ++e) {
    mu[e] = mine ? gm[grp[e]] : 0.f;
    rs[e] = mine ? gr[grp[e]] : 0.f;
  }
  if (at.kn > 0) {
    const int cs = at.slab * p.W;
    load_params<T, MODE == 2>(gamma, beta, cs, c0, p.W, d.pvec, a, b);
#pragma unroll
    for (int e = 0; e < VW; ++e) a[e] *= rs[MODE == 0 ? 0 : e];
    T* ys = y + at.n * d.L + cs;
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

// The gradient.  A CTA takes items in turn (grid_items apart), all of one slab,
// and keeps the sums of du and du * h of its channels over them in registers;
// they leave once, as row (item index * cluster + rank) of cpart: 2 x [row][C].
// The groups' means m1 and m2 of an item meet as the forward's sums do.
template <typename T, int NV, int MODE>
__global__ void __launch_bounds__(kMaxThreads)
k_gn_grad_fused(const T* dy, const T* x, const T* __restrict__ gamma, const T* __restrict__ beta, const float* mean,
                const float* inv, T* dx, float* cpart, FusedDims d) {
  constexpr int VW = dev::Vec16<T>::N;
  constexpr int EV = MODE == 0 ? 1 : VW;
  extern __shared__ __align__(16) float smem[];
  const FusedPlan& p = d.p;
  const int slots = p.samples * p.q, ents = p.phases * p.cf * VW;
  float4* xch = reinterpret_cast<float4*>(smem);
  float* ent_a = smem + (p.cluster > 1 ? 4 * slots : 0);
  float* ent_b = ent_a + ents;
  const int cols = p.samples * (MODE == 0 ? p.cf : p.W);
  float* col_a = ent_b + ents;
  float* col_b = col_a + cols;
  float* g1 = col_b + cols;
  float* g2 = g1 + slots;
  const int rank = blockIdx.x & (p.cluster - 1);
  const unsigned first = blockIdx.x / unsigned(p.cluster);
  const int trow = threadIdx.x / unsigned(p.cf), tcol = threadIdx.x - trow * p.cf;
  const int ns = p.samples == 1 ? 0 : trow / unsigned(p.per_sample);
  const bool mine = trow < p.phases;
  const float scale = 1.0f / (float(d.S) * float(d.D));
  const Entries entries(p, d.D, VW, MODE == 0);
  dev::pdl_wait();
  dev::pdl_trigger();

  float tot_a[VW], tot_b[VW], ga[VW], be[VW];
  int grp[EV];  // within the slab
#pragma unroll
  for (int e = 0; e < VW; ++e) tot_a[e] = tot_b[e] = ga[e] = be[e] = 0.f;
  int off = 0, c0 = 0, slab = 0;
  bool once = true;

  for (unsigned item = first; item < unsigned(p.items); item += unsigned(p.grid_items)) {
    const Place<T, MODE> at(d, x, item, rank, trow, tcol, ns);
    const int64_t base = at.kn > 0 ? at.n * d.L + int64_t(at.slab) * p.W : 0;
    uint4 raw[NV], rdy[NV];
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      if (k < at.kn) {
        raw[k] = at.load(x + base, k);
        rdy[k] = at.load(dy + base, k);
      }
    }
    if (once) {  // the items of a CTA share their slab, and (MODE 2) their offset
      once = false;
      slab = at.slab;
      if constexpr (MODE == 2) {
        off = dev::misalignment(x + int64_t(item) * p.samples * d.L);
      }
      c0 = MODE == 2 ? (tcol * VW + p.W - off % p.W) % p.W : tcol * VW;
      if (mine) load_params<T, MODE == 2>(gamma, beta, slab * p.W, c0, p.W, d.pvec, ga, be);
      for_channels<VW>(c0, p.W, d.D, [&](int e, int, int g) {
        if (e < EV) grp[e] = g;
      });
    }
    float mu[EV], rs[EV];
    const int64_t ng = at.n * d.G + int64_t(slab) * p.q;
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
      } else {
        float a[VW], b[VW];
#pragma unroll
        for (int e = 0; e < VW; ++e) {
          a[e] = sa[e] * ga[e];
          b[e] = sb[e] * ga[e];
        }
        put_entries(ent_a, a);
        put_entries(ent_b, b);
      }
      dev::add_pairs(tot_a, sa);
      dev::add_pairs(tot_b, sb);
    }
    __syncthreads();
    entries.run<true>(
               ent_a, ent_b, col_a, col_b, MODE != 2 && entries.reps == 1, [&](int) { return off; },
               [&](int i, float& a, float& b) {
                 a += ent_a[i];
                 b += ent_b[i];
               },
               [&](int s, int, float a, float b) {
                 if (p.cluster == 1) {
                   g1[s] = a * scale;
                   g2[s] = b * scale;
                 } else {
                   xch[s] = make_float4(a, b, 0.f, 0.f);
                 }
               });
    if (p.cluster > 1) {
      cluster_sync();
      for_slots_by_rank(slots, p.cluster, [&](int s, int r) {
        const float4 v = s < slots ? ld_rank(xch + s, r) : make_float4(0.f, 0.f, 0.f, 0.f);
        const float a = set_sum(v.x, p.cluster), b = set_sum(v.y, p.cluster);
        if (s < slots && r == 0) {
          g1[s] = a * scale;
          g2[s] = b * scale;
        }
      });
      cluster_sync();  // the next item's sums go to the same place
    } else {
      __syncthreads();
    }
    if (at.kn > 0) {
      float a1[EV], a2[EV];
#pragma unroll
      for (int e = 0; e < EV; ++e) {
        a1[e] = g1[ns * p.q + grp[e]];
        a2[e] = g2[ns * p.q + grp[e]];
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
  if (mine) {
    put_entries(ent_a, tot_a);
    put_entries(ent_b, tot_b);
  }
  __syncthreads();
  // channel c is at off + c + k W, modulo a sample's positions, in every sample
  const int np = p.per_sample * p.cf * VW, reps = np / p.W;
  const int64_t rows = p.grid_items / p.slabs * p.cluster;
  const int64_t row = (first / p.slabs) * p.cluster + rank;
  const int many = reps * p.samples;
  const int set = many >= 32 ? 32 : 1;  // lanes to a channel
  for (int c = threadIdx.x / set; c < p.W; c += blockDim.x / set) {
    float a = 0.f, b = 0.f;
    for (int i = threadIdx.x & (set - 1); i < many; i += set) {
      const int k = i % reps;
      int pos = off + c + k * p.W;
      if (pos >= np) pos -= np;
      pos += i / reps * np;
      a += ent_a[pos];
      b += ent_b[pos];
    }
    if (set == 32) {  // (a warp's lanes share c)
      a = dev::warp_sum(a);
      b = dev::warp_sum(b);
    }
    if ((threadIdx.x & (set - 1)) == 0) {
      float* out = cpart + row * d.C + slab * p.W + c;
      out[0] = a;
      out[rows * d.C] = b;
    }
  }
}

// ---------------------------------------------------------------------------
// One position a sample (S = 1), D / VW a power of two up to 32: the norm over
// each token's groups.  A group's fragments are neighbouring lanes, so its sums
// are shuffles and there is no shared memory and no barrier.  A block has `cols`
// fragment columns of a tile and `rows` tokens side by side; it takes every
// grid-th set of tokens, so its channels (and parameters) stay the same.  U
// tokens are loaded before the first is used.
// ---------------------------------------------------------------------------

struct TokenPlan {
  int cols, rows, tiles, ctas;  // ctas: of each tile
};

struct TokenDims {
  int64_t N, C;
  int G, set;                   // lanes of a group
  float eps, scale;             // scale: 1 / D
  bool silu, pvec;
  TokenPlan p;
};

template <typename T>
__global__ void __launch_bounds__(kWalkThreads)
k_gn_token(const T* x, const T* __restrict__ gamma, const T* __restrict__ beta, T* y, float* mean_out,
           float* inv_out, TokenDims d) {
  constexpr int VW = dev::Vec16<T>::N;
  constexpr int U = 4;
  dev::pdl_wait();
  dev::pdl_trigger();
  const int trow = threadIdx.x / unsigned(d.p.cols), tile = blockIdx.x % unsigned(d.p.tiles);
  const int col = tile * d.p.cols + (threadIdx.x - trow * d.p.cols);  // of fragments
  const int lead = (threadIdx.x & 31) & ~(d.set - 1);
  const bool mine = trow < d.p.rows && col * VW < d.C;  // uniform in a set
  const int64_t step = int64_t(d.p.ctas) * d.p.rows, n1 = d.N;
  int64_t n = int64_t(blockIdx.x / unsigned(d.p.tiles)) * d.p.rows + trow;
  float a[VW], b[VW];
  if (mine) load_params<T, false>(gamma, beta, 0, col * VW, 0, d.pvec, a, b);
  // every lane of a warp goes round as often as its first (the shuffles are whole warps')
  const int rounds = static_cast<int>((n1 - (int64_t(blockIdx.x / unsigned(d.p.tiles)) * d.p.rows) + step * U - 1) /
                                      (step * U));
  for (int i = 0; i < rounds; ++i, n += step * U) {
    uint4 raw[U];
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (mine && n + u * step < n1) raw[u] = dev::ld16_stream(x + (n + u * step) * d.C + col * VW);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const bool on = mine && n + u * step < n1;
      float v[VW];
      if (on) {
        dev::Conv<T>::unpack(raw[u], v);
      } else {
#pragma unroll
        for (int e = 0; e < VW; ++e) v[e] = 0.f;
      }
      const float first = __shfl_sync(0xffffffffu, v[0], lead);
      float s = 0.f, q = 0.f;
#pragma unroll
      for (int e = 0; e < VW; ++e) s += v[e] - first;
      const float m = set_sum(s, d.set) * d.scale;
      const float mu = first + m, by = m - (mu - first);
#pragma unroll
      for (int e = 0; e < VW; ++e) {
        v[e] -= mu;
        q = fmaf(v[e], v[e], q);
      }
      q = set_sum(q, d.set) * d.scale;  // relative to mu, which is rounded: `by` off the mean
      const float r = 1.0f / sqrtf(not_negative(q - by * by) + d.eps);
      if (on) {
#pragma unroll
        for (int e = 0; e < VW; ++e) {
          v[e] = fmaf(v[e], a[e] * r, b[e]);
          if (d.silu) v[e] = silu<T>(v[e]);
        }
        const int64_t t = n + u * step;
        dev::st16_stream(y + t * d.C + col * VW, dev::Conv<T>::pack(v));
        if ((threadIdx.x & 31) == lead) {
          const int64_t g = t * d.G + col / d.set;
          if (mean_out != nullptr) mean_out[g] = mu;
          if (inv_out != nullptr) inv_out[g] = r;
        }
      }
    }
  }
}

// The gradient; the sums for dgamma and dbeta run on in registers and leave as
// row blockIdx / tiles of cpart: 2 x [ctas][C].
template <typename T>
__global__ void __launch_bounds__(kWalkThreads)
k_gn_grad_token(const T* dy, const T* x, const T* __restrict__ gamma, const T* __restrict__ beta, const float* mean,
                const float* inv, T* dx, float* cpart, TokenDims d) {
  constexpr int VW = dev::Vec16<T>::N;
  constexpr int U = 2;
  __shared__ float s_a[kWalkThreads * VW], s_b[kWalkThreads * VW];
  dev::pdl_wait();
  dev::pdl_trigger();
  const int trow = threadIdx.x / unsigned(d.p.cols), tile = blockIdx.x % unsigned(d.p.tiles);
  const int row = blockIdx.x / unsigned(d.p.tiles);
  const int col = tile * d.p.cols + (threadIdx.x - trow * d.p.cols);
  const bool mine = trow < d.p.rows && col * VW < d.C;
  const int64_t step = int64_t(d.p.ctas) * d.p.rows, n1 = d.N;
  int64_t n = int64_t(row) * d.p.rows + trow;
  float ga[VW], be[VW], tot_a[VW], tot_b[VW];
#pragma unroll
  for (int e = 0; e < VW; ++e) ga[e] = be[e] = tot_a[e] = tot_b[e] = 0.f;
  if (mine) load_params<T, false>(gamma, beta, 0, col * VW, 0, d.pvec, ga, be);
  const int rounds = static_cast<int>((n1 - int64_t(row) * d.p.rows + step * U - 1) / (step * U));
  for (int i = 0; i < rounds; ++i, n += step * U) {
    uint4 rx[U], rd[U];
    float mu[U], rs[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t t = n + u * step;
      if (mine && t < n1) {
        rx[u] = dev::ld16_stream(x + t * d.C + col * VW);
        rd[u] = dev::ld16_stream(dy + t * d.C + col * VW);
        mu[u] = mean[t * d.G + col / d.set];
        rs[u] = inv[t * d.G + col / d.set];
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t t = n + u * step;
      const bool on = mine && t < n1;
      float h[VW], w[VW], p = 0.f, q = 0.f;
      if (on) {
        dev::Conv<T>::unpack(rx[u], h);
        dev::Conv<T>::unpack(rd[u], w);
#pragma unroll
        for (int e = 0; e < VW; ++e) {
          h[e] = (h[e] - mu[u]) * rs[u];
          if (d.silu) w[e] = silu_grad<T>(w[e], fmaf(h[e], ga[e], be[e]));
          tot_a[e] += w[e];
          tot_b[e] = fmaf(w[e], h[e], tot_b[e]);
          w[e] *= ga[e];
          p += w[e];
          q = fmaf(w[e], h[e], q);
        }
      }
      p = set_sum(p, d.set) * d.scale;
      q = set_sum(q, d.set) * d.scale;
      if (on) {
#pragma unroll
        for (int e = 0; e < VW; ++e) w[e] = rs[u] * ((w[e] - p) - h[e] * q);
        dev::st16_stream(dx + t * d.C + col * VW, dev::Conv<T>::pack(w));
      }
    }
  }
  if (cpart == nullptr) return;
#pragma unroll
  for (int e = 0; e < VW; ++e) {
    s_a[threadIdx.x * VW + e] = tot_a[e];
    s_b[threadIdx.x * VW + e] = tot_b[e];
  }
  __syncthreads();
  const int W = d.p.cols * VW;
  for (int c = threadIdx.x; c < W && tile * W + c < d.C; c += blockDim.x) {
    float sa = 0.f, sb = 0.f;
    for (int k = 0; k < d.p.rows; ++k) {
      sa += s_a[k * W + c];
      sb += s_b[k * W + c];
    }
    float* out = cpart + int64_t(row) * d.C + tile * W + c;
    out[0] = sa;
    out[int64_t(d.p.ctas) * d.C] = sb;
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

// Splits the rows of a sample (cf fragments each) over threads and CTAs: false
// if `nv_max` fragments a thread do not hold it.
bool split_rows(FusedPlan* p, int64_t N, int64_t rows, int nv_max) {
  if (p->cf > kMaxThreads || rows > INT_MAX / 2) return false;
  p->rows = int(rows);
  const int64_t frags = rows * p->cf;
  if (frags <= 4 * kWalkThreads) {
    // a small sample: one CTA, about 256 threads, with other samples where there
    // are enough of them (and two fragments a thread where one sample fills it)
    int phases = std::max(1, kWalkThreads / p->cf);
    p->per_sample = int(std::min<int64_t>(rows, phases));
    while ((rows + p->per_sample - 1) / p->per_sample > nv_max && p->cf * (p->per_sample + 1) <= kMaxThreads)
      p->per_sample += 1;
    if ((rows + p->per_sample - 1) / p->per_sample > nv_max) return false;
    const int64_t fit = std::max(1, phases / p->per_sample);
    p->samples = int(std::max<int64_t>(1, std::min(fit, N * p->slabs / (2 * kPlanSms))));
    p->phases = p->samples * p->per_sample;
    p->cluster = 1;
    p->rows_per_cta = int(rows);
  } else {
    const int most = kMaxThreads / p->cf;  // rows side by side
    static const int kMaxCluster = getenv("EPX_MAXK") ? atoi(getenv("EPX_MAXK")) : 16;
    if (kMaxCluster == 0) return false;
    int64_t per = rows;
    int k = 1;
    while (k < kMaxCluster && ((per = (rows + k - 1) / k) + most - 1) / most > nv_max) k *= 2;
    while (k < kMaxCluster && N * p->slabs * k < kPlanSms && (rows + k - 1) / k > most) k *= 2;
    per = (rows + k - 1) / k;
    if ((per + most - 1) / most > nv_max) return false;
    p->cluster = k;
    p->rows_per_cta = int(per);
    p->per_sample = p->phases = int(std::min<int64_t>(per, most));
    p->samples = 1;
  }
  p->threads = (p->phases * p->cf + 31) / 32 * 32;
  const int need = (p->rows_per_cta + p->per_sample - 1) / p->per_sample;
  p->nv = pow2_at_least(need);
  p->items = (N + p->samples - 1) / p->samples * p->slabs;
  p->grid_items = p->items;
  return p->items * p->cluster <= INT_MAX;
}

// slab: C % vw == 0 and 16-byte-aligned operands; else the walk over whole samples.
bool fused_plan(int vw, int64_t N, int64_t S, int64_t C, int64_t G, bool slab, int nv_max, FusedPlan* p) {
  const int64_t D = C / G;
  if (!slab) {
    p->W = int(C);
    p->slabs = 1;
    p->q = int(G);
    const int64_t period = C / std::gcd(C, int64_t(vw));
    if (period > kMaxThreads) return false;
    p->cf = int(period);
    const int64_t total = (S * C + 2 * (vw - 1)) / vw;  // fragments, wherever a sample starts
    return split_rows(p, N, (total + period - 1) / period, nv_max);
  }
  if (C % vw != 0) return false;
  auto with = [&](int64_t q) {
    p->W = int(q * D);
    p->slabs = int(G / q);
    p->q = int(q);
    p->cf = int(q * D / vw);
    return split_rows(p, N, S, nv_max);
  };
  // a small sample stays in one piece, with contiguous rows
  if (C / vw <= kMaxThreads && S * (C / vw) <= 4 * kWalkThreads) return with(G);
  // else the narrowest slab of whole groups whose rows are 128 bytes or more
  for (int64_t q = 1; q <= G; ++q) {
    if (G % q != 0 || q * D % vw != 0) continue;
    if (q * D / vw > kMaxThreads) break;
    if (q * D / vw >= 8 || q == G) return with(q);
  }
  return false;
}

// The token form applies: S = 1, aligned, and a group is 1 to 32 (a power of two) lanes.
bool token_plan(int vw, int64_t N, int64_t S, int64_t C, int64_t G, TokenPlan* p, int* set) {
  const int64_t D = C / G;
  if (S != 1 || D % vw != 0 || D / vw > 32 || (D / vw & (D / vw - 1)) != 0) return false;
  *set = int(D / vw);
  const int64_t frags = C / vw;
  p->tiles = int((frags + kWalkThreads - 1) / kWalkThreads);
  p->cols = int((frags / *set + p->tiles - 1) / p->tiles) * *set;  // whole groups
  p->rows = int(std::max<int64_t>(1, std::min<int64_t>(kWalkThreads / p->cols, (N + kPlanSms - 1) / kPlanSms)));
  // about 1024 threads an SM
  const int threads = (p->cols * p->rows + 31) / 32 * 32;
  const int64_t most = std::max<int64_t>(1, int64_t(kPlanSms) * (1024 / threads) / p->tiles);
  p->ctas = int(std::min((N + p->rows - 1) / p->rows, most));
  return true;
}

TokenDims token_dims(int64_t N, int64_t C, int64_t G, float eps, bool silu, bool pvec, const TokenPlan& p, int set) {
  return TokenDims{N, C, int(G), set, eps, 1.0f / float(C / G), silu, pvec, p};
}

inline int token_threads(const TokenPlan& p) { return (p.cols * p.rows + 31) / 32 * 32; }

template <typename T>
cudaError_t token_fwd(const GroupNormArgs& a, const TokenDims& d, cudaStream_t stream, int* launches) {
  const cudaError_t e = launch(k_gn_token<T>, dim3(unsigned(d.p.tiles * d.p.ctas)), dim3(token_threads(d.p)), 0, stream,
                               static_cast<const T*>(a.x), static_cast<const T*>(a.gamma),
                               static_cast<const T*>(a.beta), static_cast<T*>(a.y), a.mean, a.inv, d);
  if (e == cudaSuccess) *launches += 1;
  return e;
}

template <typename T>
cudaError_t token_grad(const GroupNormGradArgs& a, const TokenDims& d, float* cpart, cudaStream_t stream,
                       int* launches) {
  cudaError_t e = launch(k_gn_grad_token<T>, dim3(unsigned(d.p.tiles * d.p.ctas)), dim3(token_threads(d.p)), 0, stream,
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

template <typename... KArgs, typename... Args>
cudaError_t launch_cluster(void (*kernel)(KArgs...), unsigned grid, int threads, size_t smem, int cluster,
                           cudaStream_t stream, Args... args) {
  if (cluster > 8) {  // beyond the portable size
    const cudaError_t e = cudaFuncSetAttribute(reinterpret_cast<const void*>(kernel),
                                               cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e != cudaSuccess) return e;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = EP_PDL ? 1 : 0;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = unsigned(cluster);
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, static_cast<KArgs>(args)...);
}

// Shared memory: the cluster's exchange, the entries (MODE 2: and their counts;
// the gradient: two sets for every channel) and the groups' values.
size_t fused_smem(const FusedPlan& p, int mode, int vw, bool grad) {
  const size_t slots = size_t(p.samples) * p.q, frags = size_t(p.phases) * p.cf;
  const size_t ents = grad ? 2 * frags * vw : mode == 0 ? frags : frags * vw * (mode == 2 ? 2 : 1);
  const size_t cols = size_t(p.samples) * (mode == 0 ? p.cf : p.W) * (grad || mode == 2 ? 2 : 1);
  return 4 * (ents + cols + (p.cluster > 1 ? 4 * slots : 0) + (grad ? 2 : 3) * slots);
}
constexpr size_t kSmemMost = 48 * 1024;  // what a launch may have without opting in

template <typename T, int MODE>
cudaError_t fused_fwd(const GroupNormArgs& a, const FusedDims& d, cudaStream_t stream, int* launches) {
  const FusedPlan& p = d.p;
  auto fn = p.nv == 1   ? k_gn_fused<T, 1, MODE>
            : p.nv == 2 ? k_gn_fused<T, 2, MODE>
            : p.nv == 4 ? k_gn_fused<T, 4, MODE>
            : p.nv == 8 ? k_gn_fused<T, 8, MODE>
                        : k_gn_fused<T, 16, MODE>;
  const cudaError_t e = launch_cluster(
      fn, unsigned(p.items * p.cluster), p.threads, fused_smem(p, MODE, dev::Vec16<T>::N, false), p.cluster, stream,
      static_cast<const T*>(a.x), static_cast<const T*>(a.gamma), static_cast<const T*>(a.beta),
      static_cast<T*>(a.y), a.mean, a.inv, d);
  if (e == cudaSuccess) *launches += 1;
  return e;
}

template <typename T, int MODE>
cudaError_t fused_grad(const GroupNormGradArgs& a, const FusedDims& d, float* cpart, cudaStream_t stream,
                       int* launches) {
  const FusedPlan& p = d.p;
  auto fn = p.nv == 1   ? k_gn_grad_fused<T, 1, MODE>
            : p.nv == 2 ? k_gn_grad_fused<T, 2, MODE>
                        : k_gn_grad_fused<T, 4, MODE>;
  cudaError_t e = launch_cluster(
      fn, unsigned(p.grid_items * p.cluster), p.threads, fused_smem(p, MODE, dev::Vec16<T>::N, true), p.cluster,
      stream, static_cast<const T*>(a.dy), static_cast<const T*>(a.x), static_cast<const T*>(a.gamma),
      static_cast<const T*>(a.beta), a.mean, a.inv, static_cast<T*>(a.dx), cpart, d);
  if (e != cudaSuccess) return e;
  *launches += 1;
  if (cpart != nullptr) {
    const int64_t jobs = (int64_t(d.C) + 31) / 32 * 2;
    // the sums of du are dbeta, those of du * h are dgamma
    e = launch(k_channel_sums<T>, dim3(unsigned(jobs)), dim3(kSumsThreads), 0, stream, cpart,
               p.grid_items / p.slabs * p.cluster, int64_t(1), int64_t(d.C), 2, static_cast<T*>(a.dbeta),
               static_cast<T*>(a.dgamma));
    if (e == cudaSuccess) *launches += 1;
  }
  return e;
}

inline unsigned misalign16(const void* p) { return unsigned(reinterpret_cast<uintptr_t>(p) & 15u); }

// Items of the gradient that run at a time: all CTAs resident at about four (of
// 256 threads) an SM, a whole number of them for each slab.
void persist(FusedPlan* p) {
  const int64_t ctas = kPlanSms * std::max(1, 1024 / p->threads);
  const int64_t per_slab = std::max<int64_t>(1, ctas / (int64_t(p->slabs) * p->cluster));
  p->grid_items = std::min(p->items / p->slabs, per_slab) * p->slabs;
}

constexpr int kFwdNv = 16, kGradNv = 4;

bool grad_plan(int vw, int64_t N, int64_t S, int64_t C, int64_t G, bool slab, FusedPlan* p) {
  if (!fused_plan(vw, N, S, C, G, slab, kGradNv, p)) return false;
  persist(p);
  // a CTA's items share the offset of their channels: all samples start alike,
  // or a CTA has one sample
  if (!slab && S * C % vw != 0 && (p->samples > 1 || p->grid_items < p->items)) return false;
  return fused_smem(*p, slab ? 1 : 2, vw, true) <= kSmemMost;  // (mode 0 needs less)
}

}  // namespace

size_t group_norm_grad_fused_bytes(DType t, int64_t N, int64_t S, int64_t C, int64_t G) {
  const int vw = t == DType::F32 ? 4 : 8;
  size_t most = 0;
  TokenPlan tp;
  int set;
  if (token_plan(vw, N, S, C, G, &tp, &set)) most = size_t(tp.ctas) * size_t(C) * 8;
  for (int slab = 0; slab < 2; ++slab) {
    FusedPlan p;
    if (grad_plan(vw, N, S, C, G, slab != 0, &p))
      most = std::max(most, size_t(p.grid_items / p.slabs * p.cluster) * size_t(C) * 8);
  }
  return most;
}

cudaError_t launch_group_norm_fused(const GroupNormArgs& a, int, cudaStream_t stream, int* launches, bool* done) {
  const int vw = a.t == DType::F32 ? 4 : 8;
  const bool pvec = misalign16(a.gamma) == 0 && misalign16(a.beta) == 0;
  FusedDims d{a.N, a.S, a.S * a.C, int(a.C), int(a.G), int(a.C / a.G), a.eps, a.silu, pvec, {}};
  *done = false;
  if (misalign16(a.x) != misalign16(a.y)) return cudaSuccess;
  const bool slab = a.C % vw == 0 && misalign16(a.x) == 0;
  TokenPlan tp;
  int set;
  if (slab && token_plan(vw, a.N, a.S, a.C, a.G, &tp, &set)) {
    *done = true;
    const TokenDims t = token_dims(a.N, a.C, a.G, a.eps, a.silu, pvec, tp, set);
    switch (a.t) {
      case DType::F32: return token_fwd<float>(a, t, stream, launches);
      case DType::F16: return token_fwd<__half>(a, t, stream, launches);
      default: return token_fwd<__nv_bfloat16>(a, t, stream, launches);
    }
  }
  if (!fused_plan(vw, a.N, a.S, a.C, a.G, slab, kFwdNv, &d.p)) return cudaSuccess;
  const int mode = !slab ? 2 : d.D % vw == 0 ? 0 : 1;
  if (fused_smem(d.p, mode, vw, false) > kSmemMost) return cudaSuccess;
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

cudaError_t launch_group_norm_grad_fused(const GroupNormGradArgs& a, int, cudaStream_t stream, int* launches,
                                         bool* done) {
  const int vw = a.t == DType::F32 ? 4 : 8;
  const bool pvec = misalign16(a.gamma) == 0 && misalign16(a.beta) == 0;
  FusedDims d{a.N, a.S, a.S * a.C, int(a.C), int(a.G), int(a.C / a.G), 0.f, a.silu, pvec, {}};
  *done = false;
  if (misalign16(a.x) != misalign16(a.dy) || misalign16(a.x) != misalign16(a.dx)) return cudaSuccess;
  const bool slab = a.C % vw == 0 && misalign16(a.x) == 0;
  float* cpart = a.dgamma != nullptr || a.dbeta != nullptr ? static_cast<float*>(a.workspace) : nullptr;
  TokenPlan tp;
  int set;
  if (slab && token_plan(vw, a.N, a.S, a.C, a.G, &tp, &set)) {
    *done = true;
    const TokenDims t = token_dims(a.N, a.C, a.G, 0.f, a.silu, pvec, tp, set);
    switch (a.t) {
      case DType::F32: return token_grad<float>(a, t, cpart, stream, launches);
      case DType::F16: return token_grad<__half>(a, t, cpart, stream, launches);
      default: return token_grad<__nv_bfloat16>(a, t, cpart, stream, launches);
    }
  }
  if (!grad_plan(vw, a.N, a.S, a.C, a.G, slab, &d.p)) return cudaSuccess;
  *done = true;
  const int mode = !slab ? 2 : d.D % vw == 0 ? 0 : 1;
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

// BiasDropout and its gradient.
//
// Definition (the BiasDropout op of the contrib family that BiasAdd belongs to,
// with the mask given by a counter instead of stored):
//   Y[i]  = residual[i] + keep(i) * (X[i] + bias[i mod C]) / (1 - ratio)
//   dX[i] = keep(i) * dY[i] / (1 - ratio),  dbias[c] = sum over rows of dX
//   keep(i) = word(i) < K,  K = round((1 - ratio) 2^32), at least 1
//   word(i) = word i mod 4 of Philox4x32-10 at counter (i / 4, offset), key seed
// (J. Salmon, M. Moraes, R. Dror, D. Shaw, "Parallel random numbers: as easy as
// 1, 2, 3", SC 2011: ten rounds of two 32x32 -> 64-bit products each).  The mask
// is a function of the element's index, so the gradient makes it again and
// nothing of it is stored or read.
//
// Arithmetic is float32: X + bias and its product with 1 / (1 - ratio), then one
// fused multiply-add with the residual; one rounding to T at the store.
#include <algorithm>
#include <climits>

#include "column_walk.cuh"
#include "device_common.cuh"
#include "launch_util.h"
#include "training_internal.h"

namespace ep {
namespace {

constexpr int kThreads = 256;

// The generator's state of one call: the rounds' keys, the offset (plus *offset_dev, read
// when the kernel runs, so that a captured graph draws anew on every replay)
// and the last word that keeps an element.
constexpr int kRounds = 10;
struct DropRng {
  uint64_t offset;
  const uint64_t* offset_dev;
  uint32_t keys[2 * kRounds];  // the key words of each round
  uint32_t last_kept;
  float scale;
};

// The four words of a block.  Written in 32-bit halves, with the round keys from
// the kernel's parameters, so that a round is two wide multiplies and two
// three-input exclusive ors (as 64-bit products and running keys it took 140 us,
// not 108, for 2^27 float16 elements).  WIDE: block numbers beyond 32 bits (more
// than 2^34 elements).  Else the counter's second word is 0, and with the offset
// and the key the same in all threads the first two rounds have one product per
// thread each, not two.
template <bool WIDE>
__device__ __forceinline__ uint4 philox(uint64_t block, uint64_t offset, const DropRng& g) {
  uint32_t c0 = uint32_t(block), c1 = WIDE ? uint32_t(block >> 32) : 0u;
  uint32_t c2 = uint32_t(offset), c3 = uint32_t(offset >> 32);
#pragma unroll
  for (int r = 0; r < kRounds; ++r) {
    const uint32_t h0 = __umulhi(0xD2511F53u, c0), l0 = 0xD2511F53u * c0;
    const uint32_t h1 = __umulhi(0xCD9E8D57u, c2), l1 = 0xCD9E8D57u * c2;
    c0 = h1 ^ c1 ^ g.keys[2 * r];
    c1 = l1;
    c2 = h0 ^ c3 ^ g.keys[2 * r + 1];
    c3 = l0;
  }
  return make_uint4(c0, c1, c2, c3);
}

// v[e] = keep(i0 + e) ? v[e] : 0 for the VW elements from index i0 (a multiple of 4) on.
template <bool WIDE, int VW>
__device__ __forceinline__ void drop(int64_t i0, uint64_t offset, const DropRng& g, float (&v)[VW]) {
#pragma unroll
  for (int b = 0; b < VW; b += 4) {
    const uint4 w = philox<WIDE>(uint64_t(i0 + b) / 4, offset, g);
    v[b] = w.x <= g.last_kept ? v[b] : 0.f;
    v[b + 1] = w.y <= g.last_kept ? v[b + 1] : 0.f;
    v[b + 2] = w.z <= g.last_kept ? v[b + 2] : 0.f;
    v[b + 3] = w.w <= g.last_kept ? v[b + 3] : 0.f;
  }
}

__device__ __forceinline__ uint64_t offset_of(const DropRng& g) {
  return g.offset + (g.offset_dev != nullptr ? *g.offset_dev : 0ull);
}

// A fragment as it is loaded: 16 bytes (VEC, aligned and whole), else VW values.
template <typename T, bool VEC> struct RawFrag;
template <typename T> struct RawFrag<T, true> {
  uint4 u;
  __device__ __forceinline__ void load(const T* p, int64_t i0, int64_t) { u = dev::ld16_stream(p + i0); }
  __device__ __forceinline__ void get(float (&v)[dev::Vec16<T>::N]) const { dev::Conv<T>::unpack(u, v); }
};
template <typename T> struct RawFrag<T, false> {
  float f[dev::Vec16<T>::N];
  __device__ __forceinline__ void load(const T* p, int64_t i0, int64_t n) { dev::load_frag<T, false>(p, i0, n, f); }
  __device__ __forceinline__ void get(float (&v)[dev::Vec16<T>::N]) const {
#pragma unroll
    for (int e = 0; e < dev::Vec16<T>::N; ++e) v[e] = f[e];
  }
};

// One fragment of the forward pass: bias, scale and mask on `v`, the residual
// added, stored.
template <typename T, int BIAS, bool RES, bool VEC, bool WIDE>
__device__ __forceinline__ void drop_frag(int64_t i0, int64_t n, int64_t col, int64_t C, const T* __restrict__ bias,
                                          uint64_t offset, const DropRng& g, float (&v)[dev::Vec16<T>::N],
                                          const RawFrag<T, VEC>& res, T* y) {
  constexpr int VW = dev::Vec16<T>::N;
  if constexpr (BIAS == 1) {
    dev::add_raw<T>(dev::ld16_keep(bias + col), v);
  } else if constexpr (BIAS == 2) {
    int64_t c = col;
#pragma unroll
    for (int e = 0; e < VW; ++e) {
      v[e] = __fadd_rn(v[e], dev::ld1_keep(bias + c));
      if (++c == C) c = 0;
    }
  }
  drop<WIDE>(i0, offset, g, v);  // a dropped element is 0 from here on, whatever it was
  if constexpr (RES) {
    float r[VW];
    res.get(r);
#pragma unroll
    for (int e = 0; e < VW; ++e) v[e] = fmaf(v[e], g.scale, r[e]);
  } else {
    dev::scale_pairs(v, g.scale);
  }
  dev::store_frag<T, VEC>(y, i0, n, v);
}

// BIAS 0: none; 1: C % VW == 0 and the bias 16-byte aligned (a fragment's bias
// is one 16-byte read); 2: any other.  VEC: X, residual and Y 16-byte aligned.
// Flat fragments, so rows of any C; the last one may be partial and is done
// apart.  f16 32x8192x512 without bias and residual 106 us (537 MB, 76 % of the copy
// rate), bf16 16x1024x4096 with both 71 (403 MB, 84 %).  No unit is full (an instruction
// issued in 0.6 of the cycles, DRAM at 56 and 63 %, 42 to 51 % of the warps): a thread
// loads its fragments, makes their words and stores before it loads the next, so the
// loads and the generator's chains of wide multiplies take turns.
template <typename T, int BIAS, bool RES, bool VEC, bool WIDE>
__global__ void __launch_bounds__(kThreads)
k_bias_dropout(const T* x, const T* __restrict__ bias, const T* residual, T* y, int64_t n, int64_t C,
               int64_t col_step, DropRng g) {
  constexpr int VW = dev::Vec16<T>::N;
  constexpr int U = 4;
  dev::pdl_wait();
  dev::pdl_trigger();
  const uint64_t offset = offset_of(g);
  const int64_t nfrag = VEC ? n / VW : (n + VW - 1) / VW;
  const int64_t stride = int64_t(gridDim.x) * kThreads;
  const int64_t f00 = int64_t(blockIdx.x) * kThreads + threadIdx.x;
  int64_t col = BIAS ? (f00 * VW) % C : 0;
  for (int64_t f0 = f00; f0 < nfrag; f0 += stride * U) {
    RawFrag<T, VEC> a[U], r[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t f = f0 + u * stride;
      if (f < nfrag) {
        a[u].load(x, f * VW, n);
        if constexpr (RES) r[u].load(residual, f * VW, n);
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t f = f0 + u * stride;
      if (f < nfrag) {
        float v[VW];
        a[u].get(v);
        drop_frag<T, BIAS, RES, VEC, WIDE>(f * VW, n, col, C, bias, offset, g, v, r[u], y);
        if constexpr (BIAS != 0) {
          col += col_step;
          if (col >= C) col -= C;
        }
      }
    }
  }
  if constexpr (VEC) {  // the elements after the last whole fragment
    if (f00 == 0 && n % VW != 0) {
      const int64_t i0 = n - n % VW;
      RawFrag<T, false> r;
      float v[VW];
      dev::load_frag<T, false>(x, i0, n, v);
      if constexpr (RES) r.load(residual, i0, n);
      drop_frag<T, BIAS == 1 ? 2 : BIAS, RES, false, WIDE>(i0, n, i0 % C, C, bias, offset, g, v, r, y);
    }
  }
}

// Gradient with dbias: every thread walks one fragment column (column_walk.cuh),
// adds the dX it writes, in float32 and before they are rounded, to its VW
// sums, and leaves the sums of its chunk in `partial`: [chunk][C] where one tile covers a
// walk row (the block adds the repeats of a channel up), else [chunk][walk row].
// bf16 16x1024x4096: 58 us (268 MB, 69 % of the copy rate), with DRAM at 50 %, as above.
template <typename T, bool VEC, bool WIDE>
__global__ void __launch_bounds__(kWalkThreads, 4)
k_bias_dropout_grad(const T* dy, T* dx, int64_t n, int64_t C, WalkPlan p, int64_t full_rows, int64_t rest, DropRng g,
                    float* partial) {
  constexpr int VW = dev::Vec16<T>::N;
  constexpr int U = 3;
  __shared__ float sums[kWalkThreads * VW];
  dev::pdl_wait();
  dev::pdl_trigger();
  const uint64_t offset = offset_of(g);
  const int tile = blockIdx.x % p.tiles;
  const int64_t chunk = blockIdx.x / p.tiles;
  const int64_t j = int64_t(tile) * p.tile_frags + threadIdx.x;
  const bool mine = int(threadIdx.x) < p.tile_frags && j < p.row_frags;
  float acc[VW];
#pragma unroll
  for (int e = 0; e < VW; ++e) acc[e] = 0.f;
  auto row = [&](int64_t i0, float (&v)[VW]) {
    drop<WIDE>(i0, offset, g, v);
    dev::scale_pairs(v, g.scale);
    dev::add_pairs(acc, v);
  };
  if (mine) {
    const int64_t ra = chunk * p.rows_per_chunk, pitch = p.row_frags * VW;
    // rows of this chunk with a whole fragment in this column, and then perhaps the tensor's last, partial one
    const int64_t rb = min(full_rows + (j < rest ? 1 : 0), ra + p.rows_per_chunk);
    int64_t i0 = (ra * p.row_frags + j) * VW, r = ra;
    for (; r + U <= rb; r += U, i0 += U * pitch) {
      RawFrag<T, VEC> a[U];
#pragma unroll
      for (int u = 0; u < U; ++u) a[u].load(dy, i0 + u * pitch, n);
#pragma unroll
      for (int u = 0; u < U; ++u) {
        float v[VW];
        a[u].get(v);
        row(i0 + u * pitch, v);
        if constexpr (VEC) dev::st16_stream(dx + i0 + u * pitch, dev::Conv<T>::pack(v));
        else dev::store_frag<T, false>(dx, i0 + u * pitch, n, v);
      }
    }
    for (; r < rb; ++r, i0 += pitch) {
      RawFrag<T, VEC> a;
      float v[VW];
      a.load(dy, i0, n);
      a.get(v);
      row(i0, v);
      dev::store_frag<T, VEC>(dx, i0, n, v);
    }
    if (j == rest && n % VW != 0 && r == full_rows && r < ra + p.rows_per_chunk) {
      float v[VW];
      dev::load_frag<T, false>(dy, i0, n, v);
      row(i0, v);
      dev::store_frag<T, false>(dx, i0, n, v);
    }
  }
  if (p.tiles > 1) {
    if (mine) {
      float* out = partial + (chunk * p.row_frags + j) * VW;
#pragma unroll
      for (int e = 0; e < VW; e += 4)
        *reinterpret_cast<float4*>(out + e) = make_float4(acc[e], acc[e + 1], acc[e + 2], acc[e + 3]);
    }
    return;
  }
  if (mine) {
#pragma unroll
    for (int e = 0; e < VW; ++e) sums[threadIdx.x * VW + e] = acc[e];
  }
  __syncthreads();
  const int c32 = static_cast<int>(C), reps = static_cast<int>(p.reps);
  if (reps <= 16) {
    for (int c = threadIdx.x; c < c32; c += blockDim.x) {
      float s = 0.f;
      for (int k = 0; k < reps; ++k) s += sums[c + k * c32];
      partial[chunk * C + c] = s;
    }
  } else {  // few channels, many repeats: a warp each
    const int lane = threadIdx.x & 31;
    for (int c = threadIdx.x >> 5; c < c32; c += blockDim.x >> 5) {
      float s = 0.f;
      for (int k = lane; k < reps; k += 32) s += sums[c + k * c32];
      s = dev::warp_sum(s);
      if (lane == 0) partial[chunk * C + c] = s;
    }
  }
}

inline bool al16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

inline DropRng rng_of(const BiasDropoutArgs& a) {
  DropRng g{a.offset, a.offset_dev, {}, a.last_kept, a.scale};
  uint32_t k0 = uint32_t(a.seed), k1 = uint32_t(a.seed >> 32);
  for (int r = 0; r < kRounds; ++r) {
    g.keys[2 * r] = k0;
    g.keys[2 * r + 1] = k1;
    k0 += 0x9E3779B9u;
    k1 += 0xBB67AE85u;
  }
  return g;
}

template <typename T, int BIAS, bool RES, bool VEC, bool WIDE>
cudaError_t launch_fwd(const BiasDropoutArgs& a, int sm_count, cudaStream_t stream, int* launches) {
  constexpr int VW = dev::Vec16<T>::N;
  const int64_t nfrag = (a.n + VW - 1) / VW;
  const int64_t need = (nfrag + kThreads - 1) / kThreads;
  const int64_t grid = std::max<int64_t>(1, std::min<int64_t>(need, int64_t(sm_count) * 8));
  const int64_t step = BIAS ? (grid * kThreads * VW) % a.C : 0;
  cudaError_t e = launch(k_bias_dropout<T, BIAS, RES, VEC, WIDE>, dim3(unsigned(grid)), dim3(kThreads), 0, stream,
                         static_cast<const T*>(a.x), static_cast<const T*>(a.bias),
                         static_cast<const T*>(a.residual), static_cast<T*>(a.y), a.n, a.C, step, rng_of(a));
  if (e == cudaSuccess) *launches += 1;
  return e;
}

// Block numbers of the generator fit 32 bits.
inline bool narrow(int64_t n) { return (n + 3) / 4 <= (int64_t(1) << 32); }

template <typename T, bool RES>
cudaError_t bias_dropout_t(const BiasDropoutArgs& a, int sm_count, cudaStream_t stream, int* launches) {
  constexpr int VW = dev::Vec16<T>::N;
  const bool vec = al16(a.x) && al16(a.y) && (!RES || al16(a.residual));
  if (!narrow(a.n) || !vec) {  // the general form of both
    return a.bias == nullptr ? launch_fwd<T, 0, RES, false, true>(a, sm_count, stream, launches)
                             : launch_fwd<T, 2, RES, false, true>(a, sm_count, stream, launches);
  }
  if (a.bias == nullptr) return launch_fwd<T, 0, RES, true, false>(a, sm_count, stream, launches);
  if (a.C % VW == 0 && al16(a.bias)) return launch_fwd<T, 1, RES, true, false>(a, sm_count, stream, launches);
  return launch_fwd<T, 2, RES, true, false>(a, sm_count, stream, launches);
}

WalkPlan grad_walk(DType t, int64_t n, int64_t C) {
  return make_walk(n, C, t == DType::F32 ? 4 : 8, 1, kPlanSms * 8, 4);
}

template <typename T>
cudaError_t bias_dropout_grad_t(const BiasDropoutArgs& a, cudaStream_t stream, int* launches) {
  const WalkPlan p = grad_walk(a.t, a.n, a.C);
  float* partial = static_cast<float*>(a.workspace);
  const dim3 grid(unsigned(int64_t(p.tiles) * p.chunks));
  constexpr int VW = dev::Vec16<T>::N;
  const int64_t full_rows = a.n / VW / p.row_frags, rest = a.n / VW % p.row_frags;
  cudaError_t e;
  if (al16(a.x) && al16(a.y) && narrow(a.n))
    e = launch(k_bias_dropout_grad<T, true, false>, grid, dim3(p.threads), 0, stream, static_cast<const T*>(a.x),
               static_cast<T*>(a.y), a.n, a.C, p, full_rows, rest, rng_of(a), partial);
  else
    e = launch(k_bias_dropout_grad<T, false, true>, grid, dim3(p.threads), 0, stream, static_cast<const T*>(a.x),
               static_cast<T*>(a.y), a.n, a.C, p, full_rows, rest, rng_of(a), partial);
  if (e != cudaSuccess) return e;
  *launches += 1;
  const int64_t jobs = std::min<int64_t>((a.C + 31) / 32, INT_MAX);
  e = launch(k_channel_sums<T>, dim3(unsigned(jobs)), dim3(kSumsThreads), 0, stream, partial, int64_t(p.chunks),
             p.tiles > 1 ? p.reps : int64_t(1), a.C, 1, static_cast<T*>(a.dbias), static_cast<T*>(nullptr));
  if (e == cudaSuccess) *launches += 1;
  return e;
}

}  // namespace

cudaError_t launch_bias_dropout(const BiasDropoutArgs& a, int sm_count, cudaStream_t stream, int* launches) {
  const bool res = a.residual != nullptr;
  switch (a.t) {
    case DType::F32:
      return res ? bias_dropout_t<float, true>(a, sm_count, stream, launches)
                 : bias_dropout_t<float, false>(a, sm_count, stream, launches);
    case DType::F16:
      return res ? bias_dropout_t<__half, true>(a, sm_count, stream, launches)
                 : bias_dropout_t<__half, false>(a, sm_count, stream, launches);
    default:
      return res ? bias_dropout_t<__nv_bfloat16, true>(a, sm_count, stream, launches)
                 : bias_dropout_t<__nv_bfloat16, false>(a, sm_count, stream, launches);
  }
}

cudaError_t launch_bias_dropout_grad(const BiasDropoutArgs& a, int sm_count, cudaStream_t stream, int* launches) {
  // without dbias the gradient is the forward pass of dY, without bias and residual
  if (a.dbias == nullptr) return launch_bias_dropout(a, sm_count, stream, launches);
  switch (a.t) {
    case DType::F32: return bias_dropout_grad_t<float>(a, stream, launches);
    case DType::F16: return bias_dropout_grad_t<__half>(a, stream, launches);
    default: return bias_dropout_grad_t<__nv_bfloat16>(a, stream, launches);
  }
}

size_t bias_dropout_grad_workspace_bytes(DType t, int64_t n, int64_t C) {
  const WalkPlan p = grad_walk(t, n, C);
  const int64_t width = p.tiles > 1 ? p.row_frags * (t == DType::F32 ? 4 : 8) : C;
  return size_t(p.chunks) * size_t(width) * sizeof(float);
}

}  // namespace ep

// Tensor-core primitives of sm_103a: tcgen05 matrix products of shared-memory
// operands into tensor memory (TMEM), tiled TMA loads, and the barriers between
// them, within one CTA or a pair of CTAs (a cluster of two whose tensor cores
// work on one tile: cta_group::2).
//
// Operand tiles in shared memory are 128 bytes wide in the dimension that is
// contiguous in memory, 128-byte swizzled (as TMA writes them with
// CU_TENSOR_MAP_SWIZZLE_128B), in atoms of 8 lines of 128 bytes:
//   K-major (the summed dimension is contiguous): a line is a row's 128 bytes of K;
//     8 rows to the next 1024 bytes; 32 bytes further along the line for the next K of an MMA.
//   MN-major (16-bit only): a line is 64 rows at one k; 8 k to the next 1024 bytes, 64 k to
//     the next 64 rows (8192 bytes); 16 lines (2048 bytes) further for the next K of an MMA.
#pragma once

#include <cstdint>

#include <cuda.h>
#include <cuda_runtime.h>

#include "tma_pipe.cuh"

namespace ep {
namespace dev {

// ---------------------------------------------------------------------------
// one thread of a warp
//
// Loads and products are issued by one elected lane inside control flow that the
// whole warp follows: their operands can then live in uniform registers.  (Issued
// under a comparison of the lane's number, each cost some 70 cycles.)
// ---------------------------------------------------------------------------

__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(p));
  return p != 0;
}

// The warp's number, known to be the same in all its lanes.
__device__ __forceinline__ int warp_number() { return __shfl_sync(0xffffffffu, int(threadIdx.x >> 5), 0); }

// mbar_wait by a whole warp: all lanes have the same answer.
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity) {
  return __all_sync(0xffffffffu, mbar_wait(bar, parity));
}

// ---------------------------------------------------------------------------
// clusters
// ---------------------------------------------------------------------------

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}

// The address, in the cluster's shared memory, of the same place in CTA `rank`.
__device__ __forceinline__ uint32_t cluster_addr(uint32_t local, uint32_t rank) {
  uint32_t a;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(local), "r"(rank));
  return a;
}

// The two halves of the cluster's barrier, by all threads of converged warps.
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_sync() {
  cluster_arrive();
  cluster_wait();
}

__device__ __forceinline__ void st_cluster(uint32_t addr, uint32_t v) {
  asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}

// Arrives on a barrier anywhere in the cluster.  What it announces is read by the
// asynchronous proxy (the tensor cores read shared memory that the arriving thread
// has fenced) or is tensor memory, so the default scope does: at cluster scope each
// arrival waited for all of the thread's memory operations, 0.5 us.
__device__ __forceinline__ void mbar_arrive_cluster(uint32_t addr) {
  asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(addr) : "memory");
}

// ---------------------------------------------------------------------------
// TMA
// ---------------------------------------------------------------------------

__device__ __forceinline__ void prefetch_map(const CUtensorMap* map) {
  asm volatile("prefetch.tensormap [%0];" ::"l"(map) : "memory");
}

// A box of a two-dimensional tensor to this CTA's shared memory.  `bar`: the
// barrier's cluster address (with PAIR in either CTA of the pair).
template <bool PAIR>
__device__ __forceinline__ void tma_load(uint32_t dst, const CUtensorMap* map, uint32_t bar, int x, int y) {
  if constexpr (PAIR) {
    asm volatile(
        "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes "
        "[%0], [%1, {%3, %4}], [%2];" ::"r"(dst), "l"(map), "r"(bar), "r"(x), "r"(y)
        : "memory");
  } else {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes "
        "[%0], [%1, {%3, %4}], [%2];" ::"r"(dst), "l"(map), "r"(bar), "r"(x), "r"(y)
        : "memory");
  }
}

// ---------------------------------------------------------------------------
// tensor memory
// ---------------------------------------------------------------------------

// By one whole warp (with PAIR: of each CTA).  The address goes to shared memory.
template <bool PAIR>
__device__ __forceinline__ void tmem_alloc(uint32_t* where, uint32_t columns) {
  if constexpr (PAIR) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(where)), "r"(columns)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;");
  } else {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(where)), "r"(columns)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  }
}
template <bool PAIR>
__device__ __forceinline__ void tmem_free(uint32_t addr, uint32_t columns) {
  if constexpr (PAIR) asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(addr), "r"(columns));
  else asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(addr), "r"(columns));
}

__device__ __forceinline__ void tmem_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tmem_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }

// Waits for this thread's loads, whose registers are operands here so that no use of them moves above it.
template <int N>
__device__ __forceinline__ void tmem_wait_ld(uint32_t (&r)[N]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
  for (int i = 0; i < N; ++i) asm volatile("" : "+r"(r[i]));
}

// 8 or 32 columns of the warp's 32 lanes: register i of a lane is column i.
__device__ __forceinline__ void tmem_ld8(uint32_t addr, uint32_t (&r)[8]) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
               : "r"(addr));
}
__device__ __forceinline__ void tmem_ld32(uint32_t addr, uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
        "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
        "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(addr));
}

// ---------------------------------------------------------------------------
// matrix products
// ---------------------------------------------------------------------------

// Shared-memory descriptors: address, the strides above, 128-byte swizzle.
__device__ __forceinline__ uint64_t operand_desc(uint32_t addr, bool mn) {
  return (uint64_t(2) << 61) | (uint64_t(1) << 46) | (uint64_t(1024 >> 4) << 32) |
         (uint64_t(mn ? 8192 >> 4 : 1) << 16) | uint64_t((addr & 0x3FFFF) >> 4);
}
// What the next K of an MMA (32 bytes of K) adds to it.
__device__ __forceinline__ uint64_t operand_step(bool mn) { return mn ? 2048 >> 4 : 32 >> 4; }

// 512 bytes of scales: 32 lines of 16 bytes, no swizzle, 8 lines to 128 bytes.
__device__ __forceinline__ uint64_t scales_desc(uint32_t addr) {
  return (uint64_t(1) << 46) | (uint64_t(128 >> 4) << 32) | uint64_t((addr & 0x3FFFF) >> 4);
}

// d (+)= a b of 16-bit operands (K = 16).
template <bool PAIR>
__device__ __forceinline__ void mma_f16(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool add) {
  if constexpr (PAIR) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d), "l"(a), "l"(b), "r"(idesc), "r"(uint32_t(add))
        : "memory");
  } else {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d), "l"(a), "l"(b), "r"(idesc), "r"(uint32_t(add))
        : "memory");
  }
}

// The same of 8-bit operands (K = 32) with a scale for each row's 32 values.
template <bool PAIR>
__device__ __forceinline__ void mma_mx8(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t sfa, uint32_t sfb,
                                        bool add) {
  if constexpr (PAIR) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::mxf8f6f4.block_scale [%0], %1, %2, %3, [%5], [%6], p;\n\t}" ::"r"(d), "l"(a),
        "l"(b), "r"(idesc), "r"(uint32_t(add)), "r"(sfa), "r"(sfb)
        : "memory");
  } else {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::mxf8f6f4.block_scale [%0], %1, %2, %3, [%5], [%6], p;\n\t}" ::"r"(d), "l"(a),
        "l"(b), "r"(idesc), "r"(uint32_t(add)), "r"(sfa), "r"(sfb)
        : "memory");
  }
}

// 512 bytes of scales from shared memory to 4 columns of TMEM (line i to lane i of each quarter).
template <bool PAIR>
__device__ __forceinline__ void copy_scales(uint32_t tmem, uint64_t desc) {
  if constexpr (PAIR) asm volatile("tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;" ::"r"(tmem), "l"(desc) : "memory");
  else asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(tmem), "l"(desc) : "memory");
}

// Arrives on `bar` (with PAIR on that of the CTAs in `ctas`, a bit each) once this thread's matrix products so
// far are done.  Someone in each of those CTAs waits for it before the CTA leaves.
template <bool PAIR>
__device__ __forceinline__ void mma_commit(uint64_t* bar, uint16_t ctas = 3) {
  if constexpr (PAIR) {
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
            smem_addr(bar)),
        "h"(ctas)
        : "memory");
  } else {
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_addr(bar))
                 : "memory");
  }
}

}  // namespace dev

// Instruction descriptors: float32 sums; rows `m` and columns `n` of the tile.
inline uint32_t mma_desc_f16(bool bf16, bool a_mn, bool b_mn, int m, int n) {
  return (1u << 4) | (bf16 ? (1u << 7) | (1u << 10) : 0u) | (a_mn ? 1u << 15 : 0u) | (b_mn ? 1u << 16 : 0u) |
         (uint32_t(n >> 3) << 17) | (uint32_t(m >> 4) << 24);
}
// E4M3 with E8M0 scales; the scales' byte k of 4 is or-ed in by mma_scale_byte.
inline uint32_t mma_desc_mx8(int m, int n) { return (1u << 23) | (uint32_t(n >> 3) << 17) | (uint32_t(m >> 4) << 24); }
__device__ __forceinline__ uint32_t mma_scale_byte(int k) { return (uint32_t(k) << 4) | (uint32_t(k) << 29); }

}  // namespace ep

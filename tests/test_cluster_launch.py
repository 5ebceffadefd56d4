"""How many clusters fit is asked for each kernel, against a CUDA runtime that answers by the kernel."""
import os
import subprocess

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "transformer_epilogue_gb300", "csrc")

RUNTIME = r"""
#pragma once
#include <cstddef>
#include <cstdint>
typedef int cudaError_t; typedef void* cudaStream_t;
enum { cudaSuccess = 0, cudaDevAttrMaxSharedMemoryPerBlockOptin = 1, cudaFuncAttributeMaxDynamicSharedMemorySize = 2,
       cudaLaunchAttributeProgrammaticStreamSerialization = 3, cudaLaunchAttributeClusterDimension = 4 };
struct dim3 { unsigned x, y, z; dim3(unsigned a = 1, unsigned b = 1, unsigned c = 1) : x(a), y(b), z(c) {} };
struct cudaFuncAttributes { size_t sharedSizeBytes; };
struct cudaLaunchAttribute { int id; struct { int programmaticStreamSerializationAllowed;
                                              struct { unsigned x, y, z; } clusterDim; } val; };
struct cudaLaunchConfig_t { dim3 gridDim, blockDim; size_t dynamicSmemBytes; cudaStream_t stream;
                            cudaLaunchAttribute* attrs; int numAttrs; };
inline int g_dev, g_asked, g_grid, g_threads, g_smem, g_cluster;
inline cudaError_t cudaGetDevice(int* d) { *d = g_dev; return 0; }
inline cudaError_t cudaDeviceGetAttribute(int* v, int, int) { *v = 232448; return 0; }
inline cudaError_t cudaFuncGetAttributes(cudaFuncAttributes* a, const void*) { a->sharedSizeBytes = 64; return 0; }
inline cudaError_t cudaFuncSetAttribute(const void*, int, int) { return 0; }
// what a kernel answers, by its "registers"
int fits(const void* kernel, int threads, size_t smem);
template <typename... A> cudaError_t cudaOccupancyMaxActiveClusters(int* n, void (*k)(A...), const cudaLaunchConfig_t* c) {
  ++g_asked;
  *n = fits(reinterpret_cast<const void*>(k), int(c->blockDim.x), c->dynamicSmemBytes) / int(c->attrs[0].val.clusterDim.x);
  return 0;
}
template <typename... A> cudaError_t cudaLaunchKernelEx(const cudaLaunchConfig_t* c, void (*)(A...), const A&...) {
  g_grid = int(c->gridDim.x); g_threads = int(c->blockDim.x); g_smem = int(c->dynamicSmemBytes);
  g_cluster = int(c->attrs[1].val.clusterDim.x);
  return 0;
}
"""

PROGRAM = r"""
#include <cstdio>
#include "cluster_launch.h"
struct Args { int a; };
template <int N> void kernel(Args) { std::printf("never %d\n", N); }
int fits(const void* k, int threads, size_t smem) {
  return (k == reinterpret_cast<const void*>(&kernel<0>) ? 152 : k == reinterpret_cast<const void*>(&kernel<1>) ? 304 : 0) *
         (threads > 256 ? 1 : 2) / (smem > 100000 ? 1 : 2) / (g_dev + 1);
}
int main() {
  const auto ask = [](void (*k)(Args), unsigned threads, size_t smem, unsigned cluster) {
    int n = -1;
    return ep::resident_clusters(k, threads, smem, cluster, 152, &n) == cudaSuccess ? n : -2;
  };
  for (int round = 0; round < 3; ++round) {
    g_dev = 0;
    // two kernels of the same argument type, in either order
    if (ask(round < 2 ? kernel<0> : kernel<1>, 384, 200000, 2) != (round < 2 ? 76 : 152)) return 1;
    if (ask(kernel<1>, 384, 200000, 2) != 152 || ask(kernel<0>, 384, 200000, 2) != 76) return 2;
    // other threads, bytes, clusters and devices
    if (ask(kernel<0>, 128, 200000, 2) != 152 || ask(kernel<0>, 384, 1000, 2) != 38 || ask(kernel<0>, 384, 200000, 4) != 38) return 3;
    g_dev = 1;
    if (ask(kernel<0>, 384, 200000, 2) != 38) return 4;
    if (ask(kernel<2>, 384, 200000, 2) != 1) return 5;  // never none
  }
  if (ep::launch_cluster(kernel<0>, 76, 384, 200000, 2, nullptr, Args{1}) != cudaSuccess) return 6;
  std::printf("%d %d %d %d %d\n", g_asked, g_grid, g_threads, g_smem, g_cluster);
}
"""


def test_each_kernel_has_its_own_answer(tmp_path):
    (tmp_path / "cuda_runtime.h").write_text(RUNTIME)
    (tmp_path / "main.cpp").write_text(PROGRAM)
    exe = str(tmp_path / "main")
    subprocess.run(["g++", "-std=c++17", "-Wall", "-I", str(tmp_path), "-I", CSRC, str(tmp_path / "main.cpp"), "-o", exe],
                   check=True, timeout=120)
    p = subprocess.run([exe], capture_output=True, text=True, timeout=60)
    assert p.returncode == 0 and p.stdout.split() == ["7", "76", "384", "200000", "2"], (p.returncode, p.stdout)


def test_the_pair_kernels_ask_for_themselves():
    with open(os.path.join(CSRC, "matmul.cu"), encoding="utf-8") as f:
        src = f.read()
    assert "resident_clusters(kernel, kPairThreads, S::kSmem, 2," in src and "cudaOccupancyMaxActiveClusters" not in src

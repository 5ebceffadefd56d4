"""The host tables behind a launch, compiled against a CUDA runtime that counts calls:
GroupNorm's launches, whose threads and shared memory follow the shape, must not use up
the table of occupancy answers that the other ops' launches read."""
import os
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "transformer_epilogue_gb300", "csrc")

RUNTIME = r"""
#pragma once
#include <cstddef>
#include <cstdint>
typedef int cudaError_t; typedef void* cudaStream_t;
enum { cudaSuccess = 0, cudaDevAttrMaxSharedMemoryPerBlockOptin = 1, cudaFuncAttributeMaxDynamicSharedMemorySize = 2,
       cudaLaunchAttributeProgrammaticStreamSerialization = 3 };
struct dim3 { unsigned x, y, z; };
struct cudaFuncAttributes { size_t sharedSizeBytes; };
struct cudaLaunchAttribute { int id; struct { int programmaticStreamSerializationAllowed; } val; };
struct cudaLaunchConfig_t { dim3 gridDim, blockDim; size_t dynamicSmemBytes; cudaStream_t stream;
                            cudaLaunchAttribute* attrs; int numAttrs; };
inline int g_dev, g_occupancy, g_raised, g_last_bytes;
inline cudaError_t cudaGetDevice(int* d) { *d = g_dev; return 0; }
inline cudaError_t cudaDeviceGetAttribute(int* v, int, int) { *v = 232448; return 0; }
inline cudaError_t cudaFuncGetAttributes(cudaFuncAttributes* a, const void*) { a->sharedSizeBytes = 64; return 0; }
inline cudaError_t cudaFuncSetAttribute(const void*, int, int v) { ++g_raised; g_last_bytes = v; return 0; }
inline cudaError_t cudaOccupancyMaxActiveBlocksPerMultiprocessor(int* r, const void*, int, size_t) {
  ++g_occupancy; *r = 2; return 0;
}
template <typename... A> cudaError_t cudaLaunchKernelEx(const cudaLaunchConfig_t*, void (*)(A...), A...) { return 0; }
"""

PROGRAM = r"""
#include <cstdio>
#include "launch_util.h"
#include "smem_limit.h"
static char kernels[400];
int main() {
  // 300 kernels on 3 devices, launched over and over
  for (int round = 0; round < 4; ++round)
    for (g_dev = 0; g_dev < 3; ++g_dev)
      for (int k = 0; k < 300; ++k)
        if (ep::allow_smem(kernels + k) != cudaSuccess) return 1;
  const int raised = g_raised, bytes = g_last_bytes, asked = g_occupancy;
  // another op's kernel, at new shapes: one question each
  g_dev = 0;
  int per_sm = 0;
  for (int round = 0; round < 3; ++round)
    for (int s = 0; s < 100; ++s)
      if (ep::resident_ctas(kernels + 399, 256, 1000 + s, &per_sm) != cudaSuccess || per_sm != 2) return 2;
  std::printf("%d %d %d %d\n", raised, bytes, asked, g_occupancy);
}
"""


def test_a_kernel_takes_one_entry_whatever_its_shapes(tmp_path):
    (tmp_path / "cuda_runtime.h").write_text(RUNTIME)
    (tmp_path / "main.cpp").write_text(PROGRAM)
    exe = str(tmp_path / "main")
    subprocess.run(["g++", "-std=c++17", "-Wall", "-I", str(tmp_path), "-I", CSRC, str(tmp_path / "main.cpp"), "-o", exe],
                   check=True, timeout=120)
    out = subprocess.run([exe], check=True, capture_output=True, text=True, timeout=60).stdout.split()
    assert out == ["900", str(232448 - 64), "0", "100"]


@pytest.mark.parametrize("source", ["group_norm.cu", "group_norm_fused.cu", "bias_dropout.cu"])
def test_shape_dependent_launches_ask_no_occupancy(source):
    with open(os.path.join(CSRC, source), encoding="utf-8") as f:
        assert "resident_ctas" not in f.read()

// Host helpers for kernels of clusters: the launch, and how many clusters fit on the
// device at once (as launch_util.h for the other kernels).
#pragma once

#include <algorithm>
#include <cstddef>
#include <cstdint>
#include <mutex>

#include <cuda_runtime.h>

#include "smem_limit.h"
#include "tuning.h"

namespace ep {

template <typename Args>
inline cudaError_t launch_cluster(void (*kernel)(Args), unsigned grid, unsigned threads, size_t smem, unsigned cluster,
                                  cudaStream_t stream, const Args& args) {
  const cudaError_t e = allow_smem(reinterpret_cast<const void*>(kernel));
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = EP_PDL ? 1 : 0;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = cluster;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kernel, args);
}

// Clusters of `cluster` CTAs of `kernel` that fit on the current device, of `sm_count` SMs, at once (>= 1);
// asked once for a kernel, threads and bytes on a device.
template <typename Args>
inline cudaError_t resident_clusters(void (*kernel)(Args), unsigned threads, size_t smem, unsigned cluster, int sm_count,
                                     int* clusters) {
  struct Entry {
    const void* fn;
    int dev;
    unsigned threads, cluster;
    size_t smem;
    int clusters;
  };
  constexpr int kCache = 256;
  static std::mutex mu;
  static Entry known[kCache];
  static int n = 0;

  const void* fn = reinterpret_cast<const void*>(kernel);
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  std::lock_guard<std::mutex> lk(mu);
  for (int i = 0; i < n; ++i)
    if (known[i].fn == fn && known[i].dev == dev && known[i].threads == threads && known[i].cluster == cluster &&
        known[i].smem == smem) {
      *clusters = known[i].clusters;
      return cudaSuccess;
    }
  e = allow_smem(fn);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(unsigned(sm_count) / cluster * cluster);
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = cluster;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  int fit = 0;
  e = cudaOccupancyMaxActiveClusters(&fit, kernel, &cfg);
  if (e != cudaSuccess) return e;
  *clusters = std::max(1, fit);
  if (n < kCache) known[n++] = Entry{fn, dev, threads, cluster, smem, *clusters};
  return cudaSuccess;
}

}  // namespace ep

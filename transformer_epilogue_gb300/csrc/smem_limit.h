// Raising a kernel's dynamic shared-memory limit, for launches that need no more than
// that.  launch_util.h's resident_ctas raises it too, but keeps an answer of the
// occupancy calculator for every (kernel, device, threads, bytes) it is asked: launches
// whose threads and bytes follow the shape would fill its table for the kernels that use
// the answers.  Here an entry is a kernel on a device.
#pragma once

#include <cstddef>
#include <cstdint>
#include <mutex>

#include <cuda_runtime.h>

namespace ep {

// Lets `fn` be launched with up to the current device's opt-in maximum of dynamic shared memory.
inline cudaError_t allow_smem(const void* fn) {
  struct Entry {
    const void* fn;
    int dev;
  };
  constexpr unsigned kSlots = 4096;  // open addressing; three quarters are used at most
  static std::mutex mu;
  static Entry table[kSlots];
  static unsigned used = 0;

  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  std::lock_guard<std::mutex> lk(mu);
  unsigned at = unsigned((reinterpret_cast<uintptr_t>(fn) + unsigned(dev)) * 0x9E3779B97F4A7C15ull >> 40) % kSlots;
  for (; table[at].fn != nullptr; at = (at + 1) % kSlots)
    if (table[at].fn == fn && table[at].dev == dev) return cudaSuccess;
  int optin = 0;
  e = cudaDeviceGetAttribute(&optin, cudaDevAttrMaxSharedMemoryPerBlockOptin, dev);
  if (e != cudaSuccess) return e;
  cudaFuncAttributes fa;
  e = cudaFuncGetAttributes(&fa, fn);
  if (e != cudaSuccess) return e;
  e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize,
                           optin - static_cast<int>(fa.sharedSizeBytes));
  if (e == cudaSuccess && used < kSlots / 4 * 3) {  // (beyond: raised again on each call)
    table[at] = Entry{fn, dev};
    ++used;
  }
  return e;
}

}  // namespace ep

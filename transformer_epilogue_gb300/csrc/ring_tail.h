// The end of a ring of shared-memory stages (tma_pipe.cuh's Ring): what a loader still
// has to wait for when it has nothing more to load.
#pragma once

#include <cstdint>

#ifdef __CUDACC__
#define EP_RING_FN __device__ __forceinline__
#else
#define EP_RING_FN inline
#endif

namespace ep {
namespace dev {

// f(stage, parity) of the last `uses` uses (at most one of each stage) of a ring that
// stands at its next item, in their order, until f says no.
template <typename R, typename F>
EP_RING_FN bool last_uses(R ring, int uses, F f) {
  if (ring.st < uses) {
    ring.st += ring.n;
    ring.phase ^= 1u;
  }
  ring.st -= uses;
  for (int i = 0; i < uses; ++i, ring.next())
    if (!f(ring.st, ring.phase)) return false;
  return true;
}

}  // namespace dev
}  // namespace ep

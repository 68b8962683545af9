// The waits that a ring of asynchronous copies owes before its block exits.
//
// Stage n of a ring of `depth` slots arms the "full" barrier of slot n % depth
// for the (n / depth)-th time, so its copy has landed once that barrier's phase
// n / depth is over: a wait by the parity of n / depth. The parity tells phase
// n / depth from the one before only while no later stage has armed the slot;
// that holds for the last min(issued, depth) stages, and every earlier one of
// a slot ended before the slot was armed again.
//
// A block that ends normally owes no wait: its MMAs have waited for every
// stage. One that gives up does, whichever role gave up: the role that issued
// the copies may have ended normally long before. So the drains follow the
// block's last barrier (no role arms anything after it, and the abort flag is
// final) and look at that flag, not at the issuing role's own result.
//
// No CUDA header: a host test compiles this file alone.
#pragma once
#include <cstdint>

#if defined(__CUDACC__)
#define MOE_RING_FN __device__ __forceinline__
#else
#define MOE_RING_FN inline
#endif

namespace moe {

// wait(slot, parity) for each of the last min(issued, depth) stages.
template <typename Wait>
MOE_RING_FN void drain_ring(uint32_t issued, uint32_t depth, Wait wait) {
  const uint32_t back = issued < depth ? issued : depth;
  for (uint32_t i = 1; i <= back; ++i) {
    const uint32_t n = issued - i;
    wait(n % depth, (n / depth) & 1u);
  }
}

}  // namespace moe

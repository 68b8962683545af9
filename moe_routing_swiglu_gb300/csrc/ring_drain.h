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
// Where threads go on after a give-up (rounds with barriers that every one has to
// reach), the role that arms the stages must stop by itself: the slot that was
// given up on still has its copy in flight and its phase open, so that to arm it
// again would be an arrival too many and a second copy into the same memory, and
// the drain's parity would be of another phase. Its own waits tell it that: it
// arms a slot only after its own wait for the stage before ended with the phase.
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

// What the arming role does with its own wait's result: `next`, the first row of
// the stage that it would arm next, passes `end` for good after a give-up.
MOE_RING_FN void issue_only_after(bool waited, uint32_t& next, uint32_t end) {
  if (!waited) next = end;
}

}  // namespace moe

// Which copies of the window and paged forward's K and V ring may still be in flight when
// its copying warps have stopped.  (Plain C++, so that the rule is tested on the CPU.)
#pragma once

#include <stdint.h>

#ifdef __CUDACC__
#define ELSAA_RING_FN __host__ __device__ inline
#else
#define ELSAA_RING_FN inline
#endif

namespace elsaa {

// Load i of the ring goes into slot i % slots; K's are the loads 0, 2, .., V's 1, 3, ..
// The warps stop on their own, so one may have started more loads than the other.
struct RingDrain {
  uint32_t slots, k, v;   // k, v: loads that K's and V's warp have started
  ELSAA_RING_FN uint32_t end() const { return 2 * (k > v ? k : v); }
  // The first load that can be the last of its slot: neither warp gets further than `slots`
  // loads past one that the products have not read, and those are read in order.
  ELSAA_RING_FN uint32_t begin() const {
    const uint32_t e = end();
    return e > 2 * slots + 2 ? e - 2 * slots - 2 : 0;
  }
  ELSAA_RING_FN bool started(uint32_t i) const { return i / 2 < (i & 1 ? v : k); }
  // Load i has to be awaited: it is its slot's last.  (One that another followed was read
  // before that, and its barrier's phase is over.)
  ELSAA_RING_FN bool open(uint32_t i) const { return started(i) && !started(i + slots); }
};

}  // namespace elsaa

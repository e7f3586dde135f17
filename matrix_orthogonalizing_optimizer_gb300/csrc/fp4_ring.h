// What is left of a ring of operand loads when a wait has run out: which of its barriers can still be waited for, and how.
// Host code too (no CUDA header), so that it can be run against a model of the barriers.
#pragma once

#include <stdint.h>

#if defined(__CUDACC__)
#define GNS_RING_FN __host__ __device__ inline
#else
#define GNS_RING_FN inline
#endif

namespace gns {

// The leading CTA of a group waits until every load that the group has issued has landed. The u-th slice of a CTA goes
// to stage u % stages; its barrier, the leader's, completes a phase with the leader's arrival, which announces the
// bytes of all CTAs of the group, and those bytes. own and other: the slices that the leader and its peer have issued
// (a group of one CTA: both its own). Each ran on its own until its own wait ran out, but not past a stage whose last
// contents both have seen used, so that only the last `stages` slices can be in flight.
//   ring.forgo(s)          takes back what the leader announced for its peer
//   ring.announce(s)       arrives, and announces the peer's bytes
//   ring.wait(s, parity)   waits, with a limit; false: it ran out
template <class Ring>
GNS_RING_FN bool settle_ring(Ring& ring, uint32_t own, uint32_t other, uint32_t stages) {
  const uint32_t most = own > other ? own : other;
  bool ok = true;
  for (uint32_t u = most > stages ? most - stages : 0u; u < most; ++u) {
    const uint32_t s = u % stages;
    if (u >= other) ring.forgo(s);
    if (u >= own) ring.announce(s);
    ok = ring.wait(s, (u / stages) & 1u) && ok;
  }
  return ok;
}

}  // namespace gns

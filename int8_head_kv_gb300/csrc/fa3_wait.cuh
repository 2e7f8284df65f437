// Bounded waiting on something that is tested again and again.
#pragma once

#include <stdint.h>

namespace fa3 {

enum class Waited { kDone, kStopped, kLate };

// Tests `done` until it holds, until `stopped` does, or until more than `limit` of `ticks` have passed.  Reading the
// clock takes longer than most waits last, and how long a test that fails takes is the hardware's choice (3.94 us for a
// suspended barrier test on a GB300, nanoseconds for one that returns at once), so neither each test reads the
// clock nor does a number of tests stand for a time: the clock is read every 256 tests, from the 256th on.
template <class Done, class Stopped, class Ticks>
__host__ __device__ __forceinline__ Waited bounded_wait(Done&& done, Stopped&& stopped, Ticks&& ticks, uint32_t limit) {
  uint32_t begin = 0;
#pragma unroll 1
  for (uint32_t i = 1;; ++i) {
    if (done()) return Waited::kDone;
    if ((i & 255u) == 0u) {
      if (stopped()) return Waited::kStopped;
      const uint32_t now = ticks();
      if (i == 256u) begin = now;
      if (now - begin > limit) return Waited::kLate;
    }
  }
}

}  // namespace fa3

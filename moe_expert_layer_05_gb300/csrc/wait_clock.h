// A bounded wait by a clock that need not be right every time.
//
// The GPU's nanosecond counter is 64 bits wide: a reading may be earlier than the last one, and a single one may be
// far off (its two halves taken on two sides of a carry are 4.3 s apart, twice the limit of a wait).  So the limit is
// eight laps, each from a reading to one that is later by an eighth of the limit or by anything more; after a step back
// the lap begins anew.  One wrong reading, the first one too, adds or takes one lap at most.
//
// (The loop around a lap keeps one reading and a count, as a single lap's would: with the time added up, or the laps
// counted, inside of it the attention's forward took 377 and 370 us for 359, 8192 rows, 32/8 heads of 128.)
#pragma once

#ifdef __CUDACC__
#define MOE_WAIT_CALL __device__ __forceinline__
#else
#define MOE_WAIT_CALL inline
#endif

namespace moe {

enum class Waited { kDone, kStopped, kOver };

// Until done(); gives up when stopped(), which is asked before the clock now() is read, after every `tests` tests, or
// when `limit` ns have passed.
template <unsigned tests, class Done, class Stopped, class Now>
MOE_WAIT_CALL Waited bounded_wait(Done done, Stopped stopped, Now now, unsigned long long limit) {
  constexpr unsigned kLaps = 8;
  unsigned laps = 0;
  do {
    const unsigned long long since = now();
    for (unsigned n = 1;; ++n) {
      if (done()) return Waited::kDone;
      if (n % tests == 0) {
        if (stopped()) return Waited::kStopped;
        const unsigned long long lap = now() - since;
        if (lap > limit / kLaps) {
          laps += static_cast<long long>(lap) > 0 ? 1u : 0u;
          break;
        }
      }
    }
  } while (laps < kLaps);
  return Waited::kOver;
}

}  // namespace moe

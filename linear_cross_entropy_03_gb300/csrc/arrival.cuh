// Finding the last CTA of a launch to finish, without memory that was zeroed before:
// a 64-bit word of (tag of the call, CTAs arrived) in the call's workspace.
#pragma once

#include <atomic>
#include <chrono>

#include <cuda_runtime.h>
#include <stdint.h>

namespace flce {
namespace {

constexpr int kArrivalBits = 24;  // of the count; the tag is above

// A tag that no recent call of this process used, and never 0.
inline unsigned long long next_arrival_tag() {
  static std::atomic<unsigned long long> counter{
      static_cast<unsigned long long>(std::chrono::steady_clock::now().time_since_epoch().count())};
  unsigned long long tag;
  do {
    tag = counter.fetch_add(1, std::memory_order_relaxed) << kArrivalBits;
  } while (tag == 0);
  return tag;
}

// By one thread of the launch as it starts: puts the tag on the word, so that the CTAs
// that arrive later need one addition each.  Nothing waits for it; if the swap fails, a
// CTA that has arrived already has put the tag there.
__device__ __forceinline__ void expect_arrivals(unsigned long long* word, unsigned long long tag) {
  const unsigned long long now = *reinterpret_cast<volatile unsigned long long*>(word);
  if (now >> kArrivalBits != tag >> kArrivalBits) atomicCAS(word, now, tag);
}

// By one thread of each of `ctas` CTAs, once its CTA's results are written: true in the
// one that arrives last, which then sees all of them (through loads that pass the
// first-level cache by, such as __ldcg).  The word may hold anything at first.  A CTA
// that finds another tag on it puts (tag, 1) there by compare-and-swap, unless another
// CTA was quicker; no CTA waits for one that has yet to run.  The last one leaves 0, so
// that a graph that replays the call with the same tag finds it unused.
__device__ __forceinline__ bool arrives_last(unsigned long long* word, unsigned long long tag, unsigned int ctas) {
  constexpr unsigned long long kCount = (1ull << kArrivalBits) - 1;
  __threadfence();
  unsigned long long old = atomicAdd(word, 1ull);
  if ((old & ~kCount) != tag) {
    unsigned long long now = old + 1;  // what this CTA's addition left
    // each turn after the first, another CTA has changed the word, which each does twice at most
    for (unsigned int turn = 0;; ++turn) {
      if (turn > 2 * ctas) return false;
      if ((now & ~kCount) == tag) {
        old = atomicAdd(word, 1ull);
        break;
      }
      const unsigned long long was = atomicCAS(word, now, tag | 1ull);
      if (was == now) {
        old = tag;
        break;
      }
      now = was;
    }
  }
  if ((old & kCount) + 1 != ctas) return false;
  *word = 0;
  __threadfence();
  return true;
}

}  // namespace
}  // namespace flce

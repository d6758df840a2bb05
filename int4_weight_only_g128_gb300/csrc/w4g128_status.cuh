// The status word of an operator call (byte 0 of its workspace's first 64-bit
// word, as w4g128_workspace_status reads it), tagged with the launch that wrote
// it: a CTA that fails and the CTA that clears the word may come in any order,
// without a launch that zeroes it.
#pragma once
#include <cstdint>

#include "w4g128_ptx.cuh"

namespace w4g128 {

// The upper 56 bits of this launch's words: its grid number through an odd
// multiplier, so that leftover workspace bytes are unlikely to look like it.
__device__ __forceinline__ unsigned long long launch_tag() {
  unsigned long long g;
  asm volatile("mov.u64 %0, %%gridid;" : "=l"(g));
  return ((g + 1ull) * 0x9E3779B97F4A7C15ull) & ~0xFFull;
}

// One thread of the launch: the word says "no error" unless a thread of this
// launch has failed.
__device__ __forceinline__ void status_clear(unsigned long long* word) {
  const unsigned long long tag = launch_tag();
  unsigned long long cur = ld_relaxed_u64(word);
  while ((cur & ~0xFFull) != tag) {
    const unsigned long long prev = atomicCAS(word, cur, tag);
    if (prev == cur) return;
    cur = prev;
  }
}

// The first failure of this launch stays.
__device__ __forceinline__ void status_error(unsigned long long* word, unsigned code) {
  const unsigned long long tag = launch_tag();
  unsigned long long cur = ld_relaxed_u64(word);
  while ((cur & ~0xFFull) != tag || (cur & 0xFFull) == 0ull) {
    const unsigned long long prev = atomicCAS(word, cur, tag | code);
    if (prev == cur) return;
    cur = prev;
  }
}

}  // namespace w4g128

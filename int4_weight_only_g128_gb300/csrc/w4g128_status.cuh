// Errors that an operator's kernels find in device memory, on their way to the
// status word (the first word of the workspace, as w4g128_workspace_status
// reads it).  Any CTA of the first kernel may note one in a pending word; the
// last kernel of the call moves it to the status word and leaves "none" behind.
// The pending word needs no zeroing: without its mark it counts as "none".  (A
// tag of the launch in its place fails in a CUDA graph, whose replays all have
// the same grid number.)
#pragma once
#include <cstdint>

#include "w4g128_ptx.cuh"

namespace w4g128 {

constexpr unsigned long long kPendingMark = 0x50656E64696E6700ull;  // "Pending" above the code's byte

// The first error of a call stays.
__device__ __forceinline__ void note_error(unsigned long long* pending, unsigned code) {
  unsigned long long cur = ld_relaxed_u64(pending);
  while ((cur & ~0xFFull) != kPendingMark || (cur & 0xFFull) == 0ull) {
    const unsigned long long prev = atomicCAS(pending, cur, kPendingMark | code);
    if (prev == cur) return;
    cur = prev;
  }
}

// One thread of the last kernel.
__device__ __forceinline__ void publish_errors(unsigned long long* status, unsigned long long* pending) {
  const unsigned long long v = ld_relaxed_u64(pending);
  st_relaxed_u64(status, (v & ~0xFFull) == kPendingMark ? v & 0xFFull : 0ull);
  st_relaxed_u64(pending, kPendingMark);
}

}  // namespace w4g128

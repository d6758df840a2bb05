// Division by a value that the host knows: the compiler's divide by a variable
// is a chain of some 30 instructions, and a call that takes microseconds has
// dozens of them before its first load.
#pragma once
#include <cstdint>

namespace w4g128 {

struct Divisor {
  unsigned d, m;  // and 2^32 over it
};
inline Divisor divisor(int d) {
  return {static_cast<unsigned>(d), d == 1 ? ~0u : static_cast<unsigned>((1ull << 32) / d)};
}

// a / d for a >= 0: m falls short of 2^32 / d by less than 1, so that a m / 2^32
// falls short of a / d by less than 1.
__device__ __forceinline__ int operator/(int a, Divisor by) {
  const unsigned q = __umulhi(static_cast<unsigned>(a), by.m);
  return static_cast<int>(q + (static_cast<unsigned>(a) - q * by.d >= by.d ? 1u : 0u));
}
__device__ __forceinline__ int operator%(int a, Divisor by) { return a - (a / by) * static_cast<int>(by.d); }

}  // namespace w4g128

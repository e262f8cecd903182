// The row of x that an entry of an order leads to: the entry over `gather`, without a
// division. Plain C++, on the host and in kernels alike.
#pragma once

#include <stdint.h>

namespace mxg {

// floor(o / gather) for every o below 2^31 and gather 2..32: with 2^(shift + 1) the least
// power of two from gather on and m = floor(2^(32 + shift) / gather) + 1 < 2^32, o m
// exceeds 2^(32 + shift) o / gather by at most o, which is below 2^(32 + shift) / gather
// since that is at least 2^31: not enough to reach the next whole quotient.
struct GatherQuotient {
  uint32_t m, shift;
};

constexpr GatherQuotient gather_quotient(int32_t gather) {
  uint32_t shift = 0;
  while ((2 << shift) < gather) ++shift;
  return {gather < 2 ? 0u : (uint32_t)((((uint64_t)1 << (32 + shift)) / (uint32_t)gather) + 1),
          shift};
}

// (For an o from 2^31 on, which leads to no row, any number.)
constexpr uint32_t over_gather(uint32_t o, const GatherQuotient& q) {
  return (uint32_t)((uint64_t)o * q.m >> 32) >> q.shift;
}

}  // namespace mxg

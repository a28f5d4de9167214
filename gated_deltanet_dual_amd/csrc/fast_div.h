// fast_div.h -- division by a number that is the same for a whole launch.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace flare {

// n / d for 0 <= n < 2^31 and 1 <= d < 2^31 as a product: with s = ceil(log2 d) and
// m = floor(2^(31 + s) / d) + 1 (below 2^32), m d = 2^(31 + s) + e with 0 < e <= d <=
// 2^s, so that n m / 2^(31 + s) lies above n / d by less than n / 2^31 / d < 1 / d:
// never at or beyond the next whole number.
struct FastDiv {
  uint32_t m;
  int shift;
};
inline FastDiv make_fast_div(int32_t d) {
  int s = 0;
  while (((int64_t)1 << s) < d) ++s;
  return {(uint32_t)(((uint64_t)1 << (31 + s)) / (uint32_t)d + 1), 31 + s};
}
__device__ __forceinline__ int32_t fast_div(uint32_t n, const FastDiv &d) {
  return (int32_t)(((uint64_t)n * d.m) >> d.shift);
}

}  // namespace flare

// Division by a cache's page size.
#pragma once

#include <stdint.h>

namespace rmk {

// x / P = x * mul >> shift for 0 <= x < 2^31, P = 1..1024 (2^shift = 2^31 * the
// power of two from P on: the multiplier fits 32 bits and exceeds 2^shift / P
// by less than 1, so the quotient is too large by less than 1 / P)
struct PageDiv {
  uint32_t mul;
  int shift, P;
  __device__ __forceinline__ int floor(int x) const {
    return static_cast<int>((static_cast<unsigned long long>(static_cast<uint32_t>(x)) * mul) >> shift);
  }
  __device__ __forceinline__ int ceil(int x) const {
    const int q = floor(x);
    return q + (x - q * P > 0);
  }
};
inline PageDiv page_div(int page_size) {
  PageDiv div;
  div.P = page_size;
  div.shift = 31;
  while ((1 << (div.shift - 31)) < page_size) ++div.shift;
  div.mul = static_cast<uint32_t>(((1ull << div.shift) + page_size - 1) / page_size);
  return div;
}

}  // namespace rmk

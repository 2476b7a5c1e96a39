// Division by a divisor known at launch, as a product: for v >= 1 and n < 2^31, with s = ceil(log2 v) and
// m = floor(2^32 (2^s - v) / v) + 1,  n / v = (floor(m n / 2^32) + n) >> s  (Granlund and Montgomery,
// "Division by invariant integers using multiplication").
#pragma once
#include <cstdint>

namespace gb300 {

struct FastDiv {
  uint32_t v, mul, shift;
};

inline FastDiv fast_div(uint32_t v) {
  FastDiv d{v, 0, 0};
  while ((1ull << d.shift) < v) ++d.shift;
  d.mul = (uint32_t)((((1ull << d.shift) - v) << 32) / v + 1);
  return d;
}

#ifdef __CUDACC__
__device__ __forceinline__ uint32_t operator/(uint32_t n, const FastDiv& d) {
  return (__umulhi(d.mul, n) + n) >> d.shift;
}
#endif

}  // namespace gb300

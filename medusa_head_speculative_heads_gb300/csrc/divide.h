// Division by a number that is fixed before a launch, as one product.
#pragma once

#include <stdint.h>

#ifdef __CUDACC__
#define MEDUSA_HD __host__ __device__ __forceinline__
#else
#define MEDUSA_HD inline
#endif

namespace medusa {

// 2^31 / n, rounded up (n = 1 included, which 32 bits of fraction would not hold).
MEDUSA_HD uint32_t reciprocal(uint32_t n) { return ((1u << 31) + n - 1) / n; }

// floor(x / n), x n < 2^31, inv = reciprocal(n): inv = 2^31 / n + e with 0 <= e < 1, so
// 2 x inv 2^-32 is x / n and less than 1 / n more.  0 for inv = 0.
MEDUSA_HD uint32_t quotient(uint32_t x, uint32_t inv) {
#ifdef __CUDA_ARCH__
  return __umulhi(2 * x, inv);
#else
  return (uint32_t)(((uint64_t)(2 * x) * inv) >> 32);
#endif
}

}  // namespace medusa

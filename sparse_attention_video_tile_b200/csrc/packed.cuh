// packed.cuh - the packed fp32 product, beside ptx.cuh's sum and fma.
#pragma once

#include <cstdint>

namespace sta {
namespace ptx {

// a * b on both halves (round to nearest even)
__device__ __forceinline__ uint64_t mul_f32x2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

}  // namespace ptx
}  // namespace sta

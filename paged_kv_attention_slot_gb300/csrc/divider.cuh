#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace pkv {

// Quotients by a number that is usually a power of two.
struct Divider {
  int32_t d, shift;  // shift >= 0: d == 1 << shift
  __device__ __forceinline__ uint32_t div(uint32_t x) const { return shift >= 0 ? x >> shift : x / (uint32_t)d; }
  __device__ __forceinline__ uint32_t div64(int64_t x) const {  // x >= 0, quotient below 2^32
    if (shift >= 0) return (uint32_t)(x >> shift);
    return x >> 32 ? (uint32_t)(x / d) : (uint32_t)x / (uint32_t)d;
  }
};
inline Divider divider(int32_t d) {
  int s = 0;
  while ((1 << s) < d && s < 30) ++s;
  return Divider{d, (1 << s) == d ? s : -1};
}

}  // namespace pkv

// Pairs of 32-bit values and the instructions that work on both at once.
#pragma once

#include <stdint.h>

namespace bw {

using pair_t = uint64_t;
__device__ __forceinline__ pair_t pair(float lo, float hi) {
  return static_cast<uint64_t>(__float_as_uint(hi)) << 32 | __float_as_uint(lo);
}
__device__ __forceinline__ float first(pair_t x) { return __uint_as_float(static_cast<uint32_t>(x)); }
__device__ __forceinline__ float second(pair_t x) { return __uint_as_float(static_cast<uint32_t>(x >> 32)); }
__device__ __forceinline__ pair_t mul(pair_t a, pair_t b) {
  pair_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ pair_t fma(pair_t a, pair_t b, pair_t c) {
  pair_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ pair_t add(pair_t a, pair_t b) {
  pair_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
// a - b, rounded once as a subtraction is
__device__ __forceinline__ pair_t sub(pair_t a, pair_t b) { return fma(b, pair(-1.f, -1.f), a); }

}  // namespace bw

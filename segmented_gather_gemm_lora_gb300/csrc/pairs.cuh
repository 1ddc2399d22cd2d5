// Pairs of fp32 values: two operations in one instruction, and sums that keep what
// their rounding leaves out.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace lora {

// Two fp32 operations in one instruction.
__device__ __forceinline__ uint64_t pair_of(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ void split(uint64_t p, float& a, float& b) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(p));
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}

// An fp32 sum with what its rounding left out (hi + lo, |lo| within half a unit of
// hi): sums of hundreds of terms as exact as in doubles, which the GPU adds two a
// clock an SM.
struct Pair32 {
  float hi, lo;
};
__device__ __forceinline__ Pair32 two_sum(float a, float b) {
  const float s = __fadd_rn(a, b), t = __fsub_rn(s, a);
  return Pair32{s, __fadd_rn(__fsub_rn(a, __fsub_rn(s, t)), __fsub_rn(b, t))};
}
__device__ __forceinline__ Pair32 add_pair(const Pair32& x, const Pair32& y) {
  const Pair32 h = two_sum(x.hi, y.hi);
  // an infinite or NaN sum has nothing left out
  const float lo = fabsf(h.hi) < __int_as_float(0x7f800000) ? h.lo + (x.lo + y.lo) : 0.f;
  const float s = __fadd_rn(h.hi, lo);
  return Pair32{s, fabsf(s) < __int_as_float(0x7f800000) ? __fsub_rn(lo, __fsub_rn(s, h.hi)) : 0.f};
}

}  // namespace lora

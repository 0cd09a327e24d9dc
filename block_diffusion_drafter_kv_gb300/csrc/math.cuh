// Arithmetic that the target-side kernels share.
#pragma once

#include "ptx.cuh"

namespace dfl {

// A list of T units cut evenly over G CTAs (G <= T: none is empty): the first unit of CTA c, and the
// CTA whose range holds unit u. (A 64-bit division is a hundred instructions in a chain: products
// that fit take the 32-bit one.)
static __device__ __noinline__ long long wide_quotient(long long a, long long b) { return a / b; }
DEV long long quotient(long long a, long long b) {
  return static_cast<unsigned long long>(a | b) < (1ull << 32) ? static_cast<uint32_t>(a) / static_cast<uint32_t>(b) : wide_quotient(a, b);
}
DEV long long range_begin(long long c, long long T, int G) { return quotient(c * T, G); }
DEV int cta_of(long long u, long long T, int G) { return static_cast<int>(quotient((u + 1) * G - 1, T)); }

// 2^x by the multi-function unit (relative error about 2^-22).
DEV float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// Two fp32 operations in one instruction.
DEV float2 fma2(float2 a, float2 b, float2 c) {
  float2 d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;"
      : "=l"(*reinterpret_cast<unsigned long long*>(&d))
      : "l"(*reinterpret_cast<unsigned long long*>(&a)), "l"(*reinterpret_cast<unsigned long long*>(&b)),
        "l"(*reinterpret_cast<unsigned long long*>(&c)));
  return d;
}
DEV float2 add2(float2 a, float2 b) {
  float2 d;
  asm("add.rn.f32x2 %0, %1, %2;"
      : "=l"(*reinterpret_cast<unsigned long long*>(&d))
      : "l"(*reinterpret_cast<unsigned long long*>(&a)), "l"(*reinterpret_cast<unsigned long long*>(&b)));
  return d;
}

}  // namespace dfl

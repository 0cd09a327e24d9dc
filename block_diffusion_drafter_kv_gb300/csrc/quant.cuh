// The 8-bit rows of a paged cache. A row (one position, one KV head, K or V) is e4m3 values times
// 2^e, with e the least whole number for which max |x| <= 448 * 2^e, between -40 and 40: a power of
// two, so that scaling is exact and each value is rounded once. Its scale byte is e + 127; 255 marks
// a row with an infinity, a NaN or a value past 448 * 2^40: NaN in every column.
// Scale bytes lie [n_pages][nkv][2][64]: K's, then V's 64 positions of a page, 128 bytes a head.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "ptx.cuh"
#include "target.h"

namespace dfl {

constexpr int kScaleBias = 127, kScaleNan = 255, kScaleMax = 40;
constexpr uint32_t kLargest8 = ((127 + 8 + kScaleMax) << 23) | 0x600000;  // bits of 448 * 2^40

// Two fp32 values as e4m3, the first in the low byte.
DEV uint32_t to_e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}
// Two e4m3 values as fp16 (exact).
DEV __half2 from_e4m3x2(uint32_t v) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(static_cast<uint16_t>(v)));
  return *reinterpret_cast<const __half2*>(&r);
}
DEV float exponent_value(int e) { return __uint_as_float(static_cast<uint32_t>(e + 127) << 23); }  // 2^e, -126 <= e <= 127
// What a scale byte stands for: a NaN for 255.
DEV float scale_value(uint32_t byte) {
  return __uint_as_float(byte == kScaleNan ? 0x7fc00000u : max(byte, 1u) << 23);
}
// The scale byte of a row whose largest magnitude has these fp32 bits.
DEV int scale_byte(uint32_t top) {
  if (top > kLargest8) return kScaleNan;
  const int e = static_cast<int>(top >> 23) - 127 - 8 + ((top & 0x7fffffu) > 0x600000u);
  return max(e, -kScaleMax) + kScaleBias;
}
DEV size_t scale_index(int slot, int nkv, int head, int which) {
  return ((static_cast<size_t>(slot / kPagePos) * nkv + head) * 2 + which) * kPagePos + slot % kPagePos;
}

}  // namespace dfl

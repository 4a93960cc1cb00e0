// The arithmetic of the 8-bit token codes: codes = rint(127 x / max|x|), half
// to even.  127 x is exact in fp32 (15 significant bits), and the correctly
// rounded quotient lies on the same side of every border n + 1/2 as the exact
// one: the border is representable, so rounding cannot cross it, and a quotient
// that is not a border differs from it by at least 2^-17 (127 x and the
// maximum are integers of 15 and 8 bits times powers of two at most 2^8
// apart), more than the half ulp 2^-18 of values up to 127.
#pragma once

#include "moe_internal.h"

namespace moe {

// Bits of the largest magnitude of eight bf16 values; infinities and NaN lie
// above every finite value's.
__device__ __forceinline__ uint32_t max_magnitude(u32x4_t v) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t lo = (v[i] << 16) & 0x7FFFFFFFu, hi = v[i] & 0x7FFF0000u;
    m = m > lo ? m : lo;
    m = m > hi ? m : hi;
  }
  return m;
}

// Codes of eight bf16 values of a row whose largest magnitude is big; zeros
// where that is zero, infinite or NaN.
__device__ __forceinline__ uint64_t quantize8(u32x4_t v, float big) {
  uint32_t w[2] = {0, 0};
  if (big > 0.0f && big < __builtin_inff()) {
    const float down = big > 0x1p120f ? 0x1p-8f : 1.0f;  // keeps 127 x finite; exact where a code is not 0
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float f = i & 1 ? bf16_hi(v[i >> 1]) : bf16_lo(v[i >> 1]);
      const int q = (int)rintf(127.0f * (f * down) / (big * down));
      w[i >> 2] |= ((uint32_t)q & 0xFFu) << (8 * (i & 3));
    }
  }
  return (uint64_t)w[1] << 32 | w[0];
}

}  // namespace moe

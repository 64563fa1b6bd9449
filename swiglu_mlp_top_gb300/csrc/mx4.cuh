// 4 bits to bf16.  With a nibble's sign at bit 15 and its exponent and fraction
// at bits 8..6, the bf16 is the value times 2^-126, subnormals included; one
// multiplication by 2^(126 + e) makes it the value times its scale, exactly.
#pragma once

#include "mm_device.cuh"

namespace mm {

__device__ __forceinline__ uint32_t bf16x2_mul(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

// Eight values of a word of codes times the scale, as four pairs of bf16.
// TWO: 2^126 (0x7e80) and the scale apart, where their product overflows.
template <bool TWO>
__device__ __forceinline__ uint4 e2m1_bf16(uint32_t codes, uint32_t f1, uint32_t f2) {
  const uint32_t even = codes & 0x0f0f0f0fu, odd = (codes >> 4) & 0x0f0f0f0fu;
  uint32_t v[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    // nibbles 2i and 2i + 1 in the two halves (selector bit 3: the sign of a byte below 16, zero)
    uint32_t p;
    asm("prmt.b32 %0, %1, %2, %3;" : "=r"(p) : "r"(even), "r"(odd), "r"(0x8080 | i | (4 + i) << 8));
    v[i] = bf16x2_mul((p * 0x1040u) & 0x81c081c0u, f1);
    if constexpr (TWO) v[i] = bf16x2_mul(v[i], f2);
  }
  return make_uint4(v[0], v[1], v[2], v[3]);
}

// The factors of a scale byte, in both halves: 2^126 * 2^(byte - 127) and 1, or
// 2^126 and the scale where their product overflows (byte > 128).  255 stands
// for NaN, 0 is 2^-127.
__device__ __forceinline__ void mx4_factors(uint32_t byte, uint32_t& f1, uint32_t& f2) {
  f1 = byte <= 128u ? (byte + 126u) << 7 : 0x7e80u;
  f2 = byte == 255u ? 0x7fffu : byte <= 128u ? 0x3f80u : byte << 7;
  f1 |= f1 << 16;
  f2 |= f2 << 16;
}

}  // namespace mm

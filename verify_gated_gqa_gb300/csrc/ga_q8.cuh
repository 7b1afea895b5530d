// The 8-bit cache rows: e4m3 codes with a power-of-two scale for each block of 32 tokens and head.
//
// A power of two costs e4m3 nothing (its relative step is the same in every binade, down to the
// smallest normal code) and buys three things: a block's exponent can grow as tokens are added and
// the codes it holds move with it exactly, until they fall under 2^-6; widened values are bf16
// values; and the attention applies a scale by adding to an exponent.
#pragma once
#include <cstdint>

#include "ga_internal.h"

namespace ga {

constexpr int kQ8Block = GA_Q8_BLOCK_TOKENS;
constexpr int kQ8RowBytes = GA_Q8_ROW_BYTES;
constexpr int kQ8MinExp = -32, kQ8MaxExp = 31;   // stored as e + 32 in six bits

__device__ __forceinline__ int q8_exp(uint32_t byte) { return (int)(byte & 63u) + kQ8MinExp; }
__device__ __forceinline__ float pow2i(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }

// The largest magnitude of 8 bf16 values, as its bits (ordered as the magnitudes are).
__device__ __forceinline__ uint32_t top_of(const uint4& x) {
  const uint32_t w[4] = {x.x & 0x7FFF7FFFu, x.y & 0x7FFF7FFFu, x.z & 0x7FFF7FFFu, x.w & 0x7FFF7FFFu};
  const uint32_t m = __vmaxu2(__vmaxu2(w[0], w[1]), __vmaxu2(w[2], w[3]));
  uint32_t top = max(m & 0xFFFFu, m >> 16);
  if (top > 0x7F80u) {   // a NaN counts as 0
    top = 0u;
    for (int i = 0; i < 4; ++i) {
      const uint32_t lo = w[i] & 0xFFFFu, hi = w[i] >> 16;
      if (lo <= 0x7F80u) top = max(top, lo);
      if (hi <= 0x7F80u) top = max(top, hi);
    }
  }
  return top;
}
// Two codes, to nearest even, saturating at +-448 (lo in bits 0..7); a NaN gives the code 0x7F.
__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}
// The values of the codes in bits 0..15 as a pair of halves, exactly.
__device__ __forceinline__ uint32_t e4m3x2_f16x2(uint32_t codes) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"((uint16_t)codes));
  return r;
}
__device__ __forceinline__ float2 f16x2_f32(uint32_t h) {
  float lo, hi;
  asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\tcvt.f32.f16 %0, l;\n\tcvt.f32.f16 %1, h;\n\t}"
      : "=f"(lo), "=f"(hi)
      : "r"(h));
  return make_float2(lo, hi);
}

}  // namespace ga

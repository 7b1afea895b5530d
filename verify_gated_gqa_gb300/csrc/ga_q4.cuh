// 4-bit cache rows ("q4"): the format and its device conversions.
//
// A row is the 256 values of one (token, KV head), in 16 groups of 16 dims. A group's scale is
// a = fp32(max|x| / 7), clamped to [2^-20, 3840] and rounded to 4 significant bits (nearest,
// ties to even), s = 2^(E - 20) (1 + m / 8), stored as the byte 8 E + m (E 0..31, m 0..7: no
// sign and no subnormals, so the byte needs no second scale beside it for rows of any usual
// magnitude). A value's code is clamp(rne(x / s), -8, 7) + 8, four bits. The widened value is
// (code - 8) s: at most 4 x 4 significant bits, so it is a bf16 value exactly and widening
// rounds nothing. Every pair of code and scale bytes is a finite value.
//
// Eight dims of a row make a 32-bit little-endian word: nibble p < 4 is dim 2p, nibble 4 + p
// is dim 2p + 1, so (w >> 4p) & 0x000F000F holds the codes of the pair (2p, 2p + 1) in the
// halves of a register (integer to float through the exponent field, two values an operation: the
// published way of widening low-bit weights, Kim et al., "Who Says Elephants Can't Run", 2022). OR-ed
// into 0x4300 (bf16 128, whose last place is 1), a code n becomes
// the bf16 value 128 + n, and one fused multiply-add, (128 + n) s - 136 s, gives (n - 8) s
// with no rounding (136 s = 17 (8 + m) 2^E' has at most 8 significant bits).
#pragma once
#include <cstdint>

namespace ga {

constexpr int kQ4Group = 16;                       // values per scale
constexpr int kQ4RowBytes = 128;                   // code bytes per row of 256 values
constexpr int kQ4ScaleBytes = 256 / kQ4Group;      // scale bytes per row
constexpr int kQ4ExpBias = 20;
constexpr float kQ4MinScale = 9.5367431640625e-07f;   // 2^-20
constexpr float kQ4MaxScale = 3840.0f;                // 15/8 x 2^11

__device__ __forceinline__ uint32_t q4_fma_bf16x2(uint32_t a, uint32_t b, uint32_t c) {
  uint32_t r;
  asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(a), "r"(b), "r"(c));
  return r;
}
__device__ __forceinline__ uint32_t q4_mul_bf16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

// A group's multiplier pair: (s, s) and (-136 s, -136 s) as bf16.
struct Q4Scale {
  uint32_t s, off;
};
// From the byte b (0..255): exponent and mantissa line up with bf16's by a shift of 4.
__device__ __forceinline__ Q4Scale q4_scale(uint32_t b) {
  Q4Scale q;
  q.s = b * 0x00100010u + (((127u - kQ4ExpBias) << 7) * 0x00010001u);
  q.off = q4_mul_bf16x2(q.s, 0xC308C308u);   // x -136, exact
  return q;
}

// The pair of codes at nibble p of both halves of w as bf16 128 + n: one shift and one
// three-input logic operation (the compiler by itself makes the AND and the OR two).
__device__ __forceinline__ uint32_t q4_codes(uint32_t w, int p) {
  uint32_t r;
  asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(r) : "r"(w >> (4 * p)), "r"(0x000F000Fu), "r"(0x43004300u));
  return r;
}
// The eight bf16 values of one word, in dim order: two per register.
__device__ __forceinline__ void q4_widen(uint32_t w, Q4Scale q, uint32_t (&o)[4]) {
#pragma unroll
  for (int p = 0; p < 4; ++p) {
    o[p] = q4_fma_bf16x2(q4_codes(w, p), q.s, q.off);
  }
}

}  // namespace ga

// 4-bit cache rows in paged pools: storing rows of keys and values by slot, and widening them
// back to bf16 (the format is in ga_q4.cuh). Pools are head-major inside a page,
// [n_pages][2][page_size][128] code bytes and [n_pages][2][page_size][16] scale bytes, so the
// attention reads a key tile of one KV head as one contiguous run. Slot x of a pool is
// position x % page_size of page x / page_size, the same for both heads.
//
// 16 lanes per row, one 16-value group per lane, so a group's maximum needs no exchange between
// lanes and a row's reads and writes are contiguous runs. Both kernels are bound by the bytes they
// move (2,624 a token each), storing by its instructions nearly as much: 65,536 tokens stored and
// widened by two calls in 54 us of GPU time, 6.3 TB/s; 8,191 in 8.5. A thread takes the same group
// of a token's four rows (two heads of K and of V), all four in flight before the first is used
// and the slot looked up and divided once for them; with few tokens, of one row.
#include <cuda_bf16.h>

#include "ga_internal.h"
#include "ga_q4.cuh"
#include "ga_sm100.cuh"

namespace ga {
namespace {

constexpr int kRowThreads = 16;         // one 16-value group each
constexpr int kTokRows = 2 * kKvHeads;  // K heads 0, 1, V heads 0, 1
constexpr int kBlockThreads = 256;

// Pool row of head 0 of a slot, or -1: a negative slot (the token is not stored) or one outside
// the pool (recorded in the status word). Head 1's is page_size on.
__device__ __forceinline__ long long pool_row(const Kv4Args& a, long long slot) {
  if (slot < 0) return -1;
  if (slot >= a.n_slots) {
    atomicCAS(a.status, 0, (int)kDevBadPage);
    return -1;
  }
  // pages of 32 d slots: slot / 32 / d by one multiplication, exact below 2^25 (Kv4Args)
  const unsigned page = (unsigned)(((unsigned long long)((unsigned)slot >> 5) * a.page_mul) >> a.page_shift);
  return (long long)page * (kKvHeads * a.page_size) + ((unsigned)slot - page * (unsigned)a.page_size);
}

// A thread's place: group g of rows r0 .. r0 + kRows - 1 of token tok.
template <int kRows>
struct Place {
  int g, r0;
  long long tok;
  __device__ __forceinline__ Place() {
    constexpr int kPer = kTokRows / kRows;   // threads of a group of a token
    g = threadIdx.x % kRowThreads;
    r0 = threadIdx.x / kRowThreads % kPer * kRows;
    tok = (long long)blockIdx.x * (kBlockThreads / kRowThreads / kPer) + threadIdx.x / (kRowThreads * kPer);
  }
  __device__ __forceinline__ long long row(const Kv4Args& a) const {
    if (tok >= a.n_tok) return -1;
    return pool_row(a, a.slots ? (long long)__ldg(a.slots + tok) : tok);
  }
};

// The scale byte of a group whose largest magnitude is amax (an infinite one takes the
// largest scale). The division is correctly rounded, and a bf16 maximum cannot put fp32(a/7)
// on a rounding boundary of the scale unless a/7 itself is there, so the byte is the one of
// the exact quotient.
__device__ __forceinline__ uint32_t scale_byte(float amax) {
  const float a = fminf(fmaxf(__fdiv_rn(amax, 7.0f), kQ4MinScale), kQ4MaxScale);
  uint32_t u = __float_as_uint(a);
  u = (u + 0x7FFFFu + ((u >> 20) & 1u)) >> 20;   // 3 mantissa bits, ties to even
  return u - ((127u - kQ4ExpBias) << 3);
}
__device__ __forceinline__ float scale_of(uint32_t byte) {
  return __uint_as_float((byte + ((127u - kQ4ExpBias) << 3)) << 20);
}

// Codes without a division each. With x = X 2^a (X < 256) and s = S 2^b (8 <= S <= 15), a
// quotient that is not on a half is at least 1/960 from the nearest one (for quotients of 0.5 and
// more; smaller ones round to 0), while x times the reciprocal is within 2^-19 of it. One
// multiply-add onto 1.5 x 2^11 rounds that product to a multiple of 2^-12: a quotient on a
// half comes out on it exactly, and none is carried to or past one. One addition more rounds to
// the integer, ties to even, in the low bits of the sum.
constexpr float kSnap = 1.5f * 2048.0f, kInt = 1.5f * 8388608.0f + 8.0f - kSnap;
__device__ __forceinline__ uint64_t pack_f32x2(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ uint64_t add_f32x2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t fma_f32x2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}

// One group of 16 values (pairs in xw): its scale byte and its two code words.
__device__ __forceinline__ uint32_t quantize_group(const uint32_t (&xw)[8], uint32_t (&w)[2]) {
  // magnitudes of bf16 values are ordered as their bit patterns; NaNs come last
  uint32_t m = xw[0] & 0x7FFF7FFFu;
#pragma unroll
  for (int j = 1; j < 8; ++j) m = __vmaxu2(m, xw[j] & 0x7FFF7FFFu);
  const uint32_t top = max(m & 0xFFFFu, m >> 16);
  if (top <= 0x46D2u) {   // up to 7 x 3840: no code saturates
    const uint32_t byte = scale_byte(__uint_as_float(top << 16));
    const float inv = __fdividef(1.0f, scale_of(byte));
    const uint64_t inv2 = pack_f32x2(inv, inv), snap = pack_f32x2(kSnap, kSnap),
                   whole = pack_f32x2(kInt, kInt);
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      uint32_t acc = 0u;
#pragma unroll
      for (int j = 0; j < 4; ++j) {   // dims 2j and 2j + 1: nibbles j and 4 + j
        const uint32_t v = xw[4 * k + j];
        const uint64_t x = pack_f32x2(__uint_as_float(v << 16), __uint_as_float(v & 0xFFFF0000u));
        const uint64_t q = add_f32x2(fma_f32x2(x, inv2, snap), whole);
        // the sums' low bits hold code and constant; the constants are taken off below
        acc += (uint32_t)q * (1u << (4 * j)) + (uint32_t)(q >> 32) * (1u << (4 * j + 16));
      }
      w[k] = acc - 0x4B400000u * 0x11111111u;
    }
    return byte;
  }
  // saturating values, infinities and NaNs (which count as 0), one by one
  float v[kQ4Group], amax = 0.f;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    v[2 * j] = __uint_as_float(xw[j] << 16);
    v[2 * j + 1] = __uint_as_float(xw[j] & 0xFFFF0000u);
    amax = fmaxf(amax, fmaxf(fabsf(v[2 * j]), fabsf(v[2 * j + 1])));   // NaN is passed over
  }
  const uint32_t byte = scale_byte(amax);
  const float s = scale_of(byte);
  w[0] = w[1] = 0u;
#pragma unroll
  for (int j = 0; j < kQ4Group; ++j) {
    const float q = fminf(fmaxf(rintf(__fdiv_rn(v[j], s)), -8.0f), 7.0f);
    const uint32_t code = v[j] != v[j] ? 8u : (uint32_t)((int)q + 8);
    const int d = j & 7;
    w[j >> 3] |= code << (4 * ((d >> 1) + 4 * (d & 1)));
  }
  return byte;
}

// 32 bytes of a row by one lane: one load where every row is 32-byte aligned, else two.
__device__ __forceinline__ void load_group(const uint16_t* p, bool whole, uint32_t (&x)[8]) {
  if (whole) {
    asm volatile("ld.global.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=r"(x[0]), "=r"(x[1]), "=r"(x[2]), "=r"(x[3]), "=r"(x[4]), "=r"(x[5]), "=r"(x[6]),
                   "=r"(x[7])
                 : "l"(p));
    return;
  }
  const uint4 x0 = __ldg(reinterpret_cast<const uint4*>(p));
  const uint4 x1 = __ldg(reinterpret_cast<const uint4*>(p) + 1);
  x[0] = x0.x; x[1] = x0.y; x[2] = x0.z; x[3] = x0.w;
  x[4] = x1.x; x[5] = x1.y; x[6] = x1.z; x[7] = x1.w;
}

template <int kRows>
__global__ void __launch_bounds__(kBlockThreads) quantize_q4_kernel(
    const __grid_constant__ Kv4Args a) {
  const Place<kRows> at;
  uint32_t xw[kRows][8];
  if (at.tok < a.n_tok) {   // the rows do not wait for the slot
#pragma unroll
    for (int k = 0; k < kRows; ++k) {
      const int r = at.r0 + k;
      const uint16_t* x = r < kKvHeads ? a.k + at.tok * a.ld_k : a.v + at.tok * a.ld_v;
      load_group(x + r % kKvHeads * kDim + at.g * kQ4Group, a.in32, xw[k]);
    }
  }
  const long long row0 = at.row(a);
  if (row0 < 0) return;
#pragma unroll
  for (int k = 0; k < kRows; ++k) {
    const int r = at.r0 + k;
    const long long row = row0 + r % kKvHeads * a.page_size;
    uint32_t w[2];
    const uint32_t byte = quantize_group(xw[k], w);
    uint8_t* codes = r < kKvHeads ? a.k_codes : a.v_codes;
    uint8_t* scales = r < kKvHeads ? a.k_scales : a.v_scales;
    *reinterpret_cast<uint2*>(codes + row * kQ4RowBytes + at.g * 8) = make_uint2(w[0], w[1]);
    scales[row * kQ4ScaleBytes + at.g] = (uint8_t)byte;
  }
}

template <int kRows>
__global__ void __launch_bounds__(kBlockThreads) dequantize_q4_kernel(
    const __grid_constant__ Kv4Args a) {
  const Place<kRows> at;
  const long long row0 = at.row(a);
  if (row0 < 0) return;
  uint2 w[kRows];
  uint32_t sc[kRows];
#pragma unroll
  for (int k = 0; k < kRows; ++k) {
    const int r = at.r0 + k;
    const long long row = row0 + r % kKvHeads * a.page_size;
    w[k] = *reinterpret_cast<const uint2*>((r < kKvHeads ? a.k_codes : a.v_codes) + row * kQ4RowBytes + at.g * 8);
    sc[k] = (r < kKvHeads ? a.k_scales : a.v_scales)[row * kQ4ScaleBytes + at.g];
  }
#pragma unroll
  for (int k = 0; k < kRows; ++k) {
    const int r = at.r0 + k;
    const Q4Scale q = q4_scale(sc[k]);
    uint32_t o0[4], o1[4];
    q4_widen(w[k].x, q, o0);
    q4_widen(w[k].y, q, o1);
    uint16_t* to = (r < kKvHeads ? a.k_out : a.v_out) + (at.tok * kKvHeads + r % kKvHeads) * kDim + at.g * kQ4Group;
    if (a.out32) {   // whole sectors by one store a lane (two 16-byte stores: half sectors twice)
      const uint32_t o[8] = {o0[0], o0[1], o0[2], o0[3], o1[0], o1[1], o1[2], o1[3]};
      st_global_v8(to, o);
    } else {
      reinterpret_cast<uint4*>(to)[0] = make_uint4(o0[0], o0[1], o0[2], o0[3]);
      reinterpret_cast<uint4*>(to)[1] = make_uint4(o1[0], o1[1], o1[2], o1[3]);
    }
  }
}

unsigned kv4_grid(long long n_tok, int rows) {
  const long long per = (long long)(kBlockThreads / kRowThreads) * rows / kTokRows;
  return (unsigned)((n_tok + per - 1) / per);
}
// Four rows a thread from here on, against one: storing 4,096 tokens 3.2 against 3.4 us, 65,536
// tokens 26.6 against 34.3 (widening 28.3 against 33.5); 64 tokens 2.15 against 1.67, 3,000 tokens
// 3.2 against 2.8 (a quarter of the threads, each with four times the chain of instructions).
constexpr long long kManyToks = 4096;

}  // namespace

cudaError_t launch_quantize_q4(const Kv4Args& a, cudaStream_t s) {
  if (a.n_tok >= kManyToks)
    quantize_q4_kernel<4><<<kv4_grid(a.n_tok, 4), kBlockThreads, 0, s>>>(a);
  else
    quantize_q4_kernel<1><<<kv4_grid(a.n_tok, 1), kBlockThreads, 0, s>>>(a);
  return cudaGetLastError();
}
cudaError_t launch_dequantize_q4(const Kv4Args& a, cudaStream_t s) {
  if (a.n_tok >= kManyToks)
    dequantize_q4_kernel<4><<<kv4_grid(a.n_tok, 4), kBlockThreads, 0, s>>>(a);
  else
    dequantize_q4_kernel<1><<<kv4_grid(a.n_tok, 1), kBlockThreads, 0, s>>>(a);
  return cudaGetLastError();
}

}  // namespace ga

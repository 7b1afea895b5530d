// 4-bit cache rows in paged pools: storing rows of keys and values by slot, and widening them
// back to bf16 (the format is in ga_q4.cuh). Pools are head-major inside a page,
// [n_pages][2][page_size][128] code bytes and [n_pages][2][page_size][16] scale bytes, so the
// attention reads a key tile of one KV head as one contiguous run. Slot x of a pool is
// position x % page_size of page x / page_size, the same for both heads.
//
// 16 lanes per row, one 16-value group per lane, so a group's maximum needs no exchange between
// lanes, a row's reads and writes are contiguous runs, and the four rows of a token (two heads of
// K and of V) lie in one 64-thread stretch. Both kernels are bound by the bytes they move
// (2,624 a token); a thread takes kTok tokens, with the slots and then the rows of all of them
// in flight before the first is used, once there are enough tokens to fill the device so.
#include <cuda_bf16.h>

#include "ga_internal.h"
#include "ga_q4.cuh"
#include "ga_sm100.cuh"

namespace ga {
namespace {

constexpr int kRowThreads = 16;                           // one 16-value group each
constexpr int kTokThreads = 2 * kKvHeads * kRowThreads;   // K and V rows of a token
constexpr int kBlockThreads = 256;
constexpr int kBlockToks = kBlockThreads / kTokThreads;   // tokens a block takes at a time

// Row index in a pool of a slot's row of head h, or -1: a negative slot (the token is not
// stored) or one outside the pool (recorded in the status word).
__device__ __forceinline__ long long pool_row(const Kv4Args& a, long long slot, int h) {
  if (slot < 0) return -1;
  if (slot >= a.n_slots) {
    atomicCAS(a.status, 0, (int)kDevBadPage);
    return -1;
  }
  const unsigned page = (unsigned)slot / (unsigned)a.page_size;
  const unsigned off = (unsigned)slot - page * (unsigned)a.page_size;
  return ((long long)page * kKvHeads + h) * a.page_size + off;
}

// A thread's place in a token: a group of a head's K or V row.
struct Place {
  int g, h;
  bool is_v;
  long long tok;   // its first token; the next ones kBlockToks apart
  __device__ __forceinline__ explicit Place(int n_per_thread) {
    const int row = (threadIdx.x % kTokThreads) / kRowThreads;   // K head 0, 1, V head 0, 1
    g = threadIdx.x % kRowThreads;
    h = row % kKvHeads;
    is_v = row >= kKvHeads;
    tok = (long long)blockIdx.x * (kBlockToks * n_per_thread) + threadIdx.x / kTokThreads;
  }
};
template <int kTok>
__device__ __forceinline__ void pool_rows(const Kv4Args& a, const Place& at, long long (&row)[kTok]) {
  long long slot[kTok];
#pragma unroll
  for (int k = 0; k < kTok; ++k) {
    const long long t = at.tok + k * kBlockToks;
    slot[k] = t >= a.n_tok ? -1 : a.slots ? (long long)__ldg(a.slots + t) : t;
  }
#pragma unroll
  for (int k = 0; k < kTok; ++k) row[k] = pool_row(a, slot[k], at.h);
}

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
// more; smaller ones round to 0), while x times the reciprocal is within 2^-19 of it. Adding and
// subtracting 3072 = 1.5 x 2^11 rounds that product to a multiple of 2^-12: a quotient on a half
// comes out on it exactly, and none is carried to or past one. A last addition rounds to the
// integer, ties to even, in the low bits of the sum.
constexpr float kSnap = 1.5f * 2048.0f, kInt = 1.5f * 8388608.0f + 8.0f;
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
__device__ __forceinline__ uint64_t mul_f32x2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
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
                   back = pack_f32x2(-kSnap, -kSnap), whole = pack_f32x2(kInt, kInt);
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      uint32_t acc = 0u;
#pragma unroll
      for (int j = 0; j < 4; ++j) {   // dims 2j and 2j + 1: nibbles j and 4 + j
        const uint32_t v = xw[4 * k + j];
        uint64_t q = mul_f32x2(pack_f32x2(__uint_as_float(v << 16), __uint_as_float(v & 0xFFFF0000u)), inv2);
        q = add_f32x2(add_f32x2(add_f32x2(q, snap), back), whole);
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

// 32 bytes of a row by one lane: two 16-byte loads (the rows are 16-byte aligned).
__device__ __forceinline__ void load_group(const uint16_t* p, uint32_t (&x)[8]) {
  const uint4 x0 = __ldg(reinterpret_cast<const uint4*>(p));
  const uint4 x1 = __ldg(reinterpret_cast<const uint4*>(p) + 1);
  x[0] = x0.x; x[1] = x0.y; x[2] = x0.z; x[3] = x0.w;
  x[4] = x1.x; x[5] = x1.y; x[6] = x1.z; x[7] = x1.w;
}

template <int kTok>
__global__ void __launch_bounds__(kBlockThreads) quantize_q4_kernel(
    const __grid_constant__ Kv4Args a) {
  const Place at(kTok);
  const uint16_t* x = (at.is_v ? a.v : a.k) + at.h * kDim + at.g * kQ4Group;
  const long long ld = at.is_v ? a.ld_v : a.ld_k;
  uint32_t xw[kTok][8];
#pragma unroll
  for (int k = 0; k < kTok; ++k) {   // the rows do not wait for the slots
    const long long t = at.tok + k * kBlockToks;
    if (t < a.n_tok) load_group(x + t * ld, xw[k]);
  }
  long long row[kTok];
  pool_rows<kTok>(a, at, row);
  uint8_t* codes = at.is_v ? a.v_codes : a.k_codes;
  uint8_t* scales = at.is_v ? a.v_scales : a.k_scales;
#pragma unroll
  for (int k = 0; k < kTok; ++k) {
    if (row[k] < 0) continue;
    uint32_t w[2];
    const uint32_t byte = quantize_group(xw[k], w);
    *reinterpret_cast<uint2*>(codes + row[k] * kQ4RowBytes + at.g * 8) = make_uint2(w[0], w[1]);
    scales[row[k] * kQ4ScaleBytes + at.g] = (uint8_t)byte;
  }
}

template <int kTok>
__global__ void __launch_bounds__(kBlockThreads) dequantize_q4_kernel(
    const __grid_constant__ Kv4Args a) {
  const Place at(kTok);
  long long row[kTok];
  pool_rows<kTok>(a, at, row);
  const uint8_t* codes = at.is_v ? a.v_codes : a.k_codes;
  const uint8_t* scales = at.is_v ? a.v_scales : a.k_scales;
  uint2 w[kTok];
  uint32_t sc[kTok];
#pragma unroll
  for (int k = 0; k < kTok; ++k) {
    const long long r = row[k] < 0 ? 0 : row[k];
    w[k] = *reinterpret_cast<const uint2*>(codes + r * kQ4RowBytes + at.g * 8);
    sc[k] = scales[r * kQ4ScaleBytes + at.g];
  }
  uint16_t* out = (at.is_v ? a.v_out : a.k_out) + at.h * kDim + at.g * kQ4Group;
#pragma unroll
  for (int k = 0; k < kTok; ++k) {
    if (row[k] < 0) continue;
    const Q4Scale q = q4_scale(sc[k]);
    uint32_t o0[4], o1[4];
    q4_widen(w[k].x, q, o0);
    q4_widen(w[k].y, q, o1);
    uint16_t* to = out + (at.tok + k * kBlockToks) * (kKvHeads * kDim);
    if (a.out32) {   // whole sectors by one store a lane (two 16-byte stores: half sectors twice)
      const uint32_t o[8] = {o0[0], o0[1], o0[2], o0[3], o1[0], o1[1], o1[2], o1[3]};
      st_global_v8(to, o);
    } else {
      reinterpret_cast<uint4*>(to)[0] = make_uint4(o0[0], o0[1], o0[2], o0[3]);
      reinterpret_cast<uint4*>(to)[1] = make_uint4(o1[0], o1[1], o1[2], o1[3]);
    }
  }
}

unsigned kv4_grid(long long n_tok, int per_thread) {
  const long long per = (long long)kBlockToks * per_thread;
  return (unsigned)((n_tok + per - 1) / per);
}
// Four tokens a thread from here on (the blocks then still fill the device a few times over).
constexpr long long kManyToks = 16384;

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

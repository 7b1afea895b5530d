// 4-bit cache rows in paged pools: storing rows of keys and values by slot, and widening them
// back to bf16 (the format is in ga_q4.cuh). Pools are head-major inside a page,
// [n_pages][2][page_size][128] code bytes and [n_pages][2][page_size][16] scale bytes, so the
// attention reads a key tile of one KV head as one contiguous run. Slot x of a pool is
// position x % page_size of page x / page_size, the same for both heads.
//
// Both kernels only move bytes: 16 lanes per row, one 16-value group per lane, so a group's
// maximum needs no exchange between lanes, a row's reads and writes are contiguous runs, and
// the four rows of a token (two heads of K and of V) lie in one 64-thread stretch.
#include <cuda_bf16.h>

#include "ga_internal.h"
#include "ga_q4.cuh"
#include "ga_sm100.cuh"

namespace ga {
namespace {

constexpr int kRowThreads = 16;                           // one 16-value group each
constexpr int kTokThreads = 2 * kKvHeads * kRowThreads;   // K and V rows of a token
constexpr int kBlockThreads = 256;

// Row index in a pool of token t's row of head h, or -1: a negative slot (the token is not
// stored) or one outside the pool (recorded in the status word).
__device__ __forceinline__ long long pool_row(const Kv4Args& a, long long t, int h) {
  const long long slot = a.slots ? (long long)__ldg(a.slots + t) : t;
  if (slot < 0) return -1;
  if (slot >= a.n_slots) {
    atomicCAS(a.status, 0, (int)kDevBadPage);
    return -1;
  }
  const unsigned page = (unsigned)slot / (unsigned)a.page_size;
  const unsigned off = (unsigned)slot - page * (unsigned)a.page_size;
  return ((long long)page * kKvHeads + h) * a.page_size + off;
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

// clamp(rne(x / s), -8, 7) + 8; NaN counts as 0. A bf16 x over a 4-bit s reaches a half
// only exactly, so rounding the rounded quotient is rounding the quotient.
__device__ __forceinline__ uint32_t code_of(float x, float s) {
  float q = rintf(__fdiv_rn(x, s));
  q = fminf(fmaxf(q, -8.0f), 7.0f);
  return x != x ? 8u : (uint32_t)((int)q + 8);
}

__global__ void __launch_bounds__(kBlockThreads) quantize_q4_kernel(
    const __grid_constant__ Kv4Args a) {
  const long long i = (long long)blockIdx.x * kBlockThreads + threadIdx.x;
  const long long t = i / kTokThreads;
  if (t >= a.n_tok) return;
  const int row = (int)(i % kTokThreads) / kRowThreads;   // K head 0, 1, V head 0, 1
  const int g = (int)(i % kRowThreads);
  const int h = row % kKvHeads;
  const bool is_v = row >= kKvHeads;
  const long long dst = pool_row(a, t, h);
  if (dst < 0) return;
  const uint16_t* src = (is_v ? a.v + t * a.ld_v : a.k + t * a.ld_k) + h * kDim + g * kQ4Group;
  const uint4 x0 = __ldg(reinterpret_cast<const uint4*>(src));
  const uint4 x1 = __ldg(reinterpret_cast<const uint4*>(src) + 1);
  const uint32_t xw[8] = {x0.x, x0.y, x0.z, x0.w, x1.x, x1.y, x1.z, x1.w};
  float v[kQ4Group], amax = 0.f;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    v[2 * j] = __uint_as_float(xw[j] << 16);
    v[2 * j + 1] = __uint_as_float(xw[j] & 0xFFFF0000u);
    amax = fmaxf(amax, fmaxf(fabsf(v[2 * j]), fabsf(v[2 * j + 1])));   // NaN is passed over
  }
  const uint32_t byte = scale_byte(amax);
  const float s = __uint_as_float((byte + ((127u - kQ4ExpBias) << 3)) << 20);
  uint32_t w[2] = {0u, 0u};
#pragma unroll
  for (int j = 0; j < kQ4Group; ++j) {
    const int d = j & 7;
    w[j >> 3] |= code_of(v[j], s) << (4 * ((d >> 1) + 4 * (d & 1)));
  }
  uint8_t* codes = is_v ? a.v_codes : a.k_codes;
  uint8_t* scales = is_v ? a.v_scales : a.k_scales;
  *reinterpret_cast<uint2*>(codes + dst * kQ4RowBytes + g * 8) = make_uint2(w[0], w[1]);
  scales[dst * kQ4ScaleBytes + g] = (uint8_t)byte;
}

__global__ void __launch_bounds__(kBlockThreads) dequantize_q4_kernel(
    const __grid_constant__ Kv4Args a) {
  const long long i = (long long)blockIdx.x * kBlockThreads + threadIdx.x;
  const long long t = i / kTokThreads;
  if (t >= a.n_tok) return;
  const int row = (int)(i % kTokThreads) / kRowThreads;
  const int g = (int)(i % kRowThreads);
  const int h = row % kKvHeads;
  const bool is_v = row >= kKvHeads;
  const long long src = pool_row(a, t, h);
  if (src < 0) return;
  const uint8_t* codes = is_v ? a.v_codes : a.k_codes;
  const uint8_t* scales = is_v ? a.v_scales : a.k_scales;
  const uint2 w = *reinterpret_cast<const uint2*>(codes + src * kQ4RowBytes + g * 8);
  const Q4Scale q = q4_scale(scales[src * kQ4ScaleBytes + g]);
  uint32_t o0[4], o1[4];
  q4_widen(w.x, q, o0);
  q4_widen(w.y, q, o1);
  uint16_t* out = (is_v ? a.v_out : a.k_out) + (t * kKvHeads + h) * kDim + g * kQ4Group;
  reinterpret_cast<uint4*>(out)[0] = make_uint4(o0[0], o0[1], o0[2], o0[3]);
  reinterpret_cast<uint4*>(out)[1] = make_uint4(o1[0], o1[1], o1[2], o1[3]);
}

unsigned kv4_grid(long long n_tok) {
  return (unsigned)((n_tok * kTokThreads + kBlockThreads - 1) / kBlockThreads);
}

}  // namespace

cudaError_t launch_quantize_q4(const Kv4Args& a, cudaStream_t s) {
  quantize_q4_kernel<<<kv4_grid(a.n_tok), kBlockThreads, 0, s>>>(a);
  return cudaGetLastError();
}
cudaError_t launch_dequantize_q4(const Kv4Args& a, cudaStream_t s) {
  dequantize_q4_kernel<<<kv4_grid(a.n_tok), kBlockThreads, 0, s>>>(a);
  return cudaGetLastError();
}

}  // namespace ga

// 8-bit cache rows in paged pools: storing rows of keys and values by slot, and widening them back
// to bf16 (the format is in ga_q8.cuh). Pools are head-major inside a page, [n_pages][2][page_size]
// [256] code bytes and [n_pages][2][page_size / 32] scale bytes, so a block's codes are 8 KiB in a
// row and a key tile of one KV head is one contiguous run.
#include "ga_internal.h"
#include "ga_q8.cuh"
#include "ga_sm100.cuh"

namespace ga {
namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kChunk = 32;                       // tokens whose runs a CTA stores
constexpr int kSpan = 2 * kChunk;                // a run goes at most 31 tokens past them
constexpr int kRowsPerWarp = kSpan / kWarps;

struct Slot {
  long long row;    // pool row of head 0; head 1's is page_size on
  long long scale;  // scale byte of head 0; head 1's is page_size / 32 on
};
// A slot's place: page_size is a multiple of 32, so that blocks do not straddle pages.
__device__ __forceinline__ Slot slot_place(const Kv8Args& a, int slot) {
  const int page = slot / a.page_size, off = slot - page * a.page_size;
  return Slot{(long long)page * kKvHeads * a.page_size + off,
              (long long)page * kKvHeads * (a.page_size / kQ8Block) + off / kQ8Block};
}
// The slot of token t, or -1 where there is nothing to store or read (a negative slot, one outside
// the pool, which is recorded, or no token).
__device__ __forceinline__ int slot_of(const Kv8Args& a, long long t) {
  if (t < 0 || t >= a.n_tok) return -1;
  const int s = a.slots ? __ldg(a.slots + t) : (int)t;
  if (s >= a.n_slots) {
    atomicCAS(a.status, 0, (int)kDevBadPage);
    return -1;
  }
  return s < 0 ? -1 : s;
}

// The exponent for a largest magnitude of bf16 bits `top` (no NaN): 448 = 1.75 x 2^8.
__device__ __forceinline__ int exp_for(uint32_t top) {
  const int e = (int)(top >> 7) - 127 - 8 + ((top & 127u) > 96u ? 1 : 0);
  return min(max(e, kQ8MinExp), kQ8MaxExp);
}
__device__ __forceinline__ float scaled(uint32_t bf16_bits, float inv) {
  const float x = __uint_as_float(bf16_bits);
  return x != x ? 0.f : x * inv;   // x inv is exact, or past +-448 either way
}
__device__ __forceinline__ uint2 encode(const uint4& x, float inv) {
  const uint32_t w[4] = {x.x, x.y, x.z, x.w};
  uint32_t c[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) c[i] = e4m3x2(scaled(w[i] << 16, inv), scaled(w[i] & 0xFFFF0000u, inv));
  return make_uint2(c[0] | c[1] << 16, c[2] | c[3] << 16);
}

// A run is a row of tokens of one block. CTA (c, u) stores, for K or V (u / 2) and head u % 2, the
// runs that begin among tokens 32 c .. 32 c + 31: a prompt's chunk has one or two, a decode batch
// 32 of one token. Its tokens are dealt to the warps row by row, 8 values a lane, and stay in
// registers from the search for the maxima to their codes, so every row is read once.
__global__ void __launch_bounds__(kThreads) quantize_kernel(const __grid_constant__ Kv8Args a) {
  __shared__ uint32_t top[kChunk], written[kChunk];
  __shared__ int exps[kChunk], shift[kChunk], first[kChunk];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int kv = blockIdx.y >> 1, head = blockIdx.y & 1;
  const long long t0 = (long long)blockIdx.x * kChunk;
  const uint16_t* in = (kv ? a.v : a.k) + head * kDim;
  const long long ld = kv ? a.ld_v : a.ld_k;
  uint8_t* codes = kv ? a.v_codes : a.k_codes;
  uint8_t* scales = kv ? a.v_scales : a.k_scales;
  if (tid < kChunk) top[tid] = written[tid] = 0u;
  // every warp finds the runs: this lane's tokens are t0 + lane and t0 + 32 + lane
  const int s0 = slot_of(a, t0 + lane), s1 = slot_of(a, t0 + kChunk + lane);
  int before = __shfl_up_sync(0xffffffffu, s0, 1);
  if (lane == 0) before = slot_of(a, t0 - 1);
  const bool lead = s0 >= 0 && (before < 0 || (before >> 5) != (s0 >> 5));
  const uint32_t leads = __ballot_sync(0xffffffffu, lead);
  if (leads == 0u) return;   // (the same in every warp)
  const int last = __shfl_sync(0xffffffffu, s0, 31);
  // the last run's tokens past the chunk, 32 in all at most
  const uint32_t goes_on = __ballot_sync(0xffffffffu, last >= 0 && s1 >= 0 && (s1 >> 5) == (last >> 5));
  const int runs = __popc(leads), last_lead = 31 - __clz(leads);
  const int more = min(__ffs(~goes_on) ? __ffs(~goes_on) - 1 : 32, last_lead);
  if (warp == 0 && lead) first[__popc(leads & ((1u << lane) - 1u))] = s0;
  __syncthreads();
  uint4 x[kRowsPerWarp];
  int slot[kRowsPerWarp];
#pragma unroll
  for (int i = 0; i < kRowsPerWarp; ++i) {
    const int at = warp + kWarps * i;
    const int s = __shfl_sync(0xffffffffu, at < kChunk ? s0 : s1, at & 31);
    const bool mine = at < kChunk ? (leads & ((2u << at) - 1u)) != 0u : at - kChunk < more;
    slot[i] = mine ? s : -1;
    if (slot[i] >= 0) x[i] = __ldg(reinterpret_cast<const uint4*>(in + (t0 + at) * ld) + lane);
  }
  auto run_of = [&](int i) {
    const int at = warp + kWarps * i;
    return at < kChunk ? __popc(leads & ((2u << at) - 1u)) - 1 : runs - 1;
  };
#pragma unroll
  for (int i = 0; i < kRowsPerWarp; ++i) {
    if (slot[i] < 0) continue;
    const uint32_t m = __reduce_max_sync(0xffffffffu, top_of(x[i]));
    if (lane == 0) {
      atomicMax(&top[run_of(i)], m);
      atomicOr(&written[run_of(i)], 1u << (slot[i] & 31));
    }
  }
  __syncthreads();
  if (tid < runs) {
    uint8_t* at = scales + slot_place(a, first[tid]).scale + head * (a.page_size / kQ8Block);
    int e = exp_for(top[tid]);
    int grown = 0;
    if ((written[tid] & 1u) == 0u) {   // the block goes on
      const int was = q8_exp(*at);
      grown = max(e - was, 0);
      e = max(e, was);
    }
    *at = (uint8_t)(e - kQ8MinExp);
    exps[tid] = e;
    shift[tid] = grown;
  }
  const bool any = __syncthreads_or(tid < runs && shift[tid] > 0);
#pragma unroll
  for (int i = 0; i < kRowsPerWarp; ++i) {
    if (slot[i] < 0) continue;
    const long long row = slot_place(a, slot[i]).row + head * a.page_size;
    reinterpret_cast<uint2*>(codes + row * kQ8RowBytes)[lane] = encode(x[i], pow2i(-exps[run_of(i)]));
  }
  if (!any) return;
  // the other rows of blocks that grew
  for (int i = warp; i < runs * kQ8Block; i += kWarps) {
    const int r = i / kQ8Block, off = i % kQ8Block;
    if (shift[r] == 0 || (written[r] >> off & 1u)) continue;
    const long long row = slot_place(a, (first[r] & ~31) + off).row + head * a.page_size;
    uint2* p = reinterpret_cast<uint2*>(codes + row * kQ8RowBytes) + lane;
    const uint2 c = *p;
    const float inv = pow2i(-shift[r]);
    uint32_t w[2] = {c.x, c.y}, o[2];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const float2 lo = f16x2_f32(e4m3x2_f16x2(w[j] & 0xFFFFu)), hi = f16x2_f32(e4m3x2_f16x2(w[j] >> 16));
      o[j] = e4m3x2(lo.x * inv, lo.y * inv) | e4m3x2(hi.x * inv, hi.y * inv) << 16;
    }
    *p = make_uint2(o[0], o[1]);
  }
}

// Widening: a warp takes the four rows (two heads of K and of V) of two tokens, 8 codes a lane, all
// of them in flight before the first is used.
constexpr int kWidenTokens = 2;
__global__ void __launch_bounds__(kThreads) dequantize_kernel(const __grid_constant__ Kv8Args a) {
  const int lane = threadIdx.x & 31;
  const long long t0 = ((long long)blockIdx.x * kWarps + (threadIdx.x >> 5)) * kWidenTokens;
  uint2 c[kWidenTokens][4];
  uint32_t sc[kWidenTokens][4];
  bool live[kWidenTokens];
#pragma unroll
  for (int i = 0; i < kWidenTokens; ++i) {
    const int s = slot_of(a, t0 + i);
    live[i] = s >= 0;
    if (!live[i]) continue;
    const Slot p = slot_place(a, s);
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const long long row = p.row + (u & 1) * a.page_size;
      c[i][u] = __ldg(reinterpret_cast<const uint2*>((u < 2 ? a.k_codes : a.v_codes) + row * kQ8RowBytes) + lane);
      sc[i][u] = __ldg((u < 2 ? a.k_scales : a.v_scales) + p.scale + (u & 1) * (a.page_size / kQ8Block));
    }
  }
#pragma unroll
  for (int i = 0; i < kWidenTokens; ++i) {
    if (!live[i]) continue;
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const float s = pow2i(q8_exp(sc[i][u]));
      const uint32_t w[2] = {c[i][u].x, c[i][u].y};
      uint32_t o[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float2 v = f16x2_f32(e4m3x2_f16x2(w[j >> 1] >> (16 * (j & 1)) & 0xFFFFu));
        o[j] = pack_bf16x2(v.x * s, v.y * s);
      }
      uint16_t* out = (u < 2 ? a.k_out : a.v_out) + ((t0 + i) * kKvHeads + (u & 1)) * kDim;
      reinterpret_cast<uint4*>(out)[lane] = make_uint4(o[0], o[1], o[2], o[3]);
    }
  }
}

}  // namespace

cudaError_t launch_quantize_q8(const Kv8Args& a, cudaStream_t s) {
  quantize_kernel<<<dim3((unsigned)((a.n_tok + kChunk - 1) / kChunk), 2 * kKvHeads), kThreads, 0, s>>>(a);
  return cudaGetLastError();
}

cudaError_t launch_dequantize_q8(const Kv8Args& a, cudaStream_t s) {
  constexpr int kPer = kWarps * kWidenTokens;
  dequantize_kernel<<<(unsigned)((a.n_tok + kPer - 1) / kPer), kThreads, 0, s>>>(a);
  return cudaGetLastError();
}

}  // namespace ga

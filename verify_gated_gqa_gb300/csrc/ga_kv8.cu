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
constexpr int kRowWarps = kWarps / kKvHeads;               // warps of each head
constexpr int kKept = kChunk / kRowWarps;                  // rows that a warp keeps in registers

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
  const int s = a.slots ? ld_input(a.slots + t) : (int)t;
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
// NaNs of x made 0, which is what is stored for them. The largest magnitude's bits.
__device__ __forceinline__ uint32_t clear_nan(uint4& x) {
  auto top = [&]() {
    const uint32_t m = __vmaxu2(__vmaxu2(x.x & 0x7FFF7FFFu, x.y & 0x7FFF7FFFu),
                                __vmaxu2(x.z & 0x7FFF7FFFu, x.w & 0x7FFF7FFFu));
    return max(m & 0xFFFFu, m >> 16);
  };
  auto clear = [](uint32_t w) {
    return ((w & 0x7FFFu) > 0x7F80u ? 0u : w & 0xFFFFu) | ((w >> 16 & 0x7FFFu) > 0x7F80u ? 0u : w & 0xFFFF0000u);
  };
  uint32_t t = top();
  if (t > 0x7F80u) {
    x = make_uint4(clear(x.x), clear(x.y), clear(x.z), clear(x.w));
    t = top();
  }
  return t;
}
// x inv is exact, or past +-448 either way.
__device__ __forceinline__ uint2 encode(const uint4& x, float inv) {
  const uint32_t w[4] = {x.x, x.y, x.z, x.w};
  uint32_t c[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float lo, hi;   // both by one instruction
    asm("{\n\t.reg .b64 x, s;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 s, {%4, %4};\n\tmul.rn.f32x2 x, x, s;\n\t"
        "mov.b64 {%0, %1}, x;\n\t}"
        : "=f"(lo), "=f"(hi)
        : "r"(w[i] << 16), "r"(w[i] & 0xFFFF0000u), "f"(inv));
    c[i] = e4m3x2(lo, hi);
  }
  return make_uint2(c[0] | c[1] << 16, c[2] | c[3] << 16);
}

// A run is a row of tokens of one block. CTA (c, kv) stores the keys' or values' runs that begin among
// tokens 32 c .. 32 c + 31: a prompt's chunk has one or two, a decode batch 32 of one token. Four warps
// take each head, 8 values a lane. The rows are on their way before the slots are known. A chunk's stay
// in registers from the search for the maxima to their codes; those of a run that goes on past the
// chunk (31 at most) are read again. Bound by the bytes it moves (131,072 tokens 74 us, 5.4 TB/s) and by
// how much of the waiting for them its warps cover: 29 of 64 an SM, 61 % of the issue slots used (40,001
// tokens). With a test for NaN and a division by the page size at every use 131,072 tokens took 93 us. Four
// CTAs an SM keep everything in registers; five spill and take as long.
__global__ void __launch_bounds__(kThreads, 4) quantize_kernel(const __grid_constant__ Kv8Args a) {
  __shared__ uint32_t top[kKvHeads][kChunk], written[kChunk];
  __shared__ int exps[kKvHeads][kChunk], shift[kKvHeads][kChunk], first[kChunk];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int head = warp / kRowWarps, part = warp % kRowWarps, kv = blockIdx.y;
  const long long t0 = (long long)blockIdx.x * kChunk;
  const uint16_t* in = (kv ? a.v : a.k) + head * kDim;
  const long long ld = kv ? a.ld_v : a.ld_k;
  uint8_t* codes = kv ? a.v_codes : a.k_codes;
  uint8_t* scales = kv ? a.v_scales : a.k_scales;
  if (tid < kKvHeads * kChunk) top[tid / kChunk][tid % kChunk] = 0u;
  grid_wait();
  grid_launch_dependents();
  auto load = [&](int at) { return ld_input(reinterpret_cast<const uint4*>(in + (t0 + at) * ld) + lane); };
  uint4 x[kKept];
#pragma unroll
  for (int i = 0; i < kKept; ++i) {
    const int at = part + kRowWarps * i;
    x[i] = make_uint4(0u, 0u, 0u, 0u);
    if (t0 + at < a.n_tok) x[i] = load(at);
  }
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
  // codes' places of this lane's tokens (a division each: found once, and handed on)
  const int row0 = s0 >= 0 ? (int)slot_place(a, s0).row : -1;   // below 2^31, as the pool's rows
  const int runs = __popc(leads), last_lead = 31 - __clz(leads);
  const int more = min(__ffs(~goes_on) ? __ffs(~goes_on) - 1 : 32, last_lead);
  const int run0 = __popc(leads & ((2u << lane) - 1u)) - 1;   // of token t0 + lane, or -1
  if (warp == 0) {   // which slots of its block a run writes
    if (lead) first[run0] = s0;
    written[lane] = 0u;
    __syncwarp();
    if (s0 >= 0 && run0 >= 0) atomicOr(&written[run0], 1u << (s0 & 31));
    if (lane < more) atomicOr(&written[runs - 1], 1u << (s1 & 31));
  }
  __syncthreads();   // top is zero
#pragma unroll
  for (int i = 0; i < kKept; ++i) {
    const int at = part + kRowWarps * i;
    const int slot = __shfl_sync(0xffffffffu, s0, at), run = __shfl_sync(0xffffffffu, run0, at);
    const uint32_t m = __reduce_max_sync(0xffffffffu, clear_nan(x[i]));
    if (lane == 0 && slot >= 0 && run >= 0) atomicMax(&top[head][run], m);
  }
  for (int at = part; at < more; at += kRowWarps) {
    const uint32_t m = __reduce_max_sync(0xffffffffu, top_of(load(kChunk + at)));
    if (lane == 0) atomicMax(&top[head][runs - 1], m);
  }
  __syncthreads();
  bool grows = false;
  if (tid < kKvHeads * kChunk && tid % kChunk < runs) {
    const int r = tid / kChunk, run = tid % kChunk;   // (a head of its own: not this warp's)
    uint8_t* at = scales + slot_place(a, first[run]).scale + r * (a.page_size / kQ8Block);
    int e = exp_for(top[r][run]), grown = 0;
    if ((written[run] & 1u) == 0u) {   // the block goes on
      const int was = q8_exp(*at);
      grown = max(e - was, 0);
      e = max(e, was);
    }
    *at = (uint8_t)(e - kQ8MinExp);
    exps[r][run] = e;
    shift[r][run] = grown;
    grows = grown > 0;
  }
  const bool any = __syncthreads_or(grows);
  auto store = [&](long long row, int run, const uint4& v) {
    const long long at = row + head * a.page_size;
    reinterpret_cast<uint2*>(codes + at * kQ8RowBytes)[lane] = encode(v, pow2i(-exps[head][run]));
  };
#pragma unroll
  for (int i = 0; i < kKept; ++i) {
    const int at = part + kRowWarps * i;
    const int row = __shfl_sync(0xffffffffu, row0, at), run = __shfl_sync(0xffffffffu, run0, at);
    if (row >= 0 && run >= 0) store(row, run, x[i]);
  }
  for (int at = part; at < more; at += kRowWarps) {
    uint4 v = load(kChunk + at);
    clear_nan(v);
    store(slot_place(a, __shfl_sync(0xffffffffu, s1, at)).row, runs - 1, v);
  }
  if (!any) return;
  // the other rows of blocks that grew
  for (int i = part; i < runs * kQ8Block; i += kRowWarps) {
    const int run = i / kQ8Block, off = i % kQ8Block;
    if (shift[head][run] == 0 || (written[run] >> off & 1u)) continue;
    const long long at = slot_place(a, (first[run] & ~31) + off).row + head * a.page_size;
    uint2* p = reinterpret_cast<uint2*>(codes + at * kQ8RowBytes) + lane;
    const uint2 c = *p;
    const float inv = pow2i(-shift[head][run]);
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
  grid_wait();
  grid_launch_dependents();
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
      c[i][u] = ld_input(reinterpret_cast<const uint2*>((u < 2 ? a.k_codes : a.v_codes) + row * kQ8RowBytes) + lane);
      sc[i][u] = ld_input((u < 2 ? a.k_scales : a.v_scales) + p.scale + (u & 1) * (a.page_size / kQ8Block));
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
  cudaLaunchAttribute attr[1];
  cudaLaunchConfig_t cfg = overlapped_launch((unsigned)((a.n_tok + kChunk - 1) / kChunk), kThreads, 0, s, attr);
  cfg.gridDim.y = 2;   // keys, values
  return cudaLaunchKernelEx(&cfg, quantize_kernel, a);
}

cudaError_t launch_dequantize_q8(const Kv8Args& a, cudaStream_t s) {
  constexpr int kPer = kWarps * kWidenTokens;
  cudaLaunchAttribute attr[1];
  const cudaLaunchConfig_t cfg = overlapped_launch((unsigned)((a.n_tok + kPer - 1) / kPer), kThreads, 0, s, attr);
  return cudaLaunchKernelEx(&cfg, dequantize_kernel, a);
}

}  // namespace ga

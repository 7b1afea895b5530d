// Decode attention (one row per sequence) over 4-bit paged caches: ga_verify4.cu's results, for
// the twelve query rows that a (sequence, KV head) then has.
//
// Twelve rows would leave most of a 128-row tensor-core tile empty while every key and value
// still had to be widened through shared memory, so this form feeds mma.sync (16 rows) from
// registers: a lane's codes become its operand fragments where it holds them, and nothing
// widened is ever stored. What bounds it is the cache's bytes and the instructions that widen
// them, about equally (288 bytes and 550 warp instructions per 16 keys of a head).
//
// Work: streams (sequence, KV head) in granules of 32 keys, cut into equal runs, one per CTA, as in
// ga_v4.cuh. Eight warps a CTA; warp w takes a segment's granules w, w + 8, ... on its own: it
// loads them by TMA into two stages of its own (codes and scales of K and V, 9 KiB), forms S =
// Q K^T, a running softmax and O += P V for all 16 rows and 256 dims in registers, and meets the
// other warps only at the segment's end, where their O, M and l are joined in shared memory.
//
// Fragments (m16n8k16; lane = 4 g + t). The order of the dims within Q K^T is free as long as Q
// and K agree: lane t of a key owns its dims 64t .. 64t + 63 (two 16-byte chunks of codes; the
// widened pairs of a word are the fragments of two k-steps in their natural order). For P V, lane
// g owns dims 32g .. + 31 of each V row (one chunk), so column g of n-tile e is dim 32 g + e; the
// halves of the words of two keys are joined before they are widened, so a fragment's two keys
// come out of one operation, with the scales of both in one register. With these choices every
// 16-byte read of the swizzled codes is free of bank conflicts.
#include "ga_v4.cuh"

namespace ga {
namespace {

constexpr int kWarps = 8;
constexpr int kThreads = 32 * kWarps;
constexpr int kKeys = 32;                          // keys of a granule
constexpr int kStages = 2;
constexpr int kCodeBytes = kKeys * kQ4RowBytes, kScaleBytes = kKeys * kQ4ScaleBytes;
constexpr int kStageBytes = 2 * (kCodeBytes + kScaleBytes);
constexpr int kJoinStride = kDim + 8;              // floats between rows of the join buffer
constexpr float kLog2eOver16 = 1.4426950408889634f / 16.0f;
constexpr float kLazyRescale = 8.0f;

struct D4Smem {
  uint8_t codes[kWarps][kStages][2][kCodeBytes];   // K, V
  uint8_t scales[kWarps][kStages][2][kScaleBytes];
  uint4 q[16][32];                                 // Q fragments: k-step x lane
  float join[kWarps][8][kJoinStride];              // a segment's O by warp, eight rows at a time
  float m[kWarps][16], l[kWarps][16];
  V4Cut cut;
  uint64_t full[kWarps][kStages];
  int abort;
};
static_assert(sizeof(D4Smem) <= 232448, "227 KiB of shared memory per CTA");

__device__ __forceinline__ uint32_t lds_u32(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ void mma_16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                          uint32_t a3, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// A pair of codes at nibble p of both halves of w, widened.
__device__ __forceinline__ uint32_t widen_pair(uint32_t w, int p, Q4Scale q) {
  return q4_fma_bf16x2(q4_codes(w, p), q.s, q.off);
}
// Multipliers of two keys' groups: bytes b of ua and ub in the low and the high half.
__device__ __forceinline__ Q4Scale scale_pair(uint32_t ua, uint32_t ub, int b) {
  const uint32_t two = prmt_b32(ua, ub, b ? 0x2521u : 0x2420u);   // byte 2 of ua is zero
  Q4Scale q;
  q.s = two * 0x10u + (((127u - kQ4ExpBias) << 7) * 0x00010001u);
  q.off = q4_mul_bf16x2(q.s, 0xC308C308u);
  return q;
}

__global__ void __launch_bounds__(kThreads, 1)
    decode4_kernel(const __grid_constant__ CUtensorMap tm_kc, const __grid_constant__ CUtensorMap tm_vc,
                   const __grid_constant__ CUtensorMap tm_ks, const __grid_constant__ CUtensorMap tm_vs,
                   const __grid_constant__ Verify4Args a) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  if ((smem_u32(smem_raw) & 1023u) != 0u) {
    if (threadIdx.x == 0) record(a.status, kDevBadLaunch);
    return;
  }
  D4Smem& sm = *reinterpret_cast<D4Smem*>(smem_raw);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int g = lane >> 2, t = lane & 3;
  volatile int* abort = &sm.abort;
  if (tid == 0) {
    sm.abort = 0;
    for (int w = 0; w < kWarps; ++w)
      for (int i = 0; i < kStages; ++i) mbar_init(&sm.full[w][i], 1);
    mbar_fence_init();
  }
  if (warp == 1 && lane == 0) {
    tma_prefetch_desc(&tm_kc);
    tma_prefetch_desc(&tm_vc);
    tma_prefetch_desc(&tm_ks);
    tma_prefetch_desc(&tm_vs);
  }
  grid_wait();
  grid_launch_dependents();
  load_cut<kKeys, kThreads>(a, sm.cut, blockIdx.x == 0);
  __syncthreads();
  if (warp == 0) find_share(sm.cut, a.n_seq, kKvHeads);
  __syncthreads();

  // ---- loading: this warp's granules in order, lanes 0 .. 3 a copy each (K and V codes, K and V
  // scales). A granule on a page outside the pool (recorded) is read past the pool's end: zeros.
  const int n_rows = (int)((long long)a.n_pages * kKvHeads * a.page_size);
  const CUtensorMap* my_map = lane == 0 ? &tm_kc : lane == 1 ? &tm_vc : lane == 2 ? &tm_ks : &tm_vs;
  Walk ahead(sm.cut);
  Seg as{};
  int aj = 0;                // next granule of `as` of this warp
  uint32_t issued = 0;
  // the granule to issue next: its page-table entry (in flight until the issue reads it) and place
  // in the page; next_at < 0: none is left
  int next_page = 0, next_at = -1;
  auto find_next = [&]() {
    next_at = -1;
    while (aj >= as.n) {
      if (!ahead.next(sm.cut, a.n_seq, as)) return;
      aj = warp;
    }
    const int key0 = (as.kt0 + aj) * kKeys;
    aj += kWarps;
    const int e = key0 / a.page_size;
    next_page = __ldg(a.page_table + (size_t)as.b * a.max_pages + e);
    next_at = as.plane * a.page_size + key0 - e * a.page_size;
  };
  auto issue = [&]() {
    if (next_at < 0) return;
    int row = n_rows;
    if (next_page >= 0 && next_page < a.n_pages) row = next_page * kKvHeads * a.page_size + next_at;
    else if (lane == 0) record(a.status, kDevBadPage);
    const int st = (int)(issued % kStages);
    if (lane == 0) mbar_arrive_expect_tx(&sm.full[warp][st], kStageBytes);
    __syncwarp();
    if (lane < 4)
      tma_load_2d(lane < 2 ? sm.codes[warp][st][lane] : sm.scales[warp][st][lane - 2], my_map,
                  &sm.full[warp][st], 0, row);
    ++issued;
    find_next();
  };
  find_next();
  for (int i = 0; i < kStages; ++i) issue();

  uint32_t taken = 0;
  bool ok = true;   // a warp whose wait gave up goes on without computing, to meet the others
  Walk walk(sm.cut);
  Seg seg;
  while (walk.next(sm.cut, a.n_seq, seg)) {
    const int L = cut_len<kKeys>(sm.cut, seg.b, 1);
    // Q fragments of k-step i (of lane t's dims 64 t + 4 i .. + 3): rows g, g + 8 at the first two
    // of them, then at the last two; rows 12 .. 15 are zeros
#pragma unroll
    for (int i = 2 * warp; i < 2 * warp + 2; ++i) {
      const uint2* x = reinterpret_cast<const uint2*>(
          a.q_prep + ((size_t)seg.b * kHeads + seg.plane * kGroup + g) * kDim + 64 * t + 4 * i);
      const uint2 lo = __ldg(x);
      const uint2 hi = g < kGroup - 8 ? __ldg(x + 8 * kDim / 4) : make_uint2(0u, 0u);
      sm.q[i][lane] = make_uint4(lo.x, hi.x, lo.y, hi.y);
    }
    __syncthreads();
    const uint32_t q_at = smem_u32(&sm.q[0][lane]);
    float o[32][4];
#pragma unroll
    for (int e = 0; e < 32; ++e)
#pragma unroll
      for (int i = 0; i < 4; ++i) o[e][i] = 0.f;
    float M[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};   // rows g and g + 8

    for (int j0 = warp; j0 < seg.n; j0 += kWarps) {
      const int st = (int)(taken % kStages);
      if (ok) ok = warp_wait(&sm.full[warp][st], (taken / kStages) & 1, abort);
      ++taken;
      if (!ok) continue;
      const int key0 = (seg.kt0 + j0) * kKeys;
      const uint32_t kc = smem_u32(sm.codes[warp][st][0]), vc = smem_u32(sm.codes[warp][st][1]);
      const uint32_t ks = smem_u32(sm.scales[warp][st][0]), vs = smem_u32(sm.scales[warp][st][1]);
      // ---- S = Q K^T: n-tile n holds keys 8n .. 8n + 7, a key per g
      float s[4][4];
      uint32_t ksc[4];
#pragma unroll
      for (int n = 0; n < 4; ++n) {
#pragma unroll
        for (int i = 0; i < 4; ++i) s[n][i] = 0.f;
        ksc[n] = lds_u32(ks + (8 * n + g) * kQ4ScaleBytes + 4 * t);
      }
#pragma unroll
      for (int cc = 0; cc < 2; ++cc) {
        uint4 kw[4];
#pragma unroll
        for (int n = 0; n < 4; ++n)
          kw[n] = lds_v4(kc + (8 * n + g) * kQ4RowBytes + (((2 * t + cc) ^ g) << 4));
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const uint4 q0 = lds_v4(q_at + (8 * cc + 2 * j) * 512);       // two k-steps
          const uint4 q1 = lds_v4(q_at + (8 * cc + 2 * j + 1) * 512);
#pragma unroll
          for (int n = 0; n < 4; ++n) {
            const uint32_t w = j == 0 ? kw[n].x : j == 1 ? kw[n].y : j == 2 ? kw[n].z : kw[n].w;
            const Q4Scale sc = q4_scale((ksc[n] >> (16 * cc + 8 * (j >> 1))) & 0xFFu);
            uint32_t b[4];
            q4_widen(w, sc, b);
            mma_16816(s[n], q0.x, q0.y, q0.z, q0.w, b[0], b[1]);
            mma_16816(s[n], q1.x, q1.y, q1.z, q1.w, b[2], b[3]);
          }
        }
      }
      // ---- softmax: lane holds rows g, g + 8 at keys 8n + 2t, + 1
      if (key0 + kKeys - 1 > L) {
#pragma unroll
        for (int n = 0; n < 4; ++n)
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (key0 + 8 * n + 2 * t + (i & 1) > L) s[n][i] = -INFINITY;
      }
      bool grow = false;
      float top[2];
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        float m = fmaxf(s[0][2 * r], s[0][2 * r + 1]);
#pragma unroll
        for (int n = 1; n < 4; ++n) m = fmaxf(m, fmaxf(s[n][2 * r], s[n][2 * r + 1]));
        m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 1));
        m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 2));
        top[r] = m * kLog2eOver16;
        grow |= top[r] > M[r] + kLazyRescale;
      }
      if (__any_sync(0xffffffffu, grow)) {   // O and l to the new maxima (zeros the first time)
        float f[2];
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          const float nm = fmaxf(M[r], top[r]);
          f[r] = M[r] == -INFINITY ? 0.f : exp2f(M[r] - nm);
          M[r] = nm;
          l[r] *= f[r];
        }
#pragma unroll
        for (int e = 0; e < 32; ++e) {
          o[e][0] *= f[0];
          o[e][1] *= f[0];
          o[e][2] *= f[1];
          o[e][3] *= f[1];
        }
      }
      const float mf[2] = {M[0] == -INFINITY ? 0.f : M[0], M[1] == -INFINITY ? 0.f : M[1]};
      uint32_t p[4][2];   // P of n-tile n: rows g and g + 8
#pragma unroll
      for (int n = 0; n < 4; ++n)
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          const float p0 = ex2_approx(fmaf(s[n][2 * r], kLog2eOver16, -mf[r]));
          const float p1 = ex2_approx(fmaf(s[n][2 * r + 1], kLog2eOver16, -mf[r]));
          p[n][r] = pack_bf16x2(p0, p1);
          l[r] += lo_f(p[n][r]) + hi_f(p[n][r]);   // as rounded
        }
      // ---- O += P V: 16 keys at a time; fragment b0 is keys 2t, 2t + 1, b1 keys 2t + 8, 2t + 9
#pragma unroll
      for (int m = 0; m < 2; ++m) {
        uint4 vw[4];
        uint32_t vsc[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int row = 16 * m + 2 * t + (i & 1) + 8 * (i >> 1);
          vw[i] = lds_v4(vc + row * kQ4RowBytes + ((g ^ (row & 7)) << 4));
          vsc[i] = lds_u16(vs + row * kQ4ScaleBytes + 2 * g);
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const Q4Scale qa = scale_pair(vsc[0], vsc[1], j >> 1), qb = scale_pair(vsc[2], vsc[3], j >> 1);
          uint32_t w[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) w[i] = j == 0 ? vw[i].x : j == 1 ? vw[i].y : j == 2 ? vw[i].z : vw[i].w;
#pragma unroll
          for (int hi = 0; hi < 2; ++hi) {   // low halves of the words: even dims; high: odd
            const uint32_t x = prmt_b32(w[0], w[1], hi ? 0x7632u : 0x5410u);
            const uint32_t y = prmt_b32(w[2], w[3], hi ? 0x7632u : 0x5410u);
#pragma unroll
            for (int k = 0; k < 4; ++k)
              mma_16816(o[8 * j + 2 * k + hi], p[2 * m][0], p[2 * m][1], p[2 * m + 1][0],
                        p[2 * m + 1][1], widen_pair(x, k, qa), widen_pair(y, k, qb));
          }
        }
      }
      fence_async_smem();   // the reads come before the refill by the copy engine
      __syncwarp();
      issue();
    }

    // ---- join the warps: M, l first, then O eight rows at a time
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      l[r] += __shfl_xor_sync(0xffffffffu, l[r], 1);
      l[r] += __shfl_xor_sync(0xffffffffu, l[r], 2);
      if (t == 0) {
        sm.m[warp][g + 8 * r] = M[r];
        sm.l[warp][g + 8 * r] = l[r];
      }
    }
    __syncthreads();
    const bool whole = seg.whole;
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      float top = -INFINITY;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) top = fmaxf(top, sm.m[w][g + 8 * r]);
      const float f = M[r] == -INFINITY ? 0.f : exp2f(M[r] - top);
      if (r == 0 || g < kGroup - 8) {
#pragma unroll
        for (int e = 0; e < 32; ++e)   // column 8 e + c of a row is dim 32 c + e
          *reinterpret_cast<float2*>(&sm.join[warp][g][8 * e + 2 * t]) =
              make_float2(o[e][2 * r] * f, o[e][2 * r + 1] * f);
      }
      __syncthreads();
      // a thread sums eight dims of a row over the warps: dims 32 c + e0 .. + 7
      const int row = tid >> 5, c = (tid & 31) >> 2, e0 = 8 * (tid & 3);
      if (r == 0 || row < kGroup - 8) {
        float x[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = 0.f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w)
#pragma unroll
          for (int i = 0; i < 8; ++i) x[i] += sm.join[w][row][8 * (e0 + i) + c];
        const int hr = row + 8 * r;   // query head of the group
        float mt = -INFINITY, lt = 0.f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) mt = fmaxf(mt, sm.m[w][hr]);
#pragma unroll
        for (int w = 0; w < kWarps; ++w)
          lt += sm.m[w][hr] == -INFINITY ? 0.f : sm.l[w][hr] * exp2f(sm.m[w][hr] - mt);
        const int d = 32 * c + e0;
        if (whole) {
          const size_t at = (size_t)seg.b * kHeads + seg.plane * kGroup + hr;
          const float inv = lt > 0.f ? 1.0f / lt : (lt != lt ? lt : 0.f);
          const uint4 gt = __ldg(reinterpret_cast<const uint4*>(a.qg + at * kQgStride + kDim + d));
          const uint32_t gw[4] = {gt.x, gt.y, gt.z, gt.w};
          uint32_t res[4];
#pragma unroll
          for (int i = 0; i < 4; ++i)
            res[i] = pack_bf16x2(x[2 * i] * inv * sigmoid_f(lo_f(gw[i])),
                                 x[2 * i + 1] * inv * sigmoid_f(hi_f(gw[i])));
          *reinterpret_cast<uint4*>(a.out + at * kDim + d) = make_uint4(res[0], res[1], res[2], res[3]);
        } else {
          *part_at(a.part_o, seg.slot, d / 4, hr) = make_float4(x[0], x[1], x[2], x[3]);
          *part_at(a.part_o, seg.slot, d / 4 + 1, hr) = make_float4(x[4], x[5], x[6], x[7]);
          if ((tid & 31) == 0)
            reinterpret_cast<float2*>(a.part_ml)[(size_t)seg.slot * kV4Lanes + hr] = make_float2(mt, lt);
        }
      }
      __syncthreads();
    }
  }
  if (*abort) {   // the copies in flight land before the CTA leaves
    for (uint32_t f = issued > kStages ? issued - kStages : 0; f < issued; ++f)
      mbar_wait_quiet(&sm.full[warp][f % kStages], (f / kStages) & 1, 100000000LL);
  }
  __syncthreads();
  if (tid == 0 && sm.abort) record(a.status, sm.abort);
}

}  // namespace

cudaError_t decode4_set_attributes() {
  return cudaFuncSetAttribute(decode4_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                              (int)sizeof(D4Smem));
}

cudaError_t launch_decode4(const CUtensorMap& k_codes, const CUtensorMap& v_codes,
                           const CUtensorMap& k_scales, const CUtensorMap& v_scales,
                           const Verify4Args& a, int ctas, cudaStream_t s) {
  cudaLaunchAttribute attr[1];
  const cudaLaunchConfig_t cfg = overlapped_launch((unsigned)ctas, kThreads, sizeof(D4Smem), s, attr);
  const cudaError_t e = cudaLaunchKernelEx(&cfg, decode4_kernel, k_codes, v_codes, k_scales, v_scales, a);
  return e != cudaSuccess ? e : launch_verify4_combine(a, ctas, kKeys, ctas, s);
}

}  // namespace ga

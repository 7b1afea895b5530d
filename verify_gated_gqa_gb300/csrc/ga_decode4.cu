// Decode attention (one row per sequence) over 4-bit paged caches: ga_verify4.cu's results, for
// the twelve query rows that a (sequence, KV head) then has.
//
// Twelve rows would leave most of a 128-row tensor-core tile empty while every key and value
// still had to be widened through shared memory, so this form feeds mma.sync (16 rows) from
// registers: a lane's codes become its operand fragments where it holds them, and nothing
// widened is ever stored. What bounds it is the cache's bytes and the instructions that widen
// them, about equally (288 bytes and some 40 warp instructions a key of a head): 76 sequences of
// 16,383 keys in 161 us, 4.5 TB/s of codes; 64 of up to 8,192, ragged, in 54; one of 65,536 in 21.
//
// Work: streams (sequence, KV head) in granules of 32 keys, cut into equal runs, one per CTA, as in
// ga_v4.cuh. Eight computing warps a CTA; warp w takes a segment's granules w, w + 8, ... on its
// own, through two stages of its own (codes and scales of K and V, 9 KiB): it forms S = Q K^T, a
// running softmax and O += P V for all 16 rows and 256 dims in registers, and meets the other
// warps only at the segment's end, where their O, M and l are joined in shared memory. Four more
// warps fill the stages by TMA, each for two computing warps (done by the computing warps
// themselves, the page lookups and copies took a fifth of a granule's time).
//
// Fragments (m16n8k16; lane = 4 g + t). The order of the dims within Q K^T is free as long as Q
// and K agree: lane t of a key owns its dims 64t .. 64t + 63 (two 16-byte chunks of codes; the
// widened pairs of a word are the fragments of two k-steps in their natural order). For P V, lane
// g owns dims 32g .. + 31 of each V row (one chunk), so column g of n-tile e is dim 32 g + e; the
// halves of the words of two keys are joined before they are widened, so a fragment's two keys
// come out of one operation, with the scales of both in one register. With these choices every
// 16-byte read of the swizzled codes is free of bank conflicts.
#include <cstddef>

#include "ga_v4.cuh"

namespace ga {
namespace {

constexpr int kWarps = 8;
constexpr int kLoaders = 4;                        // loading warps, each for kWarps / kLoaders
constexpr int kThreads = 32 * (kWarps + kLoaders);
// Registers: launched at 168 a thread (384 x 168 = 64,512); the computing warps take 232, the loading
// ones keep 40: 128 x (2 x 232 + 40) = 64,512.
constexpr int kRegsCompute = 232, kRegsLoad = 40;
static_assert(128 * (2 * kRegsCompute + kRegsLoad) <= kThreads * 168, "register split");
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
  uint64_t full[kWarps][kStages], empty[kWarps][kStages];
  int abort;
};
static_assert(sizeof(D4Smem) <= 232448, "227 KiB of shared memory per CTA");
static_assert(offsetof(D4Smem, codes) % 1024 == 0 && kCodeBytes % 1024 == 0 && offsetof(D4Smem, scales) % 128 == 0,
              "tiles of the copies");
static_assert(offsetof(D4Smem, full) % 8 == 0 && offsetof(D4Smem, q) % 16 == 0 && offsetof(D4Smem, join) % 16 == 0,
              "barriers at 8 bytes, vectors at 16");

__device__ __forceinline__ void compute_sync() {   // the computing warps
  asm volatile("bar.sync 1, %0;" ::"n"(32 * kWarps) : "memory");
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

// ------------------------------------------------------------------ loading
// Loading warp lw fills the stages of computing warps 2 lw and 2 lw + 1: lane 4 i + c copies, for
// the i-th of them, c = 0: K codes, 1: V codes, 2, 3: their scales. A granule on a page outside the
// pool (recorded) is read past the pool's end: zeros.
__device__ void loader(D4Smem& sm, const CUtensorMap* tm_kc, const CUtensorMap* tm_vc,
                       const CUtensorMap* tm_ks, const CUtensorMap* tm_vs, const Verify4Args& a, int lw,
                       volatile int* abort) {
  constexpr int kEach = kWarps / kLoaders;
  const int lane = threadIdx.x & 31;
  if (lane >= 4 * kEach) return;
  const int w = kEach * lw + (lane >> 2), c = lane & 3;
  const CUtensorMap* map = c == 0 ? tm_kc : c == 1 ? tm_vc : c == 2 ? tm_ks : tm_vs;
  uint32_t issued = 0;
  Walk<kKeys> walk(sm.cut);
  Seg seg;
  while (walk.next(sm.cut, a.n_seq, seg)) {
    const int* table = a.page_table + (size_t)seg.b * a.max_pages;
    int page = 0, at = 0;   // of granule j, looked up a round ahead
    auto look_up = [&](int j) {
      if (j >= seg.n) return;
      const int key0 = (seg.kt0 + j) * kKeys, e = key0 / a.page_size;
      page = ld_input(table + e);
      at = seg.head * a.page_size + key0 - e * a.page_size;
    };
    look_up(w);
    for (int j = w; j < seg.n; j += kWarps) {
      int row = a.n_pages * kKvHeads * a.page_size;
      if (page >= 0 && page < a.n_pages) row = page * kKvHeads * a.page_size + at;
      else record(a.status, kDevBadPage);
      look_up(j + kWarps);
      const int st = (int)(issued % kStages);
      uint64_t* bar = &sm.full[w][st];
      if (!v4_wait(&sm.empty[w][st], ((issued / kStages) & 1) ^ 1, abort)) break;
      if (c == 0) mbar_arrive_expect_tx(bar, kStageBytes);   // (a copy may report its bytes before)
      tma_load_2d(c < 2 ? sm.codes[w][st][c] : sm.scales[w][st][c - 2], map, bar, 0, row);
      ++issued;
    }
    if (*abort) break;
  }
  if (*abort) {   // the copies in flight land before the CTA leaves
    for (uint32_t f = issued > kStages ? issued - kStages : 0; f < issued; ++f)
      mbar_wait_quiet(&sm.full[w][f % kStages], (f / kStages) & 1, 100000000LL);
  }
}

// ------------------------------------------------------------------ computing
// (A warp whose wait gave up goes on without computing, to meet the others at the barriers.)
__device__ void compute(D4Smem& sm, const Verify4Args& a, volatile int* abort) {
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int g = lane >> 2, t = lane & 3;
  uint32_t taken = 0;
  bool ok = true;
  Walk<kKeys> walk(sm.cut);
  Seg seg;
  while (walk.next(sm.cut, a.n_seq, seg)) {
    const int L = cut_len<kKeys>(sm.cut, seg.b, 1);
    // Q fragments of k-step i (of lane t's dims 64 t + 4 i .. + 3): rows g, g + 8 at the first two
    // of them, then at the last two; rows 12 .. 15 are zeros
#pragma unroll
    for (int i = 2 * warp; i < 2 * warp + 2; ++i) {
      const uint2* x = reinterpret_cast<const uint2*>(
          a.q_prep + ((size_t)seg.b * kHeads + seg.head * kGroup + g) * kDim + 64 * t + 4 * i);
      const uint2 lo = ld_input(x);
      const uint2 hi = g < kGroup - 8 ? ld_input(x + 8 * kDim / 4) : make_uint2(0u, 0u);
      sm.q[i][lane] = make_uint4(lo.x, hi.x, lo.y, hi.y);
    }
    compute_sync();
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
      if (lane == 0) mbar_arrive(&sm.empty[warp][st]);
    }

    // ---- join the warps: M, l first, then O eight rows at a time
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      l[r] += __shfl_xor_sync(0xffffffffu, l[r], 1);
      l[r] += __shfl_xor_sync(0xffffffffu, l[r], 2);
      if (l[r] != l[r]) M[r] = l[r];   // a NaN row weighs NaN, not nothing
      if (t == 0) {
        sm.m[warp][g + 8 * r] = M[r];
        sm.l[warp][g + 8 * r] = l[r];
      }
    }
    compute_sync();
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      float top = -INFINITY;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) top = fmaxf(top, sm.m[w][g + 8 * r]);
      const float f = M[r] == -INFINITY ? 0.f : exp2f(M[r] - top);
      if (r == 0 || g < kGroup - 8) {
#pragma unroll
        for (int e = 0; e < 32; ++e)   // place 8 e + c of a row is dim 32 c + e
          *reinterpret_cast<float2*>(&sm.join[warp][g][8 * e + 2 * t]) =
              make_float2(o[e][2 * r] * f, o[e][2 * r + 1] * f);
      }
      compute_sync();
      // a warp sums a row over the warps, a lane four neighbouring places at a time
      const int hr = warp + 8 * r;   // query head of the group
      if (hr < kGroup) {
        float mt = -INFINITY, lt = 0.f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) mt = fmaxf(mt, sm.m[w][hr]);
#pragma unroll
        for (int w = 0; w < kWarps; ++w)
          lt += sm.m[w][hr] == -INFINITY ? 0.f : sm.l[w][hr] * exp2f(sm.m[w][hr] - mt);
        const float inv = 1.0f / lt;
        const size_t out_row = (size_t)seg.b * kHeads + seg.head * kGroup + hr;
        float gate[2][4];
        if (seg.whole) {
#pragma unroll
          for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int k = 0; k < 4; ++k)
              gate[i][k] = lo_f(ld_input(a.qg + out_row * kQgStride + kDim + 32 * (4 * (lane & 1) + k) + 16 * i + (lane >> 1)));
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int p = 128 * i + 4 * lane;
          float x[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int w = 0; w < kWarps; ++w) {
            const float4 v = *reinterpret_cast<const float4*>(&sm.join[w][warp][p]);
            x[0] += v.x;
            x[1] += v.y;
            x[2] += v.z;
            x[3] += v.w;
          }
          if (seg.whole) {
            uint16_t* to = a.out + out_row * kDim + 32 * (p & 7) + (p >> 3);
#pragma unroll
            for (int k = 0; k < 4; ++k)
              to[32 * k] = (uint16_t)(pack_bf16x2(x[k] * inv * sigmoid_f(gate[i][k]), 0.f) & 0xFFFFu);
          } else {
            *part_at(a.part_o, seg.slot, p / 4, hr) = make_float4(x[0], x[1], x[2], x[3]);
            if (p == 0)
              reinterpret_cast<float2*>(a.part_ml)[(size_t)seg.slot * kV4Lanes + hr] = make_float2(lt != lt ? lt : mt, lt);
          }
        }
      }
      compute_sync();
    }
  }
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
  const int warp = threadIdx.x >> 5;
  volatile int* abort = &sm.abort;
  if (threadIdx.x == 0) {
    sm.abort = 0;
    for (int w = 0; w < kWarps; ++w)
      for (int i = 0; i < kStages; ++i) {
        mbar_init(&sm.full[w][i], 1);
        mbar_init(&sm.empty[w][i], 1);
      }
    mbar_fence_init();
  }
  if (warp == kWarps && (threadIdx.x & 31) == 0) {
    tma_prefetch_desc(&tm_kc);
    tma_prefetch_desc(&tm_vc);
    tma_prefetch_desc(&tm_ks);
    tma_prefetch_desc(&tm_vs);
  }
  grid_wait();
  grid_launch_dependents();
  make_cut<kKeys>(a, sm.cut, (int)gridDim.x, (int)blockIdx.x);   // two block barriers
  if (warp < kWarps) {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsCompute));
    compute(sm, a, abort);
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsLoad));
    loader(sm, &tm_kc, &tm_vc, &tm_ks, &tm_vs, a, warp - kWarps, abort);
  }
  __syncthreads();
  if (threadIdx.x == 0 && sm.abort) record(a.status, sm.abort);
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
  return e != cudaSuccess ? e : launch_verify4_combine(a, ctas, kKeys, s);
}

}  // namespace ga

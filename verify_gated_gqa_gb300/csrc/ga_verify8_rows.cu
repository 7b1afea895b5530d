// Verify attention over 8-bit paged caches, the form for five rows and more: query rows on the 128 rows
// of the MMAs. The numerics are those of ga_verify8.cu (queries and weights as two e4m3 parts, a scale
// per query row, and per row and block of 32 keys for the weights, sums relative to R).
//
// Why another form. With keys on the MMA's rows (ga_verify8.cu) the tensor cores read 32 KiB of codes
// twice, and the 16 G query rows or weights beside them, from shared memory for each product; at 96
// columns that and the softmax's exchanges are 390 KiB a tile, 3,100 cycles of shared memory for 1,900
// of arithmetic. Here the weights, and a quarter of the queries' parts, lie in tensor memory, each
// softmax thread has a query row of its own (its maximum, its sum and its scale need no exchange), and
// a tile costs 64 KiB + 48 KiB of operands for S and 64 KiB for O beside the 64 KiB that are loaded:
// bound by the tensor cores, 2,048 cycles a tile whatever the rows, which is why few rows take the
// other form: 8 x 65,536 keys with 4 rows 94.0 us there and 96.0 here, 64 x 8,192 keys 101 and 107, 256
// ragged sequences of up to 1,000 keys 65 and 78, 5 of up to 12,345 19.1 and 21.1 (3 rows: 93.1 and 94.5, 99
// and 105, 62 and 74, 18.6 and 20.6). With more rows, both as they were when they were compared, over 65,536
// keys: 5 rows 121 and 105, 8 rows 137 and 110, 16 rows 213 and 176.
//
// Structure (512 threads, 16 warps; the softmax's on three of the SM's four quarters):
//   warps w % 4 < 3  softmax: query rows 32 (w % 4) .. + 31, a row a lane, of the tile's keys 32 (w / 4) ..
//                    + 31, a block; they also split the queries and write the segment's result
//   warp 3           issues S = Q K^T (M = 128, N = 128 keys, K = 256 twice) of a tile, then O += W V (M =
//                    128, N = 256 dims, K = 32 keys; twice) of the tile before
//   warps 7, 11      load K and V tiles; warp 15 looks after tensor memory
// Tensor memory: O [0, 256), S [256, 384), W [384, 448) (32 columns a part), Q's first part, dims 0 ..
// 127 [448, 480), scale factors: of V, 1 and 2^-5 beside W's first and second part (256 dims, 8 columns
// each) [480, 496), of W [496, 500), of Q [500, 504). K's are V's ones.
// Every wait is bounded, as in ga_verify8.cu.
#include <cstddef>

#include "ga_v8.cuh"

namespace ga {
namespace {

constexpr int kThreads = 512;
constexpr int kTiles = 5, kKStages = 3, kVStages = kTiles - kKStages;
constexpr int kQBlockBytes = kV4Lanes * 128;           // 128 dims of one part of the query rows
constexpr uint32_t kTmemO = 0, kTmemS = 256, kTmemW = 384, kTmemQ = 448, kTmemSfV = 480, kTmemSfW = 496,
                   kTmemSfQ = 500;

struct Smem {
  uint8_t k[kKStages][kTileBytes], v[kVStages][kTileBytes];
  uint8_t q[3][kQBlockBytes];       // first part's dims 128 .. 255, second part (the MMA reads 32 rows past each)
  uint8_t q_first[kQBlockBytes];    // first part's dims 0 .. 127, on their way to tensor memory
  uint8_t sf_w[512], sf_q[512];
  float exchange[4][kV4Lanes];
  V4Cut cut;
  TileScales scales;
  uint64_t k_full[kKStages], k_empty[kKStages], v_full[kVStages], v_empty[kVStages];
  uint64_t q_full, s_full, s_free, p_full, p_free, o_done, o_free, drain;
  uint32_t tmem_base;
  int abort;
};
static_assert(sizeof(Smem) <= kSmemLimit, "227 KiB of shared memory per CTA");
static_assert(offsetof(Smem, q) % 1024 == 0 && kQBlockBytes % 1024 == 0 && offsetof(Smem, sf_w) % 128 == 0 &&
                  offsetof(Smem, scales) % 8 == 0 && offsetof(Smem, k_full) % 8 == 0,
              "swizzled blocks begin at whole atoms, barriers at 8 bytes");
static_assert(offsetof(Smem, q) + 2 * kQBlockBytes + 128 * 128 <= kSmemLimit,
              "128 rows can be read at the last query block");

// ------------------------------------------------------------------ MMA issue
#define GA_MMA "@e tcgen05.mma.cta_group::1.kind::mxf8f6f4.block_scale.scale_vec::1X "
// Four MMAs over 128 dims: A from shared memory, or from tensor memory (8 columns of it each).
__device__ __forceinline__ void mma_s_half_warp(uint32_t d, uint64_t a, uint64_t b, uint32_t id, uint32_t sf_a,
                                                uint32_t sf_b, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, e, t;\n\t.reg .b64 x, y;\n\t"
      "elect.sync _|e, 0xffffffff;\n\tsetp.ne.b32 p, %6, 0;\n\tsetp.eq.b32 t, 0, 0;\n\t"
      GA_MMA "[%0], %1, %2, %3, [%4], [%5], p;\n\t"
      "add.s64 x, %1, 2;\n\tadd.s64 y, %2, 2;\n\t" GA_MMA "[%0], x, y, %3, [%4], [%5], t;\n\t"
      "add.s64 x, %1, 4;\n\tadd.s64 y, %2, 4;\n\t" GA_MMA "[%0], x, y, %3, [%4], [%5], t;\n\t"
      "add.s64 x, %1, 6;\n\tadd.s64 y, %2, 6;\n\t" GA_MMA "[%0], x, y, %3, [%4], [%5], t;\n\t}\n" ::"r"(d),
      "l"(a), "l"(b), "r"(id), "r"(sf_a), "r"(sf_b), "r"(accumulate)
      : "memory");
}
__device__ __forceinline__ void mma_s_half_tmem_warp(uint32_t d, uint32_t a, uint64_t b, uint32_t id, uint32_t sf_a,
                                                     uint32_t sf_b, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, e, t;\n\t.reg .b32 x;\n\t.reg .b64 y;\n\t"
      "elect.sync _|e, 0xffffffff;\n\tsetp.ne.b32 p, %6, 0;\n\tsetp.eq.b32 t, 0, 0;\n\t"
      GA_MMA "[%0], [%1], %2, %3, [%4], [%5], p;\n\t"
      "add.u32 x, %1, 8;\n\tadd.s64 y, %2, 2;\n\t" GA_MMA "[%0], [x], y, %3, [%4], [%5], t;\n\t"
      "add.u32 x, %1, 16;\n\tadd.s64 y, %2, 4;\n\t" GA_MMA "[%0], [x], y, %3, [%4], [%5], t;\n\t"
      "add.u32 x, %1, 24;\n\tadd.s64 y, %2, 6;\n\t" GA_MMA "[%0], [x], y, %3, [%4], [%5], t;\n\t}\n" ::"r"(d),
      "r"(a), "l"(b), "r"(id), "r"(sf_a), "r"(sf_b), "r"(accumulate)
      : "memory");
}
// O: the blocks 0 .. steps - 1 of 32 keys of one part of the weights; block ks takes byte ks of the
// rows' scale words (bits 29, 30 of the descriptor).
__device__ __forceinline__ void mma_o_warp(uint32_t d, uint32_t a, uint64_t b, uint32_t id, uint32_t sf_a,
                                           uint32_t sf_b, uint32_t accumulate, uint32_t steps) {
  static_assert(kBoxBytes >> 4 == 256, "blocks of a tile");
  asm volatile(
      "{\n\t.reg .pred p, e, t;\n\t.reg .b32 x, i;\n\t.reg .b64 y;\n\t"
      "elect.sync _|e, 0xffffffff;\n\tsetp.ne.b32 p, %6, 0;\n\tsetp.eq.b32 t, 0, 0;\n\t"
      GA_MMA "[%0], [%1], %2, %3, [%4], [%5], p;\n\t"
      "setp.gt.and.u32 e, %7, 1, e;\n\tadd.u32 x, %1, 8;\n\tadd.s64 y, %2, 256;\n\tadd.u32 i, %3, 0x20000000;\n\t"
      GA_MMA "[%0], [x], y, i, [%4], [%5], t;\n\t"
      "setp.gt.and.u32 e, %7, 2, e;\n\tadd.u32 x, %1, 16;\n\tadd.s64 y, %2, 512;\n\tadd.u32 i, %3, 0x40000000;\n\t"
      GA_MMA "[%0], [x], y, i, [%4], [%5], t;\n\t"
      "setp.gt.and.u32 e, %7, 3, e;\n\tadd.u32 x, %1, 24;\n\tadd.s64 y, %2, 768;\n\tadd.u32 i, %3, 0x60000000;\n\t"
      GA_MMA "[%0], [x], y, i, [%4], [%5], t;\n\t}\n" ::"r"(d),
      "r"(a), "l"(b), "r"(id), "r"(sf_a), "r"(sf_b), "r"(accumulate), "r"(steps)
      : "memory");
}
#undef GA_MMA

struct Issue {
  Smem& sm;
  const uint32_t tmem;
  volatile int* abort;
  Ring k, v;
  uint32_t fs, fo;   // tiles whose S, O is issued
  __device__ __forceinline__ Issue(Smem& s, uint32_t t)
      : sm(s), tmem(t), abort(&s.abort), k(kKStages), v(kVStages), fs(0), fo(0) {}

  __device__ __forceinline__ bool s() {
    if (fs > 0 && !warp_wait(&sm.s_free, (fs - 1) & 1u, abort)) return false;
    if (!warp_wait(&sm.k_full[k.st], k.phase, abort)) return false;
    tc_fence_after();
    constexpr uint32_t kId = idesc_e4m3(kTileN, false, false);
    const uint64_t kd = sdesc_sw128(smem_u32(sm.k[k.st]), 16, 1024), qd = sdesc_sw128(smem_u32(sm.q[0]), 16, 1024);
    const uint32_t d = tmem + kTmemS, sf_q = tmem + kTmemSfQ, ones = tmem + kTmemSfV;
    mma_s_half_tmem_warp(d, tmem + kTmemQ, kd, kId, sf_q, ones, 0u);
    mma_s_half_warp(d, qd, kd + (kHalfBytes >> 4), kId, sf_q, ones, 1u);
    mma_s_half_warp(d, qd + (kQBlockBytes >> 4), kd, kId, sf_q, ones, 1u);
    mma_s_half_warp(d, qd + (2 * kQBlockBytes >> 4), kd + (kHalfBytes >> 4), kId, sf_q, ones, 1u);
    umma_commit_warp(&sm.k_empty[k.st]);
    umma_commit_warp(&sm.s_full);
    ++fs;
    k.next();
    return true;
  }

  // keys: the tile's; first: of the segment
  __device__ __forceinline__ bool o(int keys, bool first) {
    if (!warp_wait(&sm.v_full[v.st], v.phase, abort)) return false;
    const int steps = (keys + kQ8Block - 1) / kQ8Block;
    hide_values(sm.v[v.st], keys, steps);
    if (!warp_wait(&sm.p_full, fo & 1u, abort)) return false;
    tc_fence_after();
    copy_scales_warp(tmem + kTmemSfW, sdesc_plain(smem_u32(sm.sf_w), 16, 128));
    const uint64_t vd = sdesc_sw128(smem_u32(sm.v[v.st]), kHalfBytes, 1024);
    constexpr uint32_t kId = idesc_e4m3(kDim, false, true);
#pragma unroll
    for (int part = 0; part < 2; ++part)
      mma_o_warp(tmem + kTmemO, tmem + kTmemW + 32 * part, vd, kId, tmem + kTmemSfW, tmem + kTmemSfV + 8 * part,
                 !first || part > 0, (uint32_t)steps);
    umma_commit_warp(&sm.v_empty[v.st]);
    umma_commit_warp(&sm.p_free);
    ++fo;
    v.next();
    return true;
  }
};

__device__ void issue_mma(Smem& sm, const Verify4Args& a, uint32_t tmem) {
  Issue is(sm, tmem);
  Walk<kTileN, kQ8Rows> walk(sm.cut);
  Seg seg;
  uint32_t done = 0;
  while (walk.next(sm.cut, a.n_seq, seg)) {
    const int end = cut_len<kTileN>(sm.cut, seg.b, a.rows) + a.rows;
    if (!warp_wait(&sm.q_full, done & 1u, is.abort)) return;
    tc_fence_after();
    copy_scales_warp(tmem + kTmemSfQ, sdesc_plain(smem_u32(sm.sf_q), 16, 128));
    if (!is.s()) return;
    for (int j = 0; j < seg.n; ++j) {
      if (j + 1 < seg.n && !is.s()) return;
      if (j == 0 && done > 0 && !warp_wait(&sm.o_free, (done - 1) & 1u, is.abort)) return;
      if (!is.o(min(kTileN, end - (seg.kt0 + j) * kTileN), j == 0)) return;
    }
    umma_commit_warp(&sm.o_done);
    ++done;
  }
}

// ------------------------------------------------------------------ softmax
__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

__device__ void softmax_worker(Smem& sm, const Verify4Args& a, uint32_t tmem) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int quarter = warp & 3, block = warp >> 2;       // of the MMA's rows, of the tile's keys
  const int r = 32 * quarter + lane;
  const uint32_t lanes = (uint32_t)(32 * quarter) << 16;
  const int blocks = row_blocks(a.rows), heads = kGroup / blocks;
  const int rr = r / heads, hh = r - rr * heads;
  const bool valid = rr < a.rows;
  const int head_off = blocks == 2 ? heads * (int)(blockIdx.x & 1) : 0;
  volatile int* abort = &sm.abort;
  uint32_t f = 0, done = 0;
  // the four warps of the same rows meet
  auto meet = [&]() { asm volatile("bar.sync %0, 128;" ::"r"(1 + quarter) : "memory"); };
  auto meet_any = [&](bool x) { return team_any(1 + quarter, x); };
  // formed anew where it is used: the row's place, kept across the loops, would be spilled, and shared
  // memory leaves no L1 to spill to (64 x 16 rows over up to 4,096 keys 87.8 us against 82.8)
  auto anew = [](int x) {
    asm volatile("" : "+r"(x));
    return x;
  };
  // A segment's queries: eight rows a warp, eight dims a lane, so that a load takes whole lines (64 dims of
  // a row a thread touched 32 lines a load, and needed the other warps' maxima: 64 x 16 rows over up to
  // 4,096 keys 83.6 us against 81.8). Their places are free: this warp has seen the last S of the segment
  // before, so its products are done. What lies in tensor memory, a row a lane, goes there by way of
  // shared memory.
  auto load_queries = [&](const Seg& seg) {
    const int first = anew(32 * quarter + 8 * block), rows = heads * a.rows;
    uint4 x[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int row = min(first + i, rows - 1), wr = blocks == 2 ? row / (kGroup / 2) : row / kGroup;
      x[i] = ld_input(reinterpret_cast<const uint4*>(
                          a.q_prep + (uint32_t)((seg.b * a.rows + wr) * kHeads + seg.head * kGroup + head_off +
                                                row - wr * heads) * kDim) +
                      lane);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int row = first + i;
      if (row >= rows) x[i] = make_uint4(0u, 0u, 0u, 0u);
      const int e = query_exp(__reduce_max_sync(0xffffffffu, top_of(x[i])));
      const float inv = pow2i(-e);
      const uint32_t w[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
      uint32_t hi[4], lo[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float x0 = lo_f(w[k]) * inv, x1 = hi_f(w[k]) * inv;
        hi[k] = e4m3x2(x0, x1);
        const float2 y = f16x2_f32(e4m3x2_f16x2(hi[k]));
        lo[k] = e4m3x2(x0 - y.x, x1 - y.y);
      }
      // dims 0 .. 127 are the lower lanes'
      const uint32_t at = sw128_offset((uint32_t)row, (uint32_t)(lane & 15) >> 1) + (lane & 1) * 8;
      *reinterpret_cast<uint2*>((lane < 16 ? sm.q_first : sm.q[0]) + at) =
          make_uint2(hi[0] | hi[1] << 16, hi[2] | hi[3] << 16);
      *reinterpret_cast<uint2*>(sm.q[1 + (lane >> 4)] + at) = make_uint2(lo[0] | lo[1] << 16, lo[2] | lo[3] << 16);
      if (lane < 4) sm.sf_q[(row & 31) * 16 + (row >> 5) * 4 + lane] = (uint8_t)(e + kSfBias);
    }
    fence_async_smem();
    meet();
    if (block < 2) {   // 64 dims of this lane's row
      uint32_t w[16];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint4 v = *reinterpret_cast<const uint4*>(sm.q_first + sw128_offset((uint32_t)r, 4 * block + i));
        w[4 * i] = v.x; w[4 * i + 1] = v.y; w[4 * i + 2] = v.z; w[4 * i + 3] = v.w;
      }
      tc_fence_after();
      tmem_st16(tmem + kTmemQ + lanes + 16 * block, w);
      tmem_wait_st();
      tc_fence_before();
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(&sm.q_full);
  };
  const uint32_t s_at = tmem + kTmemS + lanes + 32 * block, w_at = tmem + kTmemW + lanes + 8 * block;
  const uint32_t sf_at = smem_u32(sm.sf_w) + (r & 31) * 16 + (r >> 5) * 4 + block;
  Walk<kTileN, kQ8Rows> walk(sm.cut);
  Seg seg, next;
  bool more = walk.next(sm.cut, a.n_seq, seg);
  if (more) load_queries(seg);
  for (; more; seg = next) {
    const int L = cut_len<kTileN>(sm.cut, seg.b, a.rows);
    const int limit = L + min(rr, a.rows - 1);   // the row's last visible key
    float l = 0.f, R = -INFINITY;                // of this block's keys; of the row
    for (int j = 0; j < seg.n; ++j, ++f) {
      const int key0 = (seg.kt0 + j) * kTileN + kQ8Block * block;
      const uint32_t scales = sm.scales.wait(f, block, abort);
      const float factor = pow2i(q8_exp(scales)) * kLog2eOver16;   // from S to exponents
      const int v_exp = q8_exp(scales >> 8);
      warp_wait(&sm.s_full, f & 1u, abort);
      tc_fence_after();
      uint32_t s[32];
      tmem_ld32(s_at, s);
      tmem_wait_ld(s);
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm.s_free);
      if (key0 + kQ8Block - 1 > L) {   // some key of the block is hidden from some row
#pragma unroll
        for (int i = 0; i < 32; ++i)
          if (key0 + i > limit) s[i] = 0xFF800000u;   // -inf: weight 0, never the maximum
      }
      auto v = [&](int i) { return __uint_as_float(s[i]); };
      float m0 = max3(v(0), v(1), v(2)), m1 = max3(v(3), v(4), v(5));
#pragma unroll
      for (int i = 6; i + 3 < 32; i += 4) {
        m0 = max3(m0, v(i), v(i + 1));
        m1 = max3(m1, v(i + 2), v(i + 3));
      }
      const float top = fmaxf(max3(m0, m1, v(30)), v(31));
      float E = first_exponent(top, factor), d = kTop - E;   // what the block's weights are scaled by
      if (is_large(E)) {
        E = large_exponent(E, top, factor);
        d = kTop - E;
        if (fabsf(E) >= kFar) {   // the differences to the largest score
#pragma unroll
          for (int i = 0; i < 32; ++i) s[i] = __float_as_uint(v(i) - top);
          d = kTop;
        }
      }
      if (meet_any(E - R > kMove)) {
        // R moves, for the rows of these warps (a segment's first tile: from nothing)
        sm.exchange[block][r] = E;
        meet();
        float to = R;
#pragma unroll
        for (int i = 0; i < 4; ++i) to = fmaxf(to, sm.exchange[i][r]);
        const float move = to == R ? 1.0f : ex2_approx(R - to);
        R = to;
        l *= move;
        if (j > 0) {
          // O holds every product before it is scaled, a quarter of the dims by each warp
          warp_wait(&sm.p_free, (f - 1) & 1u, abort);
          tc_fence_after();
#pragma unroll 1
          for (int c0 = 64 * block; c0 < 64 * block + 64; c0 += 32) {
            uint32_t o[32];
            tmem_ld32(tmem + kTmemO + lanes + c0, o);
            tmem_wait_ld(o);
#pragma unroll
            for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * move);
            tmem_st32(tmem + kTmemO + lanes + c0, o);
          }
          tmem_wait_st();
          tc_fence_before();
        }
        meet();   // the exchange is read
      }
      const float x = E - R - kTop;   // (E - R is exact where it matters, E - kTop is not for every E)
      float l0 = 0.f, l1 = 0.f;
      uint32_t hi[8], lo[8];
#pragma unroll
      for (int i = 0; i < 32; i += 4) {
        const float p0 = ex2_approx(fmaf(v(i), factor, d)), p1 = ex2_approx(fmaf(v(i + 1), factor, d));
        const float p2 = ex2_approx(fmaf(v(i + 2), factor, d)), p3 = ex2_approx(fmaf(v(i + 3), factor, d));
        l0 += p0 + p1;
        l1 += p2 + p3;
        split_weights(hi[i / 4], lo[i / 4], p0, p1, p2, p3);
      }
      l = fmaf(l0 + l1, ex2_approx(x), l);
      // the weights' and the scales' places: O's products of the tile before have read them
      if (f > 0) warp_wait(&sm.p_free, (f - 1) & 1u, abort);
      tc_fence_after();
      tmem_st8(w_at, hi);
      tmem_st8(w_at + 32, lo);
      asm volatile("st.shared.u8 [%0], %1;" ::"r"(sf_at), "r"(scale_byte(x, v_exp)) : "memory");
      tmem_wait_st();
      tc_fence_before();
      fence_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm.p_full);
    }
    more = walk.next(sm.cut, a.n_seq, next);
    if (more) load_queries(next);
    // the segment's result: a quarter of the dims by each warp
    warp_wait(&sm.o_done, done & 1u, abort);
    tc_fence_after();
    sm.exchange[block][r] = l;
    meet();
    const float sum = (sm.exchange[0][r] + sm.exchange[1][r]) + (sm.exchange[2][r] + sm.exchange[3][r]);
    meet();   // the exchange is read
    if (valid && !seg.whole && block == 0)   // a NaN row's part weighs NaN, not nothing
      reinterpret_cast<float2*>(a.part_ml)[(size_t)seg.slot * kV4Lanes + r] =
          make_float2(sum != sum ? sum : sum == 0.f ? -INFINITY : R, sum);
    const float inv = 1.0f / sum;
    const uint32_t row = (uint32_t)((seg.b * a.rows + anew(rr)) * kHeads + seg.head * kGroup + head_off + hh);
    const uint4* gp = reinterpret_cast<const uint4*>(a.qg + row * kQgStride + kDim + 64 * block);
    uint4* op = reinterpret_cast<uint4*>(a.out + row * kDim + 64 * block);
#pragma unroll 1
    for (int c = 0; c < 2; ++c) {
      uint4 g[4];
      if (seg.whole) {
#pragma unroll
        for (int i = 0; i < 4; ++i) g[i] = valid ? ld_input(gp + 4 * c + i) : make_uint4(0u, 0u, 0u, 0u);
      }
      uint32_t o[32];
      tmem_ld32(tmem + kTmemO + lanes + 64 * block + 32 * c, o);
      tmem_wait_ld(o);
      if (!valid) continue;
      if (seg.whole) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint32_t gw[4] = {g[i].x, g[i].y, g[i].z, g[i].w};
          uint32_t res[4];
#pragma unroll
          for (int k = 0; k < 4; ++k)
            res[k] = pack_bf16x2(__uint_as_float(o[8 * i + 2 * k]) * inv * sigmoid_f(lo_f(gw[k])),
                                 __uint_as_float(o[8 * i + 2 * k + 1]) * inv * sigmoid_f(hi_f(gw[k])));
          op[4 * c + i] = make_uint4(res[0], res[1], res[2], res[3]);
        }
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
          *part_at(a.part_o, seg.slot, 16 * block + 8 * c + i, r) =
              make_float4(__uint_as_float(o[4 * i]), __uint_as_float(o[4 * i + 1]), __uint_as_float(o[4 * i + 2]),
                          __uint_as_float(o[4 * i + 3]));
      }
    }
    tc_fence_before();
    __syncwarp();
    if (lane == 0) mbar_arrive(&sm.o_free);
    ++done;
  }
}

__global__ void __launch_bounds__(kThreads, 1)
    verify8_rows_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                        const __grid_constant__ Verify8Args a, int box_keys) {
  extern __shared__ __align__(1024) uint8_t raw[];
  if ((smem_u32(raw) & 1023u) != 0u) {
    if (threadIdx.x == 0) record(a.v.status, kDevBadLaunch);
    return;
  }
  Smem& sm = *reinterpret_cast<Smem*>(raw);
  const int warp = threadIdx.x >> 5;
  // quarters of the MMA's rows that hold query rows, four warps each
  const int quarters = (a.v.rows * (kGroup / row_blocks(a.v.rows)) + 31) / 32;
  if (threadIdx.x == 0) {
    const uint32_t warps = 4u * quarters;
    sm.abort = 0;
    for (int i = 0; i < kKStages; ++i) {
      mbar_init(&sm.k_full[i], 1);
      mbar_init(&sm.k_empty[i], 1);
    }
    for (int i = 0; i < kVStages; ++i) {
      mbar_init(&sm.v_full[i], 1);
      mbar_init(&sm.v_empty[i], 1);
    }
    sm.scales.init();
    mbar_init(&sm.q_full, warps);
    mbar_init(&sm.s_full, 1);
    mbar_init(&sm.s_free, warps);
    mbar_init(&sm.p_full, warps);
    mbar_init(&sm.p_free, 1);
    mbar_init(&sm.o_done, 1);
    mbar_init(&sm.o_free, warps);
    mbar_init(&sm.drain, 1);
    mbar_fence_init();
  }
  if (warp == 7 && (threadIdx.x & 31) == 0) {
    tma_prefetch_desc(&tm_k);
    tma_prefetch_desc(&tm_v);
  }
  // scales of the rows without a query row, whose results nothing reads
  if (threadIdx.x < 256) reinterpret_cast<uint32_t*>(sm.sf_w)[threadIdx.x] = 0u;
  grid_wait();
  grid_launch_dependents();
  if (warp == 15) {   // after the wait: the kernel before may still need tensor memory until it ends
    tmem_alloc(&sm.tmem_base, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  {   // two block barriers
    const int blocks = row_blocks(a.v.rows);
    make_cut<kTileN, kQ8Rows>(a.v, sm.cut, (int)gridDim.x / blocks, (int)blockIdx.x / blocks);
  }
  tc_fence_after();
  const uint32_t tmem = sm.tmem_base;
  if (warp < 4) {   // the values' scale factors
    uint32_t w[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) w[i] = i < 8 ? 0x7F7F7F7Fu : 0x7A7A7A7Au;
    tmem_st16(tmem + kTmemSfV + ((uint32_t)(warp * 32) << 16), w);
    tmem_wait_st();
    tc_fence_before();
  }
  fence_async_smem();
  __syncthreads();
  tc_fence_after();
  if (sm.cut.run_tiles() > 0) {
    if (warp == 3) {
      issue_mma(sm, a.v, tmem);
      umma_commit_warp(&sm.drain);
      mbar_wait_quiet(&sm.drain, 0, 100000000LL);
    } else if (warp == 7) {
      load_tiles<kQ8Rows>(a, sm.cut, &tm_k, a.k_scales, 0, sm.k[0], kKStages, box_keys, sm.k_full, sm.k_empty,
                          sm.scales, &sm.abort);
    } else if (warp == 11) {
      load_tiles<kQ8Rows>(a, sm.cut, &tm_v, a.v_scales, 1, sm.v[0], kVStages, box_keys, sm.v_full, sm.v_empty,
                          sm.scales, &sm.abort);
    } else if ((warp & 3) < quarters) {
      softmax_worker(sm, a.v, tmem);
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 15) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
  if (threadIdx.x == 0 && sm.abort) record(a.v.status, sm.abort);
}

}  // namespace

cudaError_t verify8_rows_set_attributes() {
  return cudaFuncSetAttribute(verify8_rows_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemLimit);
}

cudaError_t launch_verify8_rows(const CUtensorMap& k_codes, const CUtensorMap& v_codes, const Verify8Args& a,
                                int ctas, cudaStream_t s) {
  const int blocks = row_blocks(a.v.rows), workers = ctas / blocks;
  cudaLaunchAttribute attr[1];
  const cudaLaunchConfig_t cfg = overlapped_launch((unsigned)(workers * blocks), kThreads, kSmemLimit, s, attr);
  const cudaError_t e =
      cudaLaunchKernelEx(&cfg, verify8_rows_kernel, k_codes, v_codes, a, verify8_box_keys(a.v.page_size));
  return e != cudaSuccess ? e : launch_verify4_combine(a.v, workers, kTileN, kQ8Rows, s);
}

}  // namespace ga

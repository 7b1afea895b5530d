// Decode and verify attention over 8-bit paged caches (format: ga_q8.cuh).
//
// Per sequence with L cached tokens before the window, window row r (position L + r) sees keys
// 0 .. L + r; with s_j = q . k_j / 16, out = (sum_j e^(s_j) v_j / sum_j e^(s_j)) sigmoid(gate).
//
// The codes go from memory to the tensor cores as they are: nothing widens them. The other operand
// comes as a sum of two e4m3 parts. A bf16 query has 8 significant bits, so two parts of 4 hold it
// (to 2^-17 of its row's largest magnitude, where the second part runs out of exponents); of a
// softmax weight they keep 9 bits, one more than bf16 would. Products are summed in fp32.
// Both products are formed transposed, S^T = K Q^T and O^T = V^T W^T, with keys or dims on the 128
// rows of an MMA and the query rows on its columns, so that an MMA's size follows the rows of the
// call: 16 columns for one row of 12 heads, 96 for eight.
//
// Scales are powers of two, and the MMAs (kind::mxf8f6f4, a scale per row or column and 32 of K) take
// them back: each query row is scaled to its largest magnitude; weights are scaled per column and
// block of 32 keys, to 256 at the block's largest, and their scale carries the value block's. A key
// block's goes into the factor from S to exponents, one number for a warp. So a weight's precision is relative to its own block's largest, not the row's: the
// others keep theirs beside a key that outweighs them by far but has a small value. R, the exponent
// that a column's O and sum are kept relative to, is the first tile's and moves only when a block
// passes it by 2^64.
//
// Work. A stream is (sequence, KV head), cut into tiles of 128 keys and the tiles among the CTAs as in
// the 4-bit form (ga_v4.cuh), two CTAs side by side for more than 96 columns; parts of a stream are
// merged by its combine kernel.
//
// Structure (128 + 128 G threads; G groups of 16 columns):
//   warp 0      issues S^T = K Q^T (M = 128 keys, N = 16 G, K = 256 twice)
//   warp 1      issues O^T += V^T W^T (M = 128 dims twice, N = 16 G, K = 32 keys; twice)
//   warps 2, 3  load K and V tiles by TMA, boxes of 32 keys x 128 dims
//   warps 4 ..  softmax: four warps per group, warp q with the tile's keys 32 q .. + 31, a block, a
//               key a lane; they also split the queries and write the segment's result
// Tensor memory: O^T dims 0..127 [0, 96), dims 128..255 [96, 192), S^T two buffers [192, 384), scale
// factors 1 and 2^-5 (of K, and of V beside the weights' first and second part) [384, 392), those of
// W^T, two buffers [392, 400), of Q [400, 404).
// Every wait is bounded; a wait that gives up raises the CTA's abort flag, which the others see.
#include <cstddef>

#include "ga_q8.cuh"
#include "ga_v4.cuh"

namespace ga {
namespace {

constexpr int kCols = 16;                              // columns of a group
constexpr int kMaxGroups = kV4Lanes / kCols;           // 6
constexpr int kMaxThreads = 128 + 128 * kMaxGroups;
constexpr int kTileBytes = kTileN * kQ8RowBytes;       // 32 KiB: two blocks of [128 keys][128 dims]
constexpr int kHalfBytes = kTileBytes / 2;
constexpr int kBoxBytes = kQ8Block * 128;              // 32 keys x 128 dims
constexpr int kMaxStages = 3;                          // tiles in flight of K, and of V
constexpr int kGroupBytes = kTileN * kCols;            // a group's weights of a tile, one part
constexpr uint32_t kTmemO = 0, kTmemS = 192, kTmemSfV = 384, kTmemSfW = 392, kTmemSfQ = 400;
constexpr uint32_t kTmemBuf = kV4Lanes;                // columns between S's buffers, and O's halves
constexpr float kLog2eOver16 = 1.4426950408889634f / 16.0f;
constexpr float kTop = 8.0f;          // a block's largest weight becomes at most 2^8
constexpr float kMove = 64.0f;        // R moves when a block passes it by more than 2^64
constexpr float kNone = -1e30f;       // the exponent of a block without a visible key
constexpr int kSfBias = 127;          // of a scale factor's 8 exponent bits

struct Ctl {
  V4Cut cut;
  int vote[kMaxGroups][2];
  uint64_t k_full[kMaxStages], k_empty[kMaxStages], v_full[kMaxStages], v_empty[kMaxStages];
  uint64_t q_full, s_full[2], s_free[2], p_full[2], p_empty[2], o_done, o_free;
  uint64_t group[kMaxGroups];
  uint64_t drain_qk, drain_pv;
  uint32_t tmem_base;
  int abort;
};
// Shared memory: the tiles of K, then V, the queries (two parts of two halves of [16 G][128]), the
// weights (two buffers of two parts of G groups of [128 keys][16]), scale factors (two buffers of the
// weights', the queries'; 512 bytes each), Ctl.
struct Layout {
  int groups, stages;        // stages of K, and of V
  __host__ __device__ int k(int st) const { return st * kTileBytes; }
  __host__ __device__ int v(int st) const { return (stages + st) * kTileBytes; }
  __host__ __device__ int q() const { return 2 * stages * kTileBytes; }
  __host__ __device__ int q_part() const { return groups * kCols * kDim; }
  __host__ __device__ int p(int buf) const { return q() + 2 * q_part() + buf * 2 * groups * kGroupBytes; }
  __host__ __device__ int p_part() const { return groups * kGroupBytes; }
  __host__ __device__ int sf(int buf) const { return p(2) + buf * 512; }
  __host__ __device__ int sf_q() const { return sf(2); }
  __host__ __device__ int ctl() const { return sf(3); }
  __host__ __device__ int bytes() const { return ctl() + (int)sizeof(Ctl); }
};
constexpr int kSmemLimit = 232448;
constexpr int layout_bytes(int groups, int stages) {
  return 2 * stages * kTileBytes + groups * (2 * kCols * kDim + 4 * kGroupBytes) + 3 * 512 + (int)sizeof(Ctl);
}
static_assert(layout_bytes(kMaxGroups, 2) <= kSmemLimit, "two stages fit with every width");
static_assert(sizeof(Ctl) % 8 == 0 && offsetof(Ctl, k_full) % 8 == 0, "barriers at 8 bytes");

// ------------------------------------------------------------------ tensor cores
// Instruction descriptor of the block-scaled MMA, e4m3 operands, M = 128. Bits: [4, 6) which byte of
// B's scale words; 15, 16 A, B with rows (M, N) contiguous instead of K; [17, 23) N >> 3; 23 scales of 8
// exponent bits; [24, 29) M >> 4.
__host__ __device__ constexpr uint32_t idesc_e4m3(int N, bool rows_contiguous, uint32_t byte) {
  return (byte << 4) | (rows_contiguous ? 3u << 15 : 0u) | ((uint32_t)(N >> 3) << 17) | (1u << 23) |
         ((128u >> 4) << 24);
}
// Unswizzled operand, rows contiguous: 16 rows x 8 of K are 128 consecutive bytes; the next 8 of K
// are `lbo` bytes on, the next 16 rows `sbo`. Also the source of a copy of scale factors.
__device__ __forceinline__ uint64_t sdesc_plain(uint32_t saddr, uint32_t lbo, uint32_t sbo) {
  return (uint64_t)((saddr & 0x3FFFFu) >> 4) | ((uint64_t)((lbo >> 4) & 0x3FFFu) << 16) |
         ((uint64_t)((sbo >> 4) & 0x3FFFu) << 32) | ((uint64_t)1 << 46);
}
__device__ __forceinline__ void mma_e4m3_warp(uint32_t d, uint64_t a, uint64_t b, uint32_t id, uint32_t sf_a,
                                              uint32_t sf_b, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, e;\n\t"
      "elect.sync _|e, 0xffffffff;\n\t"
      "setp.ne.b32 p, %6, 0;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::mxf8f6f4.block_scale.scale_vec::1X [%0], %1, %2, %3, [%4], [%5], p;\n\t}\n" ::
          "r"(d),
      "l"(a), "l"(b), "r"(id), "r"(sf_a), "r"(sf_b), "r"(accumulate)
      : "memory");
}
// 512 bytes of scale factors to four columns of tensor memory, in all four quarters of its lanes:
// column n's word is at byte (n % 32) 16 + (n / 32) 4. In order with the MMAs of the same thread.
__device__ __forceinline__ void copy_scales_warp(uint32_t taddr, uint64_t desc) {
  asm volatile(
      "{\n\t.reg .pred e;\n\t"
      "elect.sync _|e, 0xffffffff;\n\t"
      "@e tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;\n\t}\n" ::"r"(taddr),
      "l"(desc)
      : "memory");
}
__device__ __forceinline__ void tmem_ld8(uint32_t taddr, uint32_t (&r)[8]) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
               : "r"(taddr));
}
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
      "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}

// A ring of stages: the stage and how often it has come round.
struct Ring {
  int st, n;
  uint32_t phase;
  __device__ __forceinline__ explicit Ring(int stages) : st(0), n(stages), phase(0u) {}
  __device__ __forceinline__ void next() {
    if (++st == n) {
      st = 0;
      phase ^= 1u;
    }
  }
};

struct Cta {
  uint8_t* smem;
  Layout lay;
  Ctl& ctl;
  const Verify8Args& a;
  uint32_t tmem;
  volatile int* abort;
  __device__ __forceinline__ int blocks() const { return row_blocks(a.v.rows); }
};

// ------------------------------------------------------------------ loading
// A tile: boxes of 32 keys x 128 dims by lanes 0 .. 7. Blocks of 32 keys without one of the sequence
// are not loaded; on a page outside the pool (recorded) they are read past its end, which gives zeros.
__device__ void load_tiles(const Cta& c, const CUtensorMap* map, bool is_v) {
  const Verify4Args& a = c.a.v;
  const int lane = threadIdx.x & 31, block = (lane >> 1) & 3, half = lane & 1;
  uint64_t* full = is_v ? c.ctl.v_full : c.ctl.k_full;
  uint64_t* empty = is_v ? c.ctl.v_empty : c.ctl.k_empty;
  const long long n_rows = (long long)a.n_pages * kKvHeads * a.page_size;
  Ring ring(c.lay.stages);
  uint32_t issued = 0;
  Walk<kTileN> walk(c.ctl.cut);
  Seg seg;
  while (walk.next(c.ctl.cut, a.n_seq, seg)) {
    const int end = cut_len<kTileN>(c.ctl.cut, seg.b, a.rows) + a.rows;
    const int* table = a.page_table + (size_t)seg.b * a.max_pages;
    int page = 0, at = 0;
    bool in = false;
    auto look_up = [&](int kt) {   // a tile ahead
      const int key0 = kt * kTileN + kQ8Block * block;
      in = key0 < end;
      if (!in) return;
      const int e = key0 / a.page_size;
      page = ld_input(table + e);
      at = seg.head * a.page_size + key0 - e * a.page_size;
    };
    look_up(seg.kt0);
    for (int j = 0; j < seg.n; ++j, ++issued, ring.next()) {
      int row = (int)n_rows;
      if (in) {
        if (page >= 0 && page < a.n_pages) row = page * kKvHeads * a.page_size + at;
        else if (lane < 8) record(a.status, kDevBadPage);
      }
      const int st = ring.st;
      if (!warp_wait(&empty[st], ring.phase ^ 1u, c.abort)) break;
      const int loaded = min(4, (end - (seg.kt0 + j) * kTileN + kQ8Block - 1) / kQ8Block);
      if (lane == 0) mbar_arrive_expect_tx(&full[st], 2 * kBoxBytes * loaded);
      __syncwarp();
      if (lane < 8 && in)
        tma_load_2d(c.smem + (is_v ? c.lay.v(st) : c.lay.k(st)) + half * kHalfBytes + block * kBoxBytes, map,
                    &full[st], 128 * half, row);
      if (j + 1 < seg.n) look_up(seg.kt0 + j + 1);
    }
    if (*c.abort) break;
  }
  if (*c.abort) {   // the copies in flight land before the CTA leaves
    const uint32_t n = c.lay.stages;
    for (uint32_t i = issued > n ? issued - n : 0; i < issued; ++i)
      mbar_wait_quiet(&full[i % n], (i / n) & 1u, 100000000LL);
  }
}

// ------------------------------------------------------------------ MMA issue
__device__ void issue_qk(const Cta& c) {
  const int N = c.lay.groups * kCols;
  const uint32_t id = idesc_e4m3(N, false, 0);
  const uint64_t q_desc = sdesc_sw128(smem_u32(c.smem + c.lay.q()), 16, 1024);
  const uint64_t k_desc = sdesc_sw128(smem_u32(c.smem), 16, 1024);
  Ring ring(c.lay.stages);
  Walk<kTileN> walk(c.ctl.cut);
  Seg seg;
  uint32_t f = 0, done = 0;
  while (walk.next(c.ctl.cut, c.a.v.n_seq, seg)) {
    if (!warp_wait(&c.ctl.q_full, done & 1u, c.abort)) return;
    tc_fence_after();
    copy_scales_warp(c.tmem + kTmemSfQ, sdesc_plain(smem_u32(c.smem + c.lay.sf_q()), 16, 128));
    for (int j = 0; j < seg.n; ++j, ++f, ring.next()) {
      const uint32_t buf = f & 1u;
      if (!warp_wait(&c.ctl.s_free[buf], ((f >> 1) & 1u) ^ 1u, c.abort)) return;
      if (!warp_wait(&c.ctl.k_full[ring.st], ring.phase, c.abort)) return;
      tc_fence_after();
      const uint64_t kd = k_desc + (uint64_t)(c.lay.k(ring.st) >> 4);
#pragma unroll
      for (int part = 0; part < 2; ++part)
#pragma unroll
        for (int ks = 0; ks < 8; ++ks)
          mma_e4m3_warp(c.tmem + kTmemS + buf * kTmemBuf, kd + (uint64_t)((ks >> 2) * (kHalfBytes >> 4) + (ks & 3) * 2),
                        q_desc + (uint64_t)((part * c.lay.q_part() + (ks >> 2) * N * 128) >> 4) + (ks & 3) * 2, id,
                        c.tmem + kTmemSfV, c.tmem + kTmemSfQ, (part > 0 || ks > 0) ? 1u : 0u);
      umma_commit_warp(&c.ctl.k_empty[ring.st]);
      umma_commit_warp(&c.ctl.s_full[buf]);
    }
    ++done;
  }
}

__device__ void issue_pv(const Cta& c) {
  const Verify4Args& a = c.a.v;
  const int N = c.lay.groups * kCols, lane = threadIdx.x & 31;
  const uint64_t v_desc = sdesc_sw128(smem_u32(c.smem), kHalfBytes, 1024);
  Ring ring(c.lay.stages);
  Walk<kTileN> walk(c.ctl.cut);
  Seg seg;
  uint32_t f = 0, done = 0;
  while (walk.next(c.ctl.cut, a.n_seq, seg)) {
    const int end = cut_len<kTileN>(c.ctl.cut, seg.b, a.rows) + a.rows;
    if (done > 0 && !warp_wait(&c.ctl.o_free, (done - 1) & 1u, c.abort)) return;
    for (int j = 0; j < seg.n; ++j, ++f, ring.next()) {
      const uint32_t buf = f & 1u;
      if (!warp_wait(&c.ctl.v_full[ring.st], ring.phase, c.abort)) return;
      const int keys = min(kTileN, end - (seg.kt0 + j) * kTileN), steps = (keys + kQ8Block - 1) / kQ8Block;
      if (keys < steps * kQ8Block) {   // whatever lies past the last key counts as 0: it may be NaN codes
        uint8_t* tile = c.smem + c.lay.v(ring.st);
        const uint32_t zero[4] = {0u, 0u, 0u, 0u};
        for (int i = keys * 8 + lane; i < steps * kQ8Block * 8; i += 32)
#pragma unroll
          for (int h = 0; h < 2; ++h) sts_v4(smem_u32(tile + h * kHalfBytes + i * 16), zero);
        fence_async_smem();
        __syncwarp();
      }
      if (!warp_wait(&c.ctl.p_full[buf], (f >> 1) & 1u, c.abort)) return;
      tc_fence_after();
      const uint32_t sf = c.tmem + kTmemSfW + 4 * buf;
      copy_scales_warp(sf, sdesc_plain(smem_u32(c.smem + c.lay.sf((int)buf)), 16, 128));
      const uint64_t vd = v_desc + (uint64_t)(c.lay.v(ring.st) >> 4);
      const uint64_t pd = sdesc_plain(smem_u32(c.smem + c.lay.p((int)buf)), 128, kGroupBytes);
#pragma unroll
      for (int part = 0; part < 2; ++part)
#pragma unroll
        for (int ks = 0; ks < 4; ++ks)
          if (ks < steps) {
#pragma unroll
            for (int h = 0; h < 2; ++h)
              mma_e4m3_warp(c.tmem + kTmemO + h * kTmemBuf, vd + (uint64_t)((h * kHalfBytes + ks * kBoxBytes) >> 4),
                            pd + (uint64_t)((part * c.lay.p_part() + ks * 512) >> 4),
                            idesc_e4m3(N, true, (uint32_t)ks), c.tmem + kTmemSfV + 4 * part, sf,
                            (j > 0 || part > 0 || ks > 0) ? 1u : 0u);
          }
      umma_commit_warp(&c.ctl.v_empty[ring.st]);
      umma_commit_warp(&c.ctl.p_empty[buf]);
    }
    umma_commit_warp(&c.ctl.o_done);
    ++done;
  }
}

// ------------------------------------------------------------------ softmax
__device__ __forceinline__ float warp_max(float x) {
  float r;
  asm("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(x));
  return r;
}
// a x + b of a pair by one operation, and a x.
__device__ __forceinline__ uint64_t pair(float lo, float hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ float2 unpair(uint64_t x) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(x));
  return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t x, uint64_t b) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(x), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t x) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(x));
  return r;
}
// 32 p - 32 hi of a pair, hi as halves; both exact.
__device__ __forceinline__ float2 rest_x32(uint64_t p32, uint32_t hi) {
  const float2 p = unpair(p32);
  float2 r;
  asm("{\n\t.reg .b16 l, h, m;\n\tmov.b32 {l, h}, %2;\n\tmov.b16 m, 0xD000;\n\t"   // -32
      "fma.rn.f32.f16 %0, l, m, %3;\n\tfma.rn.f32.f16 %1, h, m, %4;\n\t}"
      : "=f"(r.x), "=f"(r.y)
      : "r"(hi), "f"(p.x), "f"(p.y));
  return r;
}

// The exponent that a query row is divided by: its largest magnitude is at most 448 of it.
__device__ __forceinline__ int query_exp(uint32_t top) {
  const int e = (int)(top >> 7) - 127 - 8 + ((top & 127u) > 96u ? 1 : 0);
  return min(max(e, -100), 100);
}

__device__ void softmax_worker(const Cta& c) {
  const Verify4Args& a = c.a.v;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int quarter = warp & 3, group = (warp - 4) >> 2, col0 = group * kCols;
  const uint32_t lanes = (uint32_t)(quarter * 32) << 16;
  const int blocks = c.blocks(), heads = kGroup / blocks, cols = heads * a.rows;
  const int head_off = blocks == 2 ? heads * (int)(blockIdx.x & 1) : 0;
  const int key = quarter * kQ8Block + lane;   // this thread's of a tile
  uint32_t f = 0, done = 0, syncs = 0;
  // the four warps of the group
  auto arrive = [&]() {
    __syncwarp();
    if (lane == 0) mbar_arrive(&c.ctl.group[group]);
  };
  auto wait = [&]() { return warp_wait(&c.ctl.group[group], syncs++ & 1u, c.abort); };
  Walk<kTileN> walk(c.ctl.cut);
  Seg seg;
  while (walk.next(c.ctl.cut, a.n_seq, seg)) {
    const int L = cut_len<kTileN>(c.ctl.cut, seg.b, a.rows), end = L + a.rows;
    const int head0 = seg.head * kGroup + head_off;
    // this warp's block of a tile: its page, and its scales
    const int* table = a.page_table + (size_t)seg.b * a.max_pages;
    auto look_up = [&](int kt) {
      const int key0 = kt * kTileN + kQ8Block * quarter;
      return key0 < end ? ld_input(table + key0 / a.page_size) : -1;
    };
    auto scales = [&](int kt, int page, uint32_t& k, uint32_t& v) {
      k = v = (uint32_t)-kQ8MinExp;
      if (page < 0 || page >= a.n_pages) return;
      const int key0 = kt * kTileN + kQ8Block * quarter;
      const size_t at = ((size_t)page * kKvHeads + seg.head) * (a.page_size / kQ8Block) + key0 % a.page_size / kQ8Block;
      k = ld_input(c.a.k_scales + at);
      v = ld_input(c.a.v_scales + at);
    };
    uint32_t kb, vb;
    int page_next;
    {
      const int page = look_up(seg.kt0);
      page_next = seg.n > 1 ? look_up(seg.kt0 + 1) : -1;
      scales(seg.kt0, page, kb, vb);
    }
    {   // queries: four columns a warp, 8 dims a lane. Their place is free: this warp has seen the last
        // S of the segment before, so its products are done
      uint4 x[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int col = col0 + 4 * quarter + i, rr = col / heads;
        x[i] = make_uint4(0u, 0u, 0u, 0u);
        if (col < cols)
          x[i] = ld_input(reinterpret_cast<const uint4*>(
                              a.q_prep + (((size_t)seg.b * a.rows + rr) * kHeads + head0 + col - rr * heads) * kDim) +
                          lane);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int col = col0 + 4 * quarter + i;
        const int e = query_exp(__reduce_max_sync(0xffffffffu, top_of(x[i])));
        const float inv = pow2i(-e);
        const uint32_t w[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
        uint32_t hi[4], lo[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const float x0 = lo_f(w[k]) * inv, x1 = hi_f(w[k]) * inv;
          hi[k] = e4m3x2(x0, x1);
          const float2 h = f16x2_f32(e4m3x2_f16x2(hi[k]));
          lo[k] = e4m3x2(x0 - h.x, x1 - h.y);
        }
        const int N = c.lay.groups * kCols;
        uint8_t* at = c.smem + c.lay.q() + (lane >> 4) * N * 128 + sw128_offset((uint32_t)col, (uint32_t)(lane & 15) >> 1) +
                      (lane & 1) * 8;
        *reinterpret_cast<uint2*>(at) = make_uint2(hi[0] | hi[1] << 16, hi[2] | hi[3] << 16);
        *reinterpret_cast<uint2*>(at + c.lay.q_part()) = make_uint2(lo[0] | lo[1] << 16, lo[2] | lo[3] << 16);
        if (lane < 4) c.smem[c.lay.sf_q() + (col & 31) * 16 + (col >> 5) * 4 + lane] = (uint8_t)(e + kSfBias);
      }
      fence_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&c.ctl.q_full);
    }
    uint64_t l[kCols / 2];   // this key's sums, pairs of columns
#pragma unroll
    for (int i = 0; i < kCols / 2; ++i) l[i] = 0u;
    float R = -INFINITY;     // of column lane % 16
    for (int j = 0; j < seg.n; ++j, ++f) {
      const uint32_t buf = f & 1u;
      const int kt = seg.kt0 + j;
      const float factor = pow2i(q8_exp(kb)) * kLog2eOver16;   // from S to exponents
      const int v_exp = q8_exp(vb);
      if (j + 1 < seg.n) {   // the next tile's scales, and the page of the one after
        scales(kt + 1, page_next, kb, vb);
        page_next = j + 2 < seg.n ? look_up(kt + 2) : -1;
      }
      if (!warp_wait(&c.ctl.s_full[buf], (f >> 1) & 1u, c.abort)) return;
      tc_fence_after();
      uint32_t s[kCols];
      tmem_ld16(c.tmem + kTmemS + buf * kTmemBuf + lanes + col0, s);
      tmem_wait_ld(s);
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&c.ctl.s_free[buf]);
      if (kt * kTileN + kTileN - 1 > L) {   // some key of the tile is hidden from some row
        const int last = kt * kTileN + key - L;   // this key is seen by rows from `last` on
#pragma unroll
        for (int i = 0; i < kCols; ++i)
          if ((col0 + i) / heads < last) s[i] = 0xFF800000u;   // -inf: weight 0, never the maximum
      }
      // the block's exponents, a column a lane: E, what its weights are scaled by
      float top = 0.f;
#pragma unroll
      for (int i = 0; i < kCols; ++i) {
        const float m = warp_max(__uint_as_float(s[i]));
        if ((lane & 15) == i) top = m;
      }
      const float E = fmaxf(ceilf(top * factor), kNone);
      if (E > R + kMove) c.ctl.vote[group][buf] = (int)f + 1;
      arrive();
      if (!warp_wait(&c.ctl.p_empty[buf], ((f >> 1) & 1u) ^ 1u, c.abort)) return;
      if (!wait()) return;
      // this warp's part of the tile's weights: a place for exchanges until they are written
      float* slab = reinterpret_cast<float*>(c.smem + c.lay.p((int)buf) + group * kGroupBytes) + quarter * (kQ8Block * kCols / 4);
      if (*(volatile int*)&c.ctl.vote[group][buf] == (int)f + 1) {
        // R moves, for all of the group (a segment's first tile: from nothing)
        if (lane < kCols) slab[lane] = E;
        arrive();
        if (!wait()) return;
        const float* other = slab - quarter * (kQ8Block * kCols / 4) + (lane & 15);
        const float to = fmaxf(fmaxf(fmaxf(other[0], other[kQ8Block * kCols / 4]),
                                     fmaxf(other[kQ8Block * kCols / 2], other[3 * kQ8Block * kCols / 4])), R);
        const float move = to == R ? 1.0f : ex2_approx(R - to);
        R = to;
        if (j > 0) {
          // O holds every product before it is scaled
          if (!warp_wait(&c.ctl.p_empty[buf ^ 1u], ((f - 1) >> 1) & 1u, c.abort)) return;
          tc_fence_after();
#pragma unroll 1
          for (int h = 0; h < 2; ++h) {
            uint32_t o[kCols];
            tmem_ld16(c.tmem + kTmemO + h * kTmemBuf + lanes + col0, o);
            tmem_wait_ld(o);
#pragma unroll
            for (int i = 0; i < kCols; ++i)
              o[i] = __float_as_uint(__uint_as_float(o[i]) * __shfl_sync(0xffffffffu, move, i));
            tmem_st16(c.tmem + kTmemO + h * kTmemBuf + lanes + col0, o);
          }
          tmem_wait_st();
          tc_fence_before();
        }
#pragma unroll
        for (int i = 0; i < kCols; i += 2)
          l[i / 2] = mul2(l[i / 2], pair(__shfl_sync(0xffffffffu, move, i), __shfl_sync(0xffffffffu, move, i + 1)));
        arrive();   // every warp has read the exchange
        if (!wait()) return;
      }
      const float x = E - kTop - R;
      if (lane < kCols) {
        const int col = col0 + lane;
        c.smem[c.lay.sf((int)buf) + (col & 31) * 16 + (col >> 5) * 4 + quarter] =
            (uint8_t)max(0, (int)x + v_exp + kSfBias);
        slab[lane] = kTop - E;
        slab[kCols + lane] = ex2_approx(x);
      }
      __syncwarp();
      uint32_t hi[kCols / 4], lo[kCols / 4];
      const uint64_t factor2 = pair(factor, factor), x32 = pair(32.0f, 32.0f);
#pragma unroll
      for (int i = 0; i < kCols; i += 4) {
        const ulonglong2 d = *reinterpret_cast<const ulonglong2*>(slab + i);
        const ulonglong2 g = *reinterpret_cast<const ulonglong2*>(slab + kCols + i);
        uint32_t h[2], r[2];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const float2 e = unpair(fma2(pair(__uint_as_float(s[i + 2 * k]), __uint_as_float(s[i + 2 * k + 1])), factor2,
                                       k ? d.y : d.x));
          const float2 p = make_float2(ex2_approx(e.x), ex2_approx(e.y));
          const uint64_t p2 = pair(p.x, p.y);
          l[i / 2 + k] = fma2(p2, k ? g.y : g.x, l[i / 2 + k]);
          h[k] = e4m3x2(p.x, p.y);
          const float2 rest = rest_x32(mul2(p2, x32), e4m3x2_f16x2(h[k]));
          r[k] = e4m3x2(rest.x, rest.y);
        }
        hi[i / 4] = prmt_b32(h[0], h[1], 0x5410u);
        lo[i / 4] = prmt_b32(r[0], r[1], 0x5410u);
      }
      __syncwarp();   // the slab is read
      const uint32_t at = smem_u32(slab) + lane * kCols;
      sts_v4(at, hi);
      sts_v4(at + c.lay.p_part(), lo);
      fence_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&c.ctl.p_full[buf]);
    }
    // the segment's result: sums over the keys, column i's in lane i
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < kCols; ++i) {
      const float2 both = unpair(l[i / 2]);
      float x = i & 1 ? both.y : both.x;
#pragma unroll
      for (int off = 16; off; off >>= 1) x += __shfl_xor_sync(0xffffffffu, x, off);
      if (lane == i) sum = x;
    }
    if (!warp_wait(&c.ctl.o_done, done & 1u, c.abort)) return;
    tc_fence_after();
    {
      float* ex = reinterpret_cast<float*>(c.smem + c.lay.p(0) + group * kGroupBytes);
      if (lane < kCols) ex[quarter * kCols + lane] = sum;
      arrive();
      if (!wait()) return;
      if (lane < kCols) {
        sum = (ex[lane] + ex[kCols + lane]) + (ex[2 * kCols + lane] + ex[3 * kCols + lane]);
        if (!seg.whole && quarter == 0 && col0 + lane < cols)   // a NaN row's part weighs NaN, not nothing
          reinterpret_cast<float2*>(a.part_ml)[(size_t)seg.slot * kV4Lanes + col0 + lane] =
              make_float2(sum != sum ? sum : sum == 0.f ? -INFINITY : R, sum);
      }
    }
    const float inv = 1.0f / sum;
    // O, 8 columns of half of the dims at a time, a dim a lane
#pragma unroll 1
    for (int at = 0; at < 4; ++at) {
      constexpr int kAtOnce = kCols / 2;
      const int d = 128 * (at >> 1) + 32 * quarter + lane, i0 = kAtOnce * (at & 1);
      uint32_t o[kAtOnce];
      tmem_ld8(c.tmem + kTmemO + (at >> 1) * kTmemBuf + lanes + col0 + i0, o);
      tmem_wait_ld(o);
      // columns by (row, head) as they come
      int rr = (col0 + i0) / heads, hh = col0 + i0 - rr * heads;
      uint16_t gate[kAtOnce];
      if (seg.whole) {
        int r2 = rr, h2 = hh;
#pragma unroll
        for (int i = 0; i < kAtOnce; ++i) {
          gate[i] = 0;
          if (r2 < a.rows)
            gate[i] = ld_input(a.qg + (((size_t)seg.b * a.rows + r2) * kHeads + head0 + h2) * kQgStride + kDim + d);
          if (++h2 == heads) {
            h2 = 0;
            ++r2;
          }
        }
      }
#pragma unroll
      for (int i = 0; i < kAtOnce; ++i) {
        const float x = __uint_as_float(o[i]);
        const float scale = __shfl_sync(0xffffffffu, inv, i0 + i);
        if (rr < a.rows) {
          if (seg.whole)
            a.out[(((size_t)seg.b * a.rows + rr) * kHeads + head0 + hh) * kDim + d] =
                (uint16_t)(pack_bf16x2(x * scale * sigmoid_f(lo_f(gate[i])), 0.f) & 0xFFFFu);
          else
            a.part_o[((size_t)seg.slot * kV4Lanes + col0 + i0 + i) * kDim + d] = x;
        }
        if (++hh == heads) {
          hh = 0;
          ++rr;
        }
      }
    }
    tc_fence_before();
    __syncwarp();
    if (lane == 0) mbar_arrive(&c.ctl.o_free);
    ++done;
  }
}

__global__ void __launch_bounds__(kMaxThreads, 1)
    verify8_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                   const __grid_constant__ Verify8Args a, const Layout lay) {
  extern __shared__ __align__(1024) uint8_t smem[];
  if ((smem_u32(smem) & 1023u) != 0u) {
    if (threadIdx.x == 0) record(a.v.status, kDevBadLaunch);
    return;
  }
  Ctl& ctl = *reinterpret_cast<Ctl*>(smem + lay.ctl());
  const int warp = threadIdx.x >> 5;
  if (threadIdx.x == 0) {
    const uint32_t warps = 4u * lay.groups;
    ctl.abort = 0;
    for (int i = 0; i < kMaxStages; ++i) {
      mbar_init(&ctl.k_full[i], 1);
      mbar_init(&ctl.k_empty[i], 1);
      mbar_init(&ctl.v_full[i], 1);
      mbar_init(&ctl.v_empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&ctl.s_full[i], 1);
      mbar_init(&ctl.s_free[i], warps);
      mbar_init(&ctl.p_full[i], warps);
      mbar_init(&ctl.p_empty[i], 1);
    }
    for (int i = 0; i < kMaxGroups; ++i) {
      mbar_init(&ctl.group[i], 4);
      ctl.vote[i][0] = ctl.vote[i][1] = 0;
    }
    mbar_init(&ctl.q_full, warps);
    mbar_init(&ctl.o_done, 1);
    mbar_init(&ctl.o_free, warps);
    mbar_init(&ctl.drain_qk, 1);
    mbar_init(&ctl.drain_pv, 1);
    mbar_fence_init();
  }
  if (warp == 2 && (threadIdx.x & 31) == 0) {
    tma_prefetch_desc(&tm_k);
    tma_prefetch_desc(&tm_v);
  }
  // scales of columns past the groups are read by the copies and used by nothing
  for (int i = threadIdx.x; i < 3 * 512 / 4; i += blockDim.x) reinterpret_cast<uint32_t*>(smem + lay.sf(0))[i] = 0u;
  grid_wait();
  grid_launch_dependents();
  if (warp == 1) {   // after the wait: the kernel before may still need tensor memory until it ends
    tmem_alloc(&ctl.tmem_base, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  {   // two block barriers
    const int blocks = row_blocks(a.v.rows);
    make_cut<kTileN>(a.v, ctl.cut, (int)gridDim.x / blocks, (int)blockIdx.x / blocks);
  }
  tc_fence_after();
  const uint32_t tmem = ctl.tmem_base;
  if (warp >= 4 && warp < 8) {   // the values' scale factors: 1 beside the weights' first part, 2^-5
    const uint32_t w[8] = {0x7F7F7F7Fu, 0x7F7F7F7Fu, 0x7F7F7F7Fu, 0x7F7F7F7Fu,
                           0x7A7A7A7Au, 0x7A7A7A7Au, 0x7A7A7A7Au, 0x7A7A7A7Au};
    tmem_st8(tmem + kTmemSfV + ((uint32_t)((warp & 3) * 32) << 16), w);
    tmem_wait_st();
    tc_fence_before();
  }
  __syncthreads();
  tc_fence_after();
  const Cta c = {smem, lay, ctl, a, tmem, &ctl.abort};
  if (ctl.cut.run_tiles() > 0) {
    if (warp == 0) {
      issue_qk(c);
      umma_commit_warp(&ctl.drain_qk);
      mbar_wait_quiet(&ctl.drain_qk, 0, 100000000LL);
    } else if (warp == 1) {
      issue_pv(c);
      umma_commit_warp(&ctl.drain_pv);
      mbar_wait_quiet(&ctl.drain_pv, 0, 100000000LL);
    } else if (warp < 4) {
      load_tiles(c, warp == 2 ? &tm_k : &tm_v, warp == 3);
    } else {
      softmax_worker(c);
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
  if (threadIdx.x == 0 && ctl.abort) record(a.v.status, ctl.abort);
}

}  // namespace

cudaError_t verify8_set_attributes() {
  return cudaFuncSetAttribute(verify8_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemLimit);
}

cudaError_t launch_verify8(const CUtensorMap& k_codes, const CUtensorMap& v_codes, const Verify8Args& a,
                           int sm_count, cudaStream_t s) {
  const int ctas = sm_count < kV4MaxCtas ? sm_count : kV4MaxCtas;
  const int blocks = row_blocks(a.v.rows), workers = ctas / blocks;
  const int cols = a.v.rows * (kGroup / blocks);
  Layout lay;
  lay.groups = (cols + kCols - 1) / kCols;
  lay.stages = layout_bytes(lay.groups, kMaxStages) <= kSmemLimit ? kMaxStages : 2;
  cudaLaunchAttribute attr[1];
  const cudaLaunchConfig_t cfg = overlapped_launch((unsigned)(workers * blocks), (unsigned)(128 + 128 * lay.groups),
                                                   (size_t)lay.bytes(), s, attr);
  const cudaError_t e = cudaLaunchKernelEx(&cfg, verify8_kernel, k_codes, v_codes, a, lay);
  return e != cudaSuccess ? e : launch_verify4_combine(a.v, workers, kTileN, true, s);
}

}  // namespace ga

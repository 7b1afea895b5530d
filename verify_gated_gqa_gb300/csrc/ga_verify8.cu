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
// Structure (128 + 128 T threads, G groups of 16 columns, T teams of four warps with at most two groups
// each):
//   warp 0      issues S^T = K Q^T (M = 128 keys, N = 16 G, K = 256 twice) of a tile, then O^T +=
//               V^T W^T (M = 128 dims twice, N = 16 G, K = 32 keys; twice) of the tile before
//   warps 2, 3  load K and V tiles by TMA, and their blocks' scales
//   warps 4 ..  softmax: warp q of a team takes the tile's keys 32 q .. + 31, a block, a key a lane;
//               they also split the queries and write the segment's result. (A team for each group
//               left 72 registers a thread and spent half of its instructions on waits and addresses:
//               8 x 8 rows over 65,536 keys in 136 us.)
// Tensor memory: O^T dims 0..127 [0, 96), dims 128..255 [96, 192), S^T two buffers [192, 384), scale
// factors 1 and 2^-5 (of K, and of V beside the weights' first and second part) [384, 392), those of
// W^T, two buffers [392, 400), of Q [400, 404).
// Every wait is bounded; a wait that gives up raises the CTA's abort flag, which the others see. A
// team's four warps meet at a named barrier in every tile; they run all their tiles even after an
// abort (their waits then return at once), so that none is left there.
#include <cstddef>

#include "ga_q8.cuh"
#include "ga_v4.cuh"

namespace ga {
namespace {

constexpr int kCols = 16;                              // columns of a group
constexpr int kMaxGroups = kV4Lanes / kCols;           // 6
constexpr int kTeamGroups = 2;                         // of a team at most
constexpr int kMaxTeams = kMaxGroups / kTeamGroups;
constexpr int kMaxThreads = 128 + 128 * kMaxTeams;
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

constexpr int kScaleTiles = 8;        // tiles whose scales are kept (no role is that far ahead)

struct Ctl {
  V4Cut cut;
  uint8_t scales[kScaleTiles][4][2];   // a tile's blocks': of K, of V
  uint64_t scales_full[kScaleTiles];
  uint64_t k_full[kMaxStages], k_empty[kMaxStages], v_full[kMaxStages], v_empty[kMaxStages];
  uint64_t q_full, s_full[2], s_free[2], p_full[2], p_done[2], o_done, o_free, drain;
  uint32_t tmem_base;
  int abort;
};
// Shared memory: the tiles of K, then V, the queries (two parts of two halves of [16 G][128]), the
// weights (two buffers of two parts of G groups of [128 keys][16]), scale factors (two buffers of the
// weights', the queries'; 512 bytes each), Ctl.
struct Layout {
  int groups, teams, stages;   // stages of K, and of V
  int box_keys;              // of a tensor load
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
static_assert(sizeof(Ctl) % 8 == 0 && offsetof(Ctl, scales_full) % 8 == 0 && offsetof(Ctl, k_full) % 8 == 0,
              "barriers at 8 bytes");
static_assert(kScaleTiles > kMaxStages + 3, "the loaders cannot pass a tile that the softmax has yet to reach");

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
// Eight MMAs of a converged warp, issued by one lane with one election. S: both halves of the dims of
// one part of Q, operands 32 bytes on, `kb` and `qb` (in 16 bytes) at the second half.
#define GA_MMA "@e tcgen05.mma.cta_group::1.kind::mxf8f6f4.block_scale.scale_vec::1X "
__device__ __forceinline__ void mma_s_warp(uint32_t d, uint64_t a, uint64_t b, uint32_t half_b, uint32_t id,
                                           uint32_t sf_a, uint32_t sf_b, uint32_t accumulate) {
  static_assert(kHalfBytes >> 4 == 1024, "the second half of a tile");
  asm volatile(
      "{\n\t.reg .pred p, e, t;\n\t.reg .b64 a, b, h;\n\t"
      "elect.sync _|e, 0xffffffff;\n\t"
      "setp.ne.b32 p, %7, 0;\n\tsetp.eq.b32 t, 0, 0;\n\tcvt.u64.u32 h, %3;\n\t"
      GA_MMA "[%0], %1, %2, %4, [%5], [%6], p;\n\t"
      "add.s64 a, %1, 2;\n\tadd.s64 b, %2, 2;\n\t" GA_MMA "[%0], a, b, %4, [%5], [%6], t;\n\t"
      "add.s64 a, %1, 4;\n\tadd.s64 b, %2, 4;\n\t" GA_MMA "[%0], a, b, %4, [%5], [%6], t;\n\t"
      "add.s64 a, %1, 6;\n\tadd.s64 b, %2, 6;\n\t" GA_MMA "[%0], a, b, %4, [%5], [%6], t;\n\t"
      "add.s64 h, %2, h;\n\t"
      "add.s64 a, %1, 1024;\n\t" GA_MMA "[%0], a, h, %4, [%5], [%6], t;\n\t"
      "add.s64 a, %1, 1026;\n\tadd.s64 b, h, 2;\n\t" GA_MMA "[%0], a, b, %4, [%5], [%6], t;\n\t"
      "add.s64 a, %1, 1028;\n\tadd.s64 b, h, 4;\n\t" GA_MMA "[%0], a, b, %4, [%5], [%6], t;\n\t"
      "add.s64 a, %1, 1030;\n\tadd.s64 b, h, 6;\n\t" GA_MMA "[%0], a, b, %4, [%5], [%6], t;\n\t}\n" ::"r"(d),
      "l"(a), "l"(b), "r"(half_b), "r"(id), "r"(sf_a), "r"(sf_b), "r"(accumulate)
      : "memory");
}
// O: both halves of the dims for the blocks 0 .. steps - 1 of 32 keys, one part of the weights; block
// ks takes byte ks of the weights' scale words.
__device__ __forceinline__ void mma_o_warp(uint32_t d0, uint32_t d1, uint64_t a, uint64_t b, uint32_t id,
                                           uint32_t sf_a, uint32_t sf_b, uint32_t accumulate, uint32_t steps) {
  static_assert(kHalfBytes >> 4 == 1024 && kBoxBytes >> 4 == 256, "blocks of a tile");
  asm volatile(
      "{\n\t.reg .pred p, e, t;\n\t.reg .b64 x, y;\n\t.reg .b32 i;\n\t"
      "elect.sync _|e, 0xffffffff;\n\t"
      "setp.ne.b32 p, %7, 0;\n\tsetp.eq.b32 t, 0, 0;\n\t"
      GA_MMA "[%0], %2, %3, %4, [%5], [%6], p;\n\t"
      "add.s64 x, %2, 1024;\n\t" GA_MMA "[%1], x, %3, %4, [%5], [%6], p;\n\t"
      "setp.gt.and.u32 e, %8, 1, e;\n\tadd.u32 i, %4, 16;\n\tadd.s64 y, %3, 32;\n\t"
      "add.s64 x, %2, 256;\n\t" GA_MMA "[%0], x, y, i, [%5], [%6], t;\n\t"
      "add.s64 x, %2, 1280;\n\t" GA_MMA "[%1], x, y, i, [%5], [%6], t;\n\t"
      "setp.gt.and.u32 e, %8, 2, e;\n\tadd.u32 i, %4, 32;\n\tadd.s64 y, %3, 64;\n\t"
      "add.s64 x, %2, 512;\n\t" GA_MMA "[%0], x, y, i, [%5], [%6], t;\n\t"
      "add.s64 x, %2, 1536;\n\t" GA_MMA "[%1], x, y, i, [%5], [%6], t;\n\t"
      "setp.gt.and.u32 e, %8, 3, e;\n\tadd.u32 i, %4, 48;\n\tadd.s64 y, %3, 96;\n\t"
      "add.s64 x, %2, 768;\n\t" GA_MMA "[%0], x, y, i, [%5], [%6], t;\n\t"
      "add.s64 x, %2, 1792;\n\t" GA_MMA "[%1], x, y, i, [%5], [%6], t;\n\t}\n" ::"r"(d0),
      "r"(d1), "l"(a), "l"(b), "r"(id), "r"(sf_a), "r"(sf_b), "r"(accumulate), "r"(steps)
      : "memory");
}
#undef GA_MMA
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
// A box of the tile's dims 128 half .. + 127 (all of them where the box covers the tile), by one lane of
// a converged warp.
__device__ __forceinline__ void load_box_warp(uint32_t dst, const CUtensorMap* map, uint64_t* bar, int row, int half) {
  asm volatile(
      "{\n\t.reg .pred e;\n\t"
      "elect.sync _|e, 0xffffffff;\n\t"
      "@e cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5}], [%2];\n\t}\n" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(0), "r"(row), "r"(half)
      : "memory");
}
// Tiles of K or V, in boxes of as many keys as pages hold a multiple of (32, 64 or 128; a tile in one
// box, or a box for each half of the dims). Boxes without a key of the sequence are not loaded; on a
// page outside the pool (recorded) they are read past its end, which gives zeros. The warp's lanes
// look after a block of 32 keys each, lane b % 4 after block b.
__device__ void load_tiles(const Cta& c, const CUtensorMap* map, bool is_v) {
  const Verify4Args& a = c.a.v;
  const int lane = threadIdx.x & 31, block = lane & 3, box_keys = c.lay.box_keys;
  uint64_t* full = is_v ? c.ctl.v_full : c.ctl.k_full;
  uint64_t* empty = is_v ? c.ctl.v_empty : c.ctl.k_empty;
  const int n_rows = a.n_pages * kKvHeads * a.page_size;   // below 2^31
  const uint8_t* scale_pool = is_v ? c.a.v_scales : c.a.k_scales;
  Ring ring(c.lay.stages);
  uint32_t issued = 0;
  Walk<kTileN, true> walk(c.ctl.cut);
  Seg seg;
  while (walk.next(c.ctl.cut, a.n_seq, seg)) {
    const int end = cut_len<kTileN>(c.ctl.cut, seg.b, a.rows) + a.rows;
    const int* table = a.page_table + (size_t)seg.b * a.max_pages;
    // this lane's block of a tile: its page is looked up two tiles ahead, its scale loaded one
    struct Block {
      int page = -1, off = 0;
      bool in = false;
      uint32_t scale = 0;
    };
    auto look_up = [&](int j) {
      Block b;
      const int key0 = (seg.kt0 + j) * kTileN + kQ8Block * block;
      b.in = j < seg.n && key0 < end;
      if (b.in) {
        const int e = key0 / a.page_size;
        b.page = ld_input(table + e);
        b.off = key0 - e * a.page_size;
      }
      return b;
    };
    auto load_scale = [&](Block& b) {
      b.scale = (uint32_t)-kQ8MinExp;
      if (b.in && (unsigned)b.page < (unsigned)a.n_pages)
        b.scale = ld_input(scale_pool + ((size_t)b.page * kKvHeads + seg.head) * (a.page_size / kQ8Block) +
                           b.off / kQ8Block);
    };
    Block now = look_up(0), next = look_up(1);
    load_scale(now);
    for (int j = 0; j < seg.n; ++j, ++issued, ring.next()) {
      load_scale(next);
      const Block after = look_up(j + 2);
      int row = n_rows;
      if (now.in) {
        if ((unsigned)now.page < (unsigned)a.n_pages)
          row = (now.page * kKvHeads + seg.head) * a.page_size + now.off;
        else if (lane < 4) record(a.status, kDevBadPage);
      }
      const int st = ring.st, left = end - (seg.kt0 + j) * kTileN;   // keys
      if (!warp_wait(&empty[st], ring.phase ^ 1u, c.abort)) break;
      const int boxes = left >= kTileN ? kTileN / box_keys : (left + box_keys - 1) / box_keys;
      mbar_expect_tx_warp(&full[st], (uint32_t)(boxes * box_keys * kQ8RowBytes));
      __syncwarp();
      const uint32_t dst = smem_u32(c.smem + (is_v ? c.lay.v(st) : c.lay.k(st)));
      if (box_keys == kTileN) {
        load_box_warp(dst, map, &full[st], __shfl_sync(0xffffffffu, row, 0), 0);
      } else {
        for (int b = 0; b < boxes; ++b) {
          const int r = __shfl_sync(0xffffffffu, row, b * box_keys / kQ8Block);
          load_box_warp(dst + b * box_keys * 128, map, &full[st], r, 0);
          load_box_warp(dst + kHalfBytes + b * box_keys * 128, map, &full[st], r, 1);
        }
      }
      if (lane < 4) c.ctl.scales[issued % kScaleTiles][block][is_v] = (uint8_t)now.scale;
      __syncwarp();
      if (lane == 0) mbar_arrive(&c.ctl.scales_full[issued % kScaleTiles]);
      now = next;
      next = after;
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
// In this order: S of tile 0, S of 1, O of 0, S of 2, O of 1, ... of a segment, so that tile f's S
// tells that O's products of tile f - 2 are done, and their weights' place is free.
struct Issue {
  const Cta& c;
  const int N;
  const uint64_t q_desc, tile_desc_k, tile_desc_v;
  Ring k, v;
  uint32_t fs, fo;   // tiles whose S, O is issued
  __device__ __forceinline__ explicit Issue(const Cta& c_)
      : c(c_), N(c_.lay.groups * kCols), q_desc(sdesc_sw128(smem_u32(c_.smem + c_.lay.q()), 16, 1024)),
        tile_desc_k(sdesc_sw128(smem_u32(c_.smem), 16, 1024)),
        tile_desc_v(sdesc_sw128(smem_u32(c_.smem), kHalfBytes, 1024)), k(c_.lay.stages), v(c_.lay.stages), fs(0),
        fo(0) {}

  __device__ __forceinline__ bool s() {
    const uint32_t buf = fs & 1u;
    if (!warp_wait(&c.ctl.s_free[buf], ((fs >> 1) & 1u) ^ 1u, c.abort)) return false;
    if (!warp_wait(&c.ctl.k_full[k.st], k.phase, c.abort)) return false;
    tc_fence_after();
    const uint64_t kd = tile_desc_k + (uint64_t)(c.lay.k(k.st) >> 4);
#pragma unroll
    for (int part = 0; part < 2; ++part)
      mma_s_warp(c.tmem + kTmemS + buf * kTmemBuf, kd, q_desc + (uint64_t)(part * c.lay.q_part() >> 4),
                 (uint32_t)(N * 128) >> 4, idesc_e4m3(N, false, 0), c.tmem + kTmemSfV, c.tmem + kTmemSfQ, part);
    umma_commit_warp(&c.ctl.k_empty[k.st]);
    umma_commit_warp(&c.ctl.s_full[buf]);
    ++fs;
    k.next();
    return true;
  }

  // keys: the tile's; first: of the segment
  __device__ __forceinline__ bool o(int keys, bool first) {
    const uint32_t buf = fo & 1u;
    if (!warp_wait(&c.ctl.v_full[v.st], v.phase, c.abort)) return false;
    const int steps = (keys + kQ8Block - 1) / kQ8Block;
    if (keys < steps * kQ8Block) {   // whatever lies past the last key counts as 0: it may be NaN codes
      uint8_t* tile = c.smem + c.lay.v(v.st);
      const uint32_t zero[4] = {0u, 0u, 0u, 0u};
      for (int i = keys * 8 + (int)(threadIdx.x & 31); i < steps * kQ8Block * 8; i += 32)
#pragma unroll
        for (int h = 0; h < 2; ++h) sts_v4(smem_u32(tile + h * kHalfBytes + i * 16), zero);
      fence_async_smem();
      __syncwarp();
    }
    if (!warp_wait(&c.ctl.p_full[buf], (fo >> 1) & 1u, c.abort)) return false;
    tc_fence_after();
    const uint32_t sf = c.tmem + kTmemSfW + 4 * buf;
    copy_scales_warp(sf, sdesc_plain(smem_u32(c.smem + c.lay.sf((int)buf)), 16, 128));
    const uint64_t vd = tile_desc_v + (uint64_t)(c.lay.v(v.st) >> 4);
    const uint64_t pd = sdesc_plain(smem_u32(c.smem + c.lay.p((int)buf)), 128, kGroupBytes);
#pragma unroll
    for (int part = 0; part < 2; ++part)
      mma_o_warp(c.tmem + kTmemO, c.tmem + kTmemO + kTmemBuf, vd, pd + (uint64_t)(part * c.lay.p_part() >> 4),
                 idesc_e4m3(N, true, 0), c.tmem + kTmemSfV + 4 * part, sf, !first || part > 0, (uint32_t)steps);
    umma_commit_warp(&c.ctl.v_empty[v.st]);
    umma_commit_warp(&c.ctl.p_done[buf]);
    ++fo;
    v.next();
    return true;
  }
};

__device__ void issue_mma(const Cta& c) {
  const Verify4Args& a = c.a.v;
  Issue is(c);
  Walk<kTileN, true> walk(c.ctl.cut);
  Seg seg;
  uint32_t done = 0;
  while (walk.next(c.ctl.cut, a.n_seq, seg)) {
    const int end = cut_len<kTileN>(c.ctl.cut, seg.b, a.rows) + a.rows;
    if (!warp_wait(&c.ctl.q_full, done & 1u, c.abort)) return;
    tc_fence_after();
    copy_scales_warp(c.tmem + kTmemSfQ, sdesc_plain(smem_u32(c.smem + c.lay.sf_q()), 16, 128));
    if (!is.s()) return;
    for (int j = 0; j < seg.n; ++j) {
      if (j + 1 < seg.n && !is.s()) return;
      if (j == 0 && done > 0 && !warp_wait(&c.ctl.o_free, (done - 1) & 1u, c.abort)) return;
      if (!is.o(min(kTileN, end - (seg.kt0 + j) * kTileN), j == 0)) return;
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
// Four weights as two e4m3 parts: hi, to nearest, and lo = 32 (p - hi), which is exact before it is
// rounded.
__device__ __forceinline__ void split_weights(uint32_t& hi, uint32_t& lo, float p0, float p1, float p2, float p3) {
  asm("{\n\t.reg .b16 a, b, x, y, m;\n\t.reg .b32 h, g;\n\t.reg .f32 r0, r1, r2, r3;\n\t"
      "cvt.rn.satfinite.e4m3x2.f32 a, %3, %2;\n\tcvt.rn.satfinite.e4m3x2.f32 b, %5, %4;\n\t"
      "mov.b32 %0, {a, b};\n\t"
      "cvt.rn.f16x2.e4m3x2 h, a;\n\tcvt.rn.f16x2.e4m3x2 g, b;\n\t"
      "mul.f32 r0, %2, 0f42000000;\n\tmul.f32 r1, %3, 0f42000000;\n\t"   // 32
      "mul.f32 r2, %4, 0f42000000;\n\tmul.f32 r3, %5, 0f42000000;\n\t"
      "mov.b16 m, 0xD000;\n\t"                                              // -32 as a half
      "mov.b32 {x, y}, h;\n\tfma.rn.f32.f16 r0, x, m, r0;\n\tfma.rn.f32.f16 r1, y, m, r1;\n\t"
      "mov.b32 {x, y}, g;\n\tfma.rn.f32.f16 r2, x, m, r2;\n\tfma.rn.f32.f16 r3, y, m, r3;\n\t"
      "cvt.rn.satfinite.e4m3x2.f32 a, r1, r0;\n\tcvt.rn.satfinite.e4m3x2.f32 b, r3, r2;\n\t"
      "mov.b32 %1, {a, b};\n\t}"
      : "=&r"(hi), "=r"(lo)
      : "f"(p0), "f"(p1), "f"(p2), "f"(p3));
}
__device__ __forceinline__ float lds_f32(uint32_t addr) { return __uint_as_float(lds_u32(addr)); }
__device__ __forceinline__ void sts_f32(uint32_t addr, float v) {
  asm volatile("st.shared.f32 [%0], %1;" ::"r"(addr), "f"(v) : "memory");
}
__device__ __forceinline__ float4 lds_f32x4(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}

// The exponent that a query row is divided by: its largest magnitude is at most 448 of it.
__device__ __forceinline__ int query_exp(uint32_t top) {
  const int e = (int)(top >> 7) - 127 - 8 + ((top & 127u) > 96u ? 1 : 0);
  return min(max(e, -100), 100);
}

// Team `team` takes the groups team, team + teams, .. (kGroups of them at most).
template <int kGroups>
__device__ void softmax_worker(const Cta& c) {
  const Verify4Args& a = c.a.v;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int quarter = warp & 3, team = (warp - 4) >> 2, teams = c.lay.teams;
  const int mine = kGroups == 1 || team + teams < c.lay.groups ? kGroups : 1;   // groups of this team
  const uint32_t lanes = (uint32_t)(quarter * 32) << 16;
  const int blocks = c.blocks(), heads = kGroup / blocks, cols = heads * a.rows;
  const int head_off = blocks == 2 ? heads * (int)(blockIdx.x & 1) : 0;
  const int key = quarter * kQ8Block + lane;   // this thread's of a tile
  uint32_t f = 0, done = 0;
  auto col_of = [&](int u) { return (team + u * teams) * kCols; };   // group u's first column
  // the four warps of the team meet
  auto meet = [&]() { asm volatile("bar.sync %0, 128;" ::"r"(1 + team) : "memory"); };
  auto meet_any = [&](bool x) {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\tbarrier.cta.red.or.pred q, %2, 128, p;\n\t"
        "selp.u32 %0, 1, 0, q;\n\t}\n"
        : "=r"(r)
        : "r"((uint32_t)x), "r"(1 + team)
        : "memory");
    return r != 0u;
  };
  // a segment's queries: four columns of a group a warp, 8 dims a lane. Their place is free: this warp
  // has seen the last S of the segment before, so its products are done
  auto load_queries = [&](const Seg& seg) {
    const int N = c.lay.groups * kCols, head0 = seg.head * kGroup + head_off;
#pragma unroll
    for (int u = 0; u < kGroups; ++u) {
      if (u >= mine) break;
      uint4 x[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int col = col_of(u) + 4 * quarter + i, rr = col / heads;
        x[i] = make_uint4(0u, 0u, 0u, 0u);
        if (col < cols)
          x[i] = ld_input(reinterpret_cast<const uint4*>(
                              a.q_prep + (((size_t)seg.b * a.rows + rr) * kHeads + head0 + col - rr * heads) * kDim) +
                          lane);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int col = col_of(u) + 4 * quarter + i;
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
        uint8_t* at = c.smem + c.lay.q() + (lane >> 4) * N * 128 +
                      sw128_offset((uint32_t)col, (uint32_t)(lane & 15) >> 1) + (lane & 1) * 8;
        *reinterpret_cast<uint2*>(at) = make_uint2(hi[0] | hi[1] << 16, hi[2] | hi[3] << 16);
        *reinterpret_cast<uint2*>(at + c.lay.q_part()) = make_uint2(lo[0] | lo[1] << 16, lo[2] | lo[3] << 16);
        if (lane < 4) c.smem[c.lay.sf_q() + (col & 31) * 16 + (col >> 5) * 4 + lane] = (uint8_t)(e + kSfBias);
      }
    }
    fence_async_smem();
    __syncwarp();
    if (lane == 0) mbar_arrive(&c.ctl.q_full);
  };
  // places of buffer 0 of S, of this warp's part of the weights (a place for exchanges until they are
  // written), of its columns' scales, for the first group; what the second and buffer 1 are on
  const uint32_t s_at = c.tmem + kTmemS + lanes + col_of(0);
  const uint32_t slab0 = smem_u32(c.smem + c.lay.p(0)) + team * kGroupBytes + quarter * (kQ8Block * kCols);
  const uint32_t slab_group = teams * kGroupBytes, slab_buf = c.lay.p(1) - c.lay.p(0), part_step = c.lay.p_part();
  const uint32_t sf0 = smem_u32(c.smem + c.lay.sf(0)) + quarter;
  const uint32_t scales0 = smem_u32(c.ctl.scales[0][quarter]), scales_full = smem_u32(c.ctl.scales_full);
  const uint32_t s_full = smem_u32(c.ctl.s_full), s_free = smem_u32(c.ctl.s_free), p_full = smem_u32(c.ctl.p_full);
  Walk<kTileN, true> walk(c.ctl.cut);
  Seg seg, next;
  bool more = walk.next(c.ctl.cut, a.n_seq, seg);
  if (more) load_queries(seg);
  for (; more; seg = next) {
    const int L = cut_len<kTileN>(c.ctl.cut, seg.b, a.rows);
    float l[kGroups][kCols], R[kGroups];   // this key's sums; R of column lane % 16
#pragma unroll
    for (int u = 0; u < kGroups; ++u) {
      R[u] = -INFINITY;
#pragma unroll
      for (int i = 0; i < kCols; ++i) l[u][i] = 0.f;
    }
    for (int j = 0; j < seg.n; ++j, ++f) {
      const uint32_t buf = f & 1u, slab = slab0 + (buf ? slab_buf : 0u);
      const int kt = seg.kt0 + j;
      warp_wait(scales_full + 8 * (f % kScaleTiles), (f / kScaleTiles) & 1u, c.abort);
      const uint32_t scales = lds_u16(scales0 + (f % kScaleTiles) * (uint32_t)sizeof(c.ctl.scales[0]));
      const float factor = pow2i(q8_exp(scales)) * kLog2eOver16;   // from S to exponents
      const int v_exp = q8_exp(scales >> 8);
      warp_wait(s_full + 8 * buf, (f >> 1) & 1u, c.abort);
      tc_fence_after();
      uint32_t s[kGroups][kCols];
#pragma unroll
      for (int u = 0; u < kGroups; ++u)
        if (u < mine) tmem_ld16(s_at + buf * kTmemBuf + u * teams * kCols, s[u]);
#pragma unroll
      for (int u = 0; u < kGroups; ++u) tmem_wait_ld(s[u]);
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(s_free + 8 * buf);
      if (kt * kTileN + kTileN - 1 > L) {   // some key of the tile is hidden from some row
        const int last = kt * kTileN + key - L;   // this key is seen by rows from `last` on
#pragma unroll
        for (int u = 0; u < kGroups; ++u) {
          int rr = col_of(u) / heads, left = heads - (col_of(u) - rr * heads);
#pragma unroll
          for (int i = 0; i < kCols; ++i) {
            if (rr < last) s[u][i] = 0xFF800000u;   // -inf: weight 0, never the maximum
            if (--left == 0) {
              left = heads;
              ++rr;
            }
          }
        }
      }
      // the block's exponents, a column a lane: E, what its weights are scaled by
      float E[kGroups];
      bool over = false;
#pragma unroll
      for (int u = 0; u < kGroups; ++u) {
        if (u >= mine) break;
#pragma unroll
        for (int i = 0; i < kCols; i += 4) {
          uint32_t m[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) m[k] = __float_as_uint(warp_max(__uint_as_float(s[u][i + k])));
          if (lane == 0) sts_v4(slab + u * slab_group + 4 * i, m);
        }
      }
      __syncwarp();
#pragma unroll
      for (int u = 0; u < kGroups; ++u) {
        if (u >= mine) break;
        E[u] = fmaxf(ceilf(lds_f32(slab + u * slab_group + 4 * (lane & 15)) * factor), kNone);
        over |= E[u] > R[u] + kMove;
      }
      if (meet_any(over)) {
        // R moves, for all of the team (a segment's first tile: from nothing)
        if (lane < kCols) {
#pragma unroll
          for (int u = 0; u < kGroups; ++u)
            if (u < mine) sts_f32(slab + u * slab_group + 4 * lane, E[u]);
        }
        meet();
        // O holds every product before it is scaled
        if (j > 0) warp_wait(&c.ctl.p_done[buf ^ 1u], ((f - 1) >> 1) & 1u, c.abort);
        tc_fence_after();
#pragma unroll
        for (int u = 0; u < kGroups; ++u) {
          if (u >= mine) break;
          float to = R[u];
#pragma unroll
          for (int q = 0; q < 4; ++q)
            to = fmaxf(to, lds_f32(slab + u * slab_group + (q - quarter) * (kQ8Block * kCols) + 4 * (lane & 15)));
          const float move = to == R[u] ? 1.0f : ex2_approx(R[u] - to);
          R[u] = to;
          if (j > 0) {
#pragma unroll 1
            for (int h = 0; h < 2; ++h) {
              const uint32_t at = c.tmem + kTmemO + h * kTmemBuf + lanes + col_of(u);
              uint32_t o[kCols];
              tmem_ld16(at, o);
              tmem_wait_ld(o);
#pragma unroll
              for (int i = 0; i < kCols; ++i)
                o[i] = __float_as_uint(__uint_as_float(o[i]) * __shfl_sync(0xffffffffu, move, i));
              tmem_st16(at, o);
            }
          }
#pragma unroll
          for (int i = 0; i < kCols; ++i) l[u][i] *= __shfl_sync(0xffffffffu, move, i);
        }
        tmem_wait_st();
        tc_fence_before();
        meet();   // every warp has read the exchange
      }
#pragma unroll
      for (int u = 0; u < kGroups; ++u) {
        if (u >= mine) break;
        const float x = E[u] - kTop - R[u];
        if (lane < kCols) {
          const int col = col_of(u) + lane;
          asm volatile("st.shared.u8 [%0], %1;" ::"r"(sf0 + 512 * buf + (col & 31) * 16 + (col >> 5) * 4),
                       "r"(max(0, (int)x + v_exp + kSfBias))
                       : "memory");
          sts_f32(slab + u * slab_group + 4 * lane, kTop - E[u]);
          sts_f32(slab + u * slab_group + 4 * kCols + 4 * lane, ex2_approx(x));
        }
      }
      __syncwarp();
#pragma unroll
      for (int u = 0; u < kGroups; ++u) {
        if (u >= mine) break;
        const uint32_t at = slab + u * slab_group;
        uint32_t hi[kCols / 4], lo[kCols / 4];
#pragma unroll
        for (int i = 0; i < kCols; i += 4) {
          const float4 d = lds_f32x4(at + 4 * i), g = lds_f32x4(at + 4 * kCols + 4 * i);
          const float p0 = ex2_approx(fmaf(__uint_as_float(s[u][i]), factor, d.x));
          const float p1 = ex2_approx(fmaf(__uint_as_float(s[u][i + 1]), factor, d.y));
          const float p2 = ex2_approx(fmaf(__uint_as_float(s[u][i + 2]), factor, d.z));
          const float p3 = ex2_approx(fmaf(__uint_as_float(s[u][i + 3]), factor, d.w));
          l[u][i] = fmaf(p0, g.x, l[u][i]);
          l[u][i + 1] = fmaf(p1, g.y, l[u][i + 1]);
          l[u][i + 2] = fmaf(p2, g.z, l[u][i + 2]);
          l[u][i + 3] = fmaf(p3, g.w, l[u][i + 3]);
          split_weights(hi[i / 4], lo[i / 4], p0, p1, p2, p3);
        }
        __syncwarp();   // the slab is read
        sts_v4(at + lane * kCols, hi);
        sts_v4(at + lane * kCols + part_step, lo);
      }
      fence_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(p_full + 8 * buf);
    }
    more = walk.next(c.ctl.cut, a.n_seq, next);
    if (more) load_queries(next);
    // the segment's result: sums over the keys, column i's in lane i
    float sum[kGroups];
#pragma unroll
    for (int u = 0; u < kGroups; ++u) {
      sum[u] = 0.f;
#pragma unroll
      for (int i = 0; i < kCols; ++i) {
        float x = l[u][i];
#pragma unroll
        for (int off = 16; off; off >>= 1) x += __shfl_xor_sync(0xffffffffu, x, off);
        if (lane == i) sum[u] = x;
      }
    }
    warp_wait(&c.ctl.o_done, done & 1u, c.abort);
    tc_fence_after();
    if (lane < kCols) {
#pragma unroll
      for (int u = 0; u < kGroups; ++u)
        if (u < mine) sts_f32(slab0 + u * slab_group + 4 * lane, sum[u]);
    }
    meet();
    if (lane < kCols) {
#pragma unroll
      for (int u = 0; u < kGroups; ++u) {
        if (u >= mine) break;
        const uint32_t at = slab0 + u * slab_group - quarter * (kQ8Block * kCols) + 4 * lane;
        sum[u] = (lds_f32(at) + lds_f32(at + kQ8Block * kCols)) +
                 (lds_f32(at + 2 * kQ8Block * kCols) + lds_f32(at + 3 * kQ8Block * kCols));
        const int col = col_of(u) + lane;
        if (!seg.whole && quarter == 0 && col < cols)   // a NaN row's part weighs NaN, not nothing
          reinterpret_cast<float2*>(a.part_ml)[(size_t)seg.slot * kV4Lanes + col] =
              make_float2(sum[u] != sum[u] ? sum[u] : sum[u] == 0.f ? -INFINITY : R[u], sum[u]);
      }
    }
    meet();   // every warp has read the sums: the next segment writes there
    const int head0 = seg.head * kGroup + head_off;
#pragma unroll
    for (int u = 0; u < kGroups; ++u) {
      if (u >= mine) break;
      const float inv = 1.0f / sum[u];
      // O, 8 columns of half of the dims at a time, a dim a lane
#pragma unroll 1
      for (int at = 0; at < 4; ++at) {
        constexpr int kAtOnce = kCols / 2;
        const int d = 128 * (at >> 1) + 32 * quarter + lane, i0 = kAtOnce * (at & 1), first = col_of(u) + i0;
        uint32_t o[kAtOnce];
        tmem_ld8(c.tmem + kTmemO + (at >> 1) * kTmemBuf + lanes + first, o);
        tmem_wait_ld(o);
        // columns by (row, head) as they come
        int rr = first / heads, hh = first - rr * heads;
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
              a.part_o[((size_t)seg.slot * kV4Lanes + first + i) * kDim + d] = x;
          }
          if (++hh == heads) {
            hh = 0;
            ++rr;
          }
        }
      }
    }
    tc_fence_before();
    __syncwarp();
    if (lane == 0) mbar_arrive(&c.ctl.o_free);
    ++done;
  }
}

template <int kGroups>
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
    const uint32_t warps = 4u * lay.teams;
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
      mbar_init(&ctl.p_done[i], 1);
    }
    for (int i = 0; i < kScaleTiles; ++i) mbar_init(&ctl.scales_full[i], 2);
    mbar_init(&ctl.q_full, warps);
    mbar_init(&ctl.o_done, 1);
    mbar_init(&ctl.o_free, warps);
    mbar_init(&ctl.drain, 1);
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
    make_cut<kTileN, true>(a.v, ctl.cut, (int)gridDim.x / blocks, (int)blockIdx.x / blocks);
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
      issue_mma(c);
      umma_commit_warp(&ctl.drain);
      mbar_wait_quiet(&ctl.drain, 0, 100000000LL);
    } else if (warp == 2 || warp == 3) {
      load_tiles(c, warp == 2 ? &tm_k : &tm_v, warp == 3);
    } else if (warp >= 4) {
      softmax_worker<kGroups>(c);
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

int verify8_box_keys(int page_size) {
  return page_size % kTileN == 0 ? kTileN : page_size % (kTileN / 2) == 0 ? kTileN / 2 : kQ8Block;
}

cudaError_t verify8_set_attributes() {
  const cudaError_t e = cudaFuncSetAttribute(verify8_kernel<1>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemLimit);
  return e != cudaSuccess ? e
                          : cudaFuncSetAttribute(verify8_kernel<kTeamGroups>,
                                                 cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemLimit);
}

cudaError_t launch_verify8(const CUtensorMap& k_codes, const CUtensorMap& v_codes, const Verify8Args& a,
                           int sm_count, cudaStream_t s) {
  const int ctas = sm_count < kV4MaxCtas ? sm_count : kV4MaxCtas;
  const int blocks = row_blocks(a.v.rows), workers = ctas / blocks;
  const int cols = a.v.rows * (kGroup / blocks);
  Layout lay;
  lay.groups = (cols + kCols - 1) / kCols;
  const int per_team = lay.groups > kMaxTeams ? kTeamGroups : 1;
  lay.teams = (lay.groups + per_team - 1) / per_team;
  lay.stages = layout_bytes(lay.groups, kMaxStages) <= kSmemLimit ? kMaxStages : 2;
  lay.box_keys = verify8_box_keys(a.v.page_size);
  cudaLaunchAttribute attr[1];
  const cudaLaunchConfig_t cfg = overlapped_launch((unsigned)(workers * blocks), (unsigned)(128 + 128 * lay.teams),
                                                   (size_t)lay.bytes(), s, attr);
  const cudaError_t e = cudaLaunchKernelEx(&cfg, per_team == 1 ? verify8_kernel<1> : verify8_kernel<kTeamGroups>,
                                           k_codes, v_codes, a, lay);
  return e != cudaSuccess ? e : launch_verify4_combine(a.v, workers, kTileN, true, s);
}

}  // namespace ga

// What the two forms of the attention over 8-bit paged caches share (ga_verify8.cu, ga_verify8_rows.cu).
#pragma once
#include "ga_q8.cuh"
#include "ga_v4.cuh"

namespace ga {

constexpr int kTileBytes = kTileN * kQ8RowBytes;       // 32 KiB: two blocks of [128 keys][128 dims]
constexpr int kHalfBytes = kTileBytes / 2;
constexpr int kBoxBytes = kQ8Block * 128;              // 32 keys x 128 dims
constexpr int kSmemLimit = 232448;
constexpr float kLog2eOver16 = 1.4426950408889634f / 16.0f;
constexpr float kTop = 8.0f;          // a block's largest weight becomes at most 2^8 (large_exponent)
constexpr float kMove = 64.0f;        // R moves when a block passes it by more than 2^64
constexpr float kNone = -1e30f;       // the exponent of a block without a visible key
constexpr int kSfBias = 127;          // of a scale factor's 8 exponent bits

// ------------------------------------------------------------------ tensor cores
// Instruction descriptor of the block-scaled MMA, e4m3 operands, M = 128. Bits: [4, 6) which byte of
// B's scale words; 15, 16 A, B with rows (M, N) contiguous instead of K; [17, 23) N >> 3; 23 scales of 8
// exponent bits; [24, 29) M >> 4; [29, 31) which byte of A's scale words.
__host__ __device__ constexpr uint32_t idesc_e4m3(int N, bool a_rows, bool b_rows) {
  return (a_rows ? 1u << 15 : 0u) | (b_rows ? 1u << 16 : 0u) | ((uint32_t)(N >> 3) << 17) | (1u << 23) |
         ((128u >> 4) << 24);
}
// Unswizzled operand, rows contiguous: 16 rows x 8 of K are 128 consecutive bytes; the next 8 of K
// are `lbo` bytes on, the next 16 rows `sbo`. Also the source of a copy of scale factors.
__device__ __forceinline__ uint64_t sdesc_plain(uint32_t saddr, uint32_t lbo, uint32_t sbo) {
  return (uint64_t)((saddr & 0x3FFFFu) >> 4) | ((uint64_t)((lbo >> 4) & 0x3FFFu) << 16) |
         ((uint64_t)((sbo >> 4) & 0x3FFFu) << 32) | ((uint64_t)1 << 46);
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

// The OR over the 128 threads that meet at a named barrier.
__device__ __forceinline__ bool team_any(int barrier, bool x) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\tbarrier.cta.red.or.pred q, %2, 128, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}\n"
      : "=r"(r)
      : "r"((uint32_t)x), "r"(barrier)
      : "memory");
  return r != 0u;
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

// The scales of the tiles that are loaded, from the loaders (K's and V's) to the softmax. No loader can
// pass a tile that the softmax has yet to reach: with at most 3 stages it is 6 tiles ahead.
struct TileScales {
  static constexpr uint32_t kTiles = 8;
  uint64_t full[kTiles];
  uint8_t bytes[kTiles][4][2];   // a tile's blocks': of K, of V
  __device__ __forceinline__ void init() {
    for (uint32_t i = 0; i < kTiles; ++i) mbar_init(&full[i], 2);
  }
  // By a loader's warp: lane b < 4 has block b's.
  __device__ __forceinline__ void put(uint32_t tile, int block, int is_v, uint32_t scale) {
    if ((threadIdx.x & 31) < 4) bytes[tile % kTiles][block][is_v] = (uint8_t)scale;
    __syncwarp();
    if ((threadIdx.x & 31) == 0) mbar_arrive(&full[tile % kTiles]);
  }
  // Tile `tile`'s of a block: K's byte, V's above it.
  __device__ __forceinline__ uint32_t wait(uint32_t tile, int block, volatile int* abort) {
    warp_wait(&full[tile % kTiles], (tile / kTiles) & 1u, abort);
    return lds_u16(smem_u32(bytes[tile % kTiles][block]));
  }
};

// ------------------------------------------------------------------ loading
// A box of the tile's dims 128 half .. + 127 (all of them where the box covers the tile), by one lane of
// a converged warp.
__device__ __forceinline__ void load_box_warp(uint32_t dst, const CUtensorMap* map, uint64_t* bar, int row,
                                              int half) {
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
template <int kForm>
__device__ __forceinline__ void load_tiles(const Verify8Args& args, V4Cut& cut, const CUtensorMap* map,
                                           const uint8_t* scale_pool, int is_v, uint8_t* tiles, int stages,
                                           int box_keys, uint64_t* full, uint64_t* empty, TileScales& scales,
                                           volatile int* abort) {
  const Verify4Args& a = args.v;
  const int lane = threadIdx.x & 31, block = lane & 3;
  const int n_rows = a.n_pages * kKvHeads * a.page_size;   // below 2^31
  Ring ring(stages);
  uint32_t issued = 0;
  Walk<kTileN, kForm> walk(cut);
  Seg seg;
  while (walk.next(cut, a.n_seq, seg)) {
    const int end = cut_len<kTileN>(cut, seg.b, a.rows) + a.rows;
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
      if (!warp_wait(&empty[st], ring.phase ^ 1u, abort)) break;
      const int boxes = left >= kTileN ? kTileN / box_keys : (left + box_keys - 1) / box_keys;
      mbar_expect_tx_warp(&full[st], (uint32_t)(boxes * box_keys * kQ8RowBytes));
      __syncwarp();
      const uint32_t dst = smem_u32(tiles + st * kTileBytes);
      if (box_keys == kTileN) {
        load_box_warp(dst, map, &full[st], __shfl_sync(0xffffffffu, row, 0), 0);
      } else {
        for (int b = 0; b < boxes; ++b) {
          const int r = __shfl_sync(0xffffffffu, row, b * box_keys / kQ8Block);
          load_box_warp(dst + b * box_keys * 128, map, &full[st], r, 0);
          load_box_warp(dst + kHalfBytes + b * box_keys * 128, map, &full[st], r, 1);
        }
      }
      scales.put(issued, block, is_v, now.scale);
      now = next;
      next = after;
    }
    if (*abort) break;
  }
  if (*abort) {   // the copies in flight land before the CTA leaves
    const uint32_t n = stages;
    for (uint32_t i = issued > n ? issued - n : 0; i < issued; ++i)
      mbar_wait_quiet(&full[i % n], (i / n) & 1u, 100000000LL);
  }
}

// Rows of a value tile past the tile's last key count as 0 (they may be NaN codes), as far as the MMAs
// read: `steps` blocks of 32. By a warp, before its MMAs.
__device__ __forceinline__ void hide_values(uint8_t* tile, int keys, int steps) {
  if (keys >= steps * kQ8Block) return;
  const uint32_t zero[4] = {0u, 0u, 0u, 0u};
  for (int i = keys * 8 + (int)(threadIdx.x & 31); i < steps * kQ8Block * 8; i += 32)
#pragma unroll
    for (int h = 0; h < 2; ++h) sts_v4(smem_u32(tile + h * kHalfBytes + i * 16), zero);
  fence_async_smem();
  __syncwarp();
}

// ------------------------------------------------------------------ numerics
// A block's weights are 2^(t - E + 8), t = s factor (the scores as exponents), E about the largest t; they are
// formed as 2^fma(s, factor, a), whose product is exact. Two parts hold a weight up to 2^8 and little more
// (from a remainder of 14 on, at 270, the second part saturates, and the sum would not see it). E is ceil of
// the rounded product, which up to 2^20 is less than t by 1/32 at most: 262. Past it E is moved up where it is
// less. It is a multiple of its own step, so below 2^27, where that is at most 8, a = 8 - E is exact, and the
// largest weight is between 1 (2^7 below 2^24) and 2^8. From kFar on neither holds, and scores that differ at
// all are half that step apart: E is t rounded down, and the caller sees to it that the largest score has the
// weight 2^8.
// first_exponent is what serves up to 2^20 (is_large: past it), large_exponent what serves at any magnitude.
constexpr float kLarge = 1048576.0f, kFar = 134217728.0f;   // 2^20, 2^27
__device__ __forceinline__ float first_exponent(float top, float factor) {
  return fmaxf(ceilf(top * factor), kNone);
}
__device__ __forceinline__ bool is_large(float E) { return fabsf(E) > kLarge && E > kNone; }
__device__ __forceinline__ float large_exponent(float E, float top, float factor) {
  if (fmaf(top, factor, -E) > 0.f)   // to the next integer, or the next value (E = 0: NaN, which is passed over)
    E = fmaxf(E + 1.f, __int_as_float(__float_as_int(E) + (E > 0.f ? 1 : -1)));
  return fabsf(E) >= kFar ? fmaxf(__fmul_rd(top, factor), kNone) : E;
}
__device__ __forceinline__ float min_or_nan(float a, float b) {
  float r;
  asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// Four weights as two e4m3 parts: hi, to nearest, and lo = 32 (p - hi), which is exact before it is
// rounded. 9 bits, so that the codes of V meet them in 8-bit MMAs, two for each product; one part alone would
// keep 4; bf16 weights, which V would have to be widened for, keep 8. The sums take p itself: rounded
// weights would cost a conversion each, and be nearer only where one key has nearly all the weight, by 2^-9
// of the output at most.
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
// The scale byte of a block's weights, 2^x of what O is relative to, for values of exponent v_exp: 0 (2^-127)
// from there down. (x is about kNone for a block that the row does not see: more than an int holds.)
__host__ __device__ __forceinline__ uint32_t scale_byte(float x, int v_exp) {
  const int e = (int)fmaxf(x, -512.f) + v_exp + kSfBias;
  return e > 0 ? (uint32_t)e : 0u;
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

}  // namespace ga

// Decode and verify attention over 8-bit paged caches (format: ga_q8.cuh): up to four rows, keys and dims
// on the rows of the MMAs (five and more: ga_verify8_rows.cu).
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
// call: 16 columns for one row of 12 heads, 48 for four.
//
// Scales are powers of two, and the MMAs (kind::mxf8f6f4, a scale per row or column and 32 of K) take
// them back: each query row is scaled to its largest magnitude; weights are scaled per column and
// block of 32 keys, to 256 at the block's largest, and their scale carries the value block's. A key
// block's goes into the factor from S to exponents, one number for a warp. So a weight's precision is
// relative to its own block's largest, not the row's: the others keep theirs beside a key that
// outweighs them by far but has a small value. R, the exponent that a column's O and sum are kept
// relative to, is the first tile's and moves only when a block passes it by 2^64.
//
// Work. A stream is (sequence, KV head), cut into tiles of 128 keys and the tiles among the CTAs as in
// the 4-bit form (ga_v4.cuh); parts of a stream are merged by its combine kernel.
//
// Structure (128 + 256 G threads, G groups of 16 columns):
//   warp 0      issues S^T = K Q^T (M = 128 keys, N = 16 G, K = 256 twice) of a tile, then O^T +=
//               V^T W^T (M = 128 dims twice, N = 16 G, K = 32 keys; twice) of the tile before
//   warps 2, 3  load K and V tiles by TMA, and their blocks' scales
//   4 .. 3 + 4 G  softmax: a team of four warps per group, warp q with the tile's keys 32 q .. + 31, a
//               block, a key a lane
//   the others  a team per group that splits the next segment's queries once this one's S are done, and
//               writes the result of the segment before (O and the sums have two places). These are two
//               and more dependent loads, each behind the tiles that are in flight (1.6 us); in the softmax
//               warps they kept a segment's end from its successor's tiles for 5 to 10 us
// Tensor memory: two buffers of O^T (dims 0..127, then 128..255, 48 columns each) [0, 192), of S^T [192,
// 288), scale factors 1 and 2^-5 (of K, and of V beside the weights' first and second part) [288, 296),
// those of W^T, two buffers [296, 304), of Q [304, 308).
// Every wait is bounded; a wait that gives up raises the CTA's abort flag, which the others see. A
// team's four warps meet at a named barrier in every tile; they run all their tiles even after an
// abort (their waits then return at once), so that none is left there.
#include <cstddef>

#include "ga_v8.cuh"

namespace ga {
namespace {

constexpr int kCols = 16;                              // columns of a group
constexpr int kMaxGroups = 3;
constexpr int kMaxCols = kCols * kMaxGroups;           // 48: four rows of 12 heads
constexpr int kStages = 3;                             // tiles in flight of K, and of V (2 with 2 or 3 groups)
constexpr int kGroupBytes = kTileN * kCols;            // a group's weights of a tile, one part
constexpr uint32_t kTmemBuf = kMaxCols;                // columns between S's buffers, and O's halves
constexpr uint32_t kTmemO = 0, kTmemOBuf = 2 * kTmemBuf, kTmemS = 2 * kTmemOBuf, kTmemSfV = kTmemS + 2 * kTmemBuf,
                   kTmemSfW = kTmemSfV + 8, kTmemSfQ = kTmemSfW + 8, kTmemCols = 512;
static_assert(kTmemSfQ + 4 <= kTmemCols, "tensor memory");

struct Ctl {
  V4Cut cut;
  TileScales scales;
  uint64_t k_full[kStages], k_empty[kStages], v_full[kStages], v_empty[kStages];
  uint64_t q_full, q_free, s_full[2], s_free[2], p_full[2], p_done[2], sums_full[2], o_done[2], o_free[2], drain;
  float sums[2][4][kMaxCols], refs[2][kMaxCols];   // a segment's: of a quarter of the keys; R
  uint32_t tmem_base;
  int abort;
};
// Shared memory: the tiles of K, then V, the queries (two parts of two halves of [16 G][128]), the
// weights (two buffers of two parts of G groups of [128 keys][16]), scale factors (two buffers of the
// weights', the queries'; 512 bytes each), Ctl.
template <int kGroups>
struct Layout {
  static constexpr int v_stages = kGroups == 1 ? kStages : kStages - 1;
  __host__ __device__ static constexpr int k(int st) { return st * kTileBytes; }
  __host__ __device__ static constexpr int v(int st) { return (kStages + st) * kTileBytes; }
  static constexpr int q = (kStages + v_stages) * kTileBytes, q_part = kGroups * kCols * kDim;
  static constexpr int p_part = kGroups * kGroupBytes;
  __host__ __device__ static constexpr int p(int buf) { return q + 2 * q_part + buf * 2 * p_part; }
  __host__ __device__ static constexpr int sf(int buf) { return p(2) + buf * 512; }
  static constexpr int sf_q = q + 2 * q_part + 4 * p_part + 2 * 512, ctl = sf_q + 512, bytes = ctl + (int)sizeof(Ctl);
  static_assert(bytes <= kSmemLimit, "227 KiB of shared memory per CTA");
};
static_assert(sizeof(Ctl) % 8 == 0 && offsetof(Ctl, scales) % 8 == 0 && offsetof(Ctl, k_full) % 8 == 0,
              "barriers at 8 bytes");

// ------------------------------------------------------------------ tensor cores
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
template <int kGroups>
struct Cta {
  using Lay = Layout<kGroups>;
  uint8_t* smem;
  Ctl& ctl;
  const Verify8Args& a;
  uint32_t tmem;
  volatile int* abort;
};

// ------------------------------------------------------------------ MMA issue
// In this order: S of tile 0, S of 1, O of 0, S of 2, O of 1, ... of a segment, so that tile f's S
// tells that O's products of tile f - 2 are done, and their weights' place is free.
template <int kGroups>
struct Issue {
  using Lay = Layout<kGroups>;
  static constexpr int N = kGroups * kCols;
  const Cta<kGroups>& c;
  const uint64_t q_desc, tile_desc_k, tile_desc_v;
  Ring k, v;
  uint32_t fs, fo;   // tiles whose S, O is issued
  __device__ __forceinline__ explicit Issue(const Cta<kGroups>& c_)
      : c(c_), q_desc(sdesc_sw128(smem_u32(c_.smem + Lay::q), 16, 1024)),
        tile_desc_k(sdesc_sw128(smem_u32(c_.smem), 16, 1024)),
        tile_desc_v(sdesc_sw128(smem_u32(c_.smem), kHalfBytes, 1024)), k(kStages), v(Lay::v_stages), fs(0),
        fo(0) {}

  __device__ __forceinline__ bool s() {
    const uint32_t buf = fs & 1u;
    if (!warp_wait(&c.ctl.s_free[buf], ((fs >> 1) & 1u) ^ 1u, c.abort)) return false;
    if (!warp_wait(&c.ctl.k_full[k.st], k.phase, c.abort)) return false;
    tc_fence_after();
    const uint64_t kd = tile_desc_k + (uint64_t)(Lay::k(k.st) >> 4);
#pragma unroll
    for (int part = 0; part < 2; ++part)
      mma_s_warp(c.tmem + kTmemS + buf * kTmemBuf, kd, q_desc + (uint64_t)(part * Lay::q_part >> 4),
                 (uint32_t)(N * 128) >> 4, idesc_e4m3(N, false, false), c.tmem + kTmemSfV, c.tmem + kTmemSfQ, part);
    umma_commit_warp(&c.ctl.k_empty[k.st]);
    umma_commit_warp(&c.ctl.s_full[buf]);
    ++fs;
    k.next();
    return true;
  }

  // keys: the tile's; first: of the segment, whose O is at o_at
  __device__ __forceinline__ bool o(uint32_t o_at, int keys, bool first) {
    const uint32_t buf = fo & 1u;
    if (!warp_wait(&c.ctl.v_full[v.st], v.phase, c.abort)) return false;
    const int steps = (keys + kQ8Block - 1) / kQ8Block;
    hide_values(c.smem + Lay::v(v.st), keys, steps);
    if (!warp_wait(&c.ctl.p_full[buf], (fo >> 1) & 1u, c.abort)) return false;
    tc_fence_after();
    const uint32_t sf = c.tmem + kTmemSfW + 4 * buf;
    copy_scales_warp(sf, sdesc_plain(smem_u32(c.smem + Lay::sf((int)buf)), 16, 128));
    const uint64_t vd = tile_desc_v + (uint64_t)(Lay::v(v.st) >> 4);
    const uint64_t pd = sdesc_plain(smem_u32(c.smem + Lay::p((int)buf)), 128, kGroupBytes);
#pragma unroll
    for (int part = 0; part < 2; ++part)
      mma_o_warp(o_at, o_at + kTmemBuf, vd, pd + (uint64_t)(part * Lay::p_part >> 4),
                 idesc_e4m3(N, true, true), c.tmem + kTmemSfV + 4 * part, sf, !first || part > 0, (uint32_t)steps);
    umma_commit_warp(&c.ctl.v_empty[v.st]);
    umma_commit_warp(&c.ctl.p_done[buf]);
    ++fo;
    v.next();
    return true;
  }
};

template <int kGroups>
__device__ void issue_mma(const Cta<kGroups>& c) {
  const Verify4Args& a = c.a.v;
  using Lay = Layout<kGroups>;
  Issue<kGroups> is(c);
  Walk<kTileN, kQ8Columns> walk(c.ctl.cut);
  Seg seg;
  uint32_t done = 0;
  while (walk.next(c.ctl.cut, a.n_seq, seg)) {
    const int end = cut_len<kTileN>(c.ctl.cut, seg.b, a.rows) + a.rows;
    if (!warp_wait(&c.ctl.q_full, done & 1u, c.abort)) return;
    tc_fence_after();
    copy_scales_warp(c.tmem + kTmemSfQ, sdesc_plain(smem_u32(c.smem + Lay::sf_q), 16, 128));
    const uint32_t buf = done & 1u, o_at = c.tmem + kTmemO + buf * kTmemOBuf;
    if (!is.s()) return;
    for (int j = 0; j < seg.n; ++j) {
      if (j + 1 < seg.n && !is.s()) return;
      if (j == max(seg.n - 2, 0)) umma_commit_warp(&c.ctl.q_free);   // after the last S
      if (j == 0 && !warp_wait(&c.ctl.o_free[buf], ((done >> 1) & 1u) ^ 1u, c.abort)) return;
      if (!is.o(o_at, min(kTileN, end - (seg.kt0 + j) * kTileN), j == 0)) return;
    }
    umma_commit_warp(&c.ctl.o_done[buf]);
    ++done;
  }
}

// ------------------------------------------------------------------ softmax
__device__ __forceinline__ float warp_max(float x) {
  float r;
  asm("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(x));
  return r;
}

// Team g takes group g.
template <int kGroups>
__device__ void softmax_worker(const Cta<kGroups>& c) {
  using Lay = Layout<kGroups>;
  const Verify4Args& a = c.a.v;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int quarter = warp & 3, team = (warp - 4) >> 2, col0 = team * kCols;
  const uint32_t lanes = (uint32_t)(quarter * 32) << 16;
  const int key = quarter * kQ8Block + lane;   // this thread's of a tile
  uint32_t f = 0, done = 0;
  // the four warps of the team meet
  auto meet = [&]() { asm volatile("bar.sync %0, 128;" ::"r"(1 + team) : "memory"); };
  auto factor_of = [](uint32_t scales) { return pow2i(q8_exp(scales)) * kLog2eOver16; };   // from S to exponents
  // places of buffer 0 of S, of this warp's part of the weights (a place for exchanges until they are
  // written), of its columns' scales, what buffer 1 is on
  const uint32_t s_at = c.tmem + kTmemS + lanes + col0;
  const uint32_t slab0 = smem_u32(c.smem + Lay::p(0)) + team * kGroupBytes + quarter * (kQ8Block * kCols);
  const uint32_t slab_buf = Lay::p(1) - Lay::p(0), part_step = Lay::p_part;
  const uint32_t sf0 = smem_u32(c.smem + Lay::sf(0)) + quarter;
  const uint32_t s_full = smem_u32(c.ctl.s_full), s_free = smem_u32(c.ctl.s_free), p_full = smem_u32(c.ctl.p_full);
  Walk<kTileN, kQ8Columns> walk(c.ctl.cut);
  Seg seg;
  for (; walk.next(c.ctl.cut, a.n_seq, seg); ++done) {
    const int L = cut_len<kTileN>(c.ctl.cut, seg.b, a.rows);
    float l[kCols], R = -INFINITY;   // this key's sums; R of column lane % 16
#pragma unroll
    for (int i = 0; i < kCols; ++i) l[i] = 0.f;
    for (int j = 0; j < seg.n; ++j, ++f) {
      const uint32_t buf = f & 1u, slab = slab0 + (buf ? slab_buf : 0u);
      const int kt = seg.kt0 + j;
      uint32_t scales = c.ctl.scales.wait(f, quarter, c.abort);
      const float factor = factor_of(scales);
      warp_wait(s_full + 8 * buf, (f >> 1) & 1u, c.abort);
      tc_fence_after();
      uint32_t s[kCols];
      tmem_ld16(s_at + buf * kTmemBuf, s);
      tmem_wait_ld(s);
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(s_free + 8 * buf);
      if (kt * kTileN + kTileN - 1 > L) {   // some key of the tile is hidden from some row
        const int last = kt * kTileN + key - L;   // this key is seen by rows from `last` on
        int rr = col0 / kGroup, left = kGroup - (col0 - rr * kGroup);
#pragma unroll
        for (int i = 0; i < kCols; ++i) {
          if (rr < last) s[i] = 0xFF800000u;   // -inf: weight 0, never the maximum
          if (--left == 0) {
            left = kGroup;
            ++rr;
          }
        }
      }
      // the block's exponents, a column a lane: E, what its weights are scaled by
#pragma unroll
      for (int i = 0; i < kCols; i += 4) {
        uint32_t m[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) m[k] = __float_as_uint(warp_max(__uint_as_float(s[i + k])));
        if (lane == 0) sts_v4(slab + 4 * i, m);
      }
      __syncwarp();
      const float top = lds_f32(slab + 4 * (lane & 15));
      // (without asking is_large: a branch takes longer, 256 x 2 rows of up to 1,000 keys 56.4 us for 55.7)
      const float E = large_exponent(first_exponent(top, factor), top, factor);
      if (team_any(1 + team, E - R > kMove)) {
        // R moves, for all of the team (a segment's first tile: from nothing)
        if (lane < kCols) sts_f32(slab + 4 * lane, E);
        meet();
        // O holds every product before it is scaled
        if (j > 0) warp_wait(&c.ctl.p_done[buf ^ 1u], ((f - 1) >> 1) & 1u, c.abort);
        tc_fence_after();
        float to = R;
#pragma unroll
        for (int q = 0; q < 4; ++q)
          to = fmaxf(to, lds_f32(slab + (q - quarter) * (kQ8Block * kCols) + 4 * (lane & 15)));
        const float move = to == R ? 1.0f : ex2_approx(R - to);
        R = to;
        if (j > 0) {
#pragma unroll 1
          for (int h = 0; h < 2; ++h) {
            const uint32_t at = c.tmem + kTmemO + (done & 1u) * kTmemOBuf + h * kTmemBuf + lanes + col0;
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
        for (int i = 0; i < kCols; ++i) l[i] *= __shfl_sync(0xffffffffu, move, i);
        tmem_wait_st();
        tc_fence_before();
        meet();   // every warp has read the exchange
      }
      asm volatile("" : "+r"(scales));   // formed anew: both kept from above, three groups' would be spilled
      const float factor2 = factor_of(scales);
      const int v_exp = q8_exp(scales >> 8);
      const float x = E - R - kTop;   // (E - R is exact where it matters, E - kTop is not for every E)
      if (lane < kCols) {
        const int col = col0 + lane;
        asm volatile("st.shared.u8 [%0], %1;" ::"r"(sf0 + 512 * buf + (col & 31) * 16 + (col >> 5) * 4),
                     "r"(scale_byte(x, v_exp))
                     : "memory");
        sts_f32(slab + 4 * lane, __fsub_ru(kTop, E));   // with E from kFar on, the largest is 2^8 or more: clamped
        sts_f32(slab + 4 * kCols + 4 * lane, ex2_approx(x));
      }
      __syncwarp();
      // (the clamp, and not other code for scores from kFar on: that was 16 columns' worth of instructions to
      // fetch in every segment, 256 x 1 row of up to 1,000 keys 52.9 us for 51.5, 49.8 with neither)
      uint32_t hi[kCols / 4], lo[kCols / 4];
#pragma unroll
      for (int i = 0; i < kCols; i += 4) {
        const float4 a = lds_f32x4(slab + 4 * i), g = lds_f32x4(slab + 4 * kCols + 4 * i);
        const float p0 = ex2_approx(min_or_nan(fmaf(__uint_as_float(s[i]), factor2, a.x), kTop));
        const float p1 = ex2_approx(min_or_nan(fmaf(__uint_as_float(s[i + 1]), factor2, a.y), kTop));
        const float p2 = ex2_approx(min_or_nan(fmaf(__uint_as_float(s[i + 2]), factor2, a.z), kTop));
        const float p3 = ex2_approx(min_or_nan(fmaf(__uint_as_float(s[i + 3]), factor2, a.w), kTop));
        l[i] = fmaf(p0, g.x, l[i]);
        l[i + 1] = fmaf(p1, g.y, l[i + 1]);
        l[i + 2] = fmaf(p2, g.z, l[i + 2]);
        l[i + 3] = fmaf(p3, g.w, l[i + 3]);
        split_weights(hi[i / 4], lo[i / 4], p0, p1, p2, p3);
      }
      __syncwarp();   // the slab is read
      sts_v4(slab + lane * kCols, hi);
      sts_v4(slab + lane * kCols + part_step, lo);
      fence_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(p_full + 8 * buf);
    }
    // the sums over the warp's keys: each step adds halves of the columns across lanes; column i's
    // in lanes i and 16 + i
#pragma unroll
    for (int w = kCols / 2; w; w >>= 1) {
      const bool upper = (lane & w) != 0;
#pragma unroll
      for (int i = 0; i < w; ++i) {
        const float send = upper ? l[i] : l[i + w];
        l[i] = (upper ? l[i + w] : l[i]) + __shfl_xor_sync(0xffffffffu, send, w);
      }
    }
    l[0] += __shfl_xor_sync(0xffffffffu, l[0], kCols);
    warp_wait(&c.ctl.o_free[done & 1u], ((done >> 1) & 1u) ^ 1u, c.abort);   // their place is read
    if (lane < kCols) {
      c.ctl.sums[done & 1u][quarter][col0 + lane] = l[0];
      if (quarter == 0) c.ctl.refs[done & 1u][col0 + lane] = R;
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(&c.ctl.sums_full[done & 1u]);
  }
}

// ------------------------------------------------------------------ queries and results
// Team g has group g, each warp a quarter of the dims of O^T, or of the group's queries.
template <int kGroups>
__device__ void segment_worker(const Cta<kGroups>& c) {
  using Lay = Layout<kGroups>;
  const Verify4Args& a = c.a.v;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, quarter = warp & 3;
  constexpr int N = kGroups * kCols;
  const int cols = kGroup * a.rows, col0 = ((warp - 4) / 4 - kGroups) * kCols;
  const uint32_t o_at = c.tmem + kTmemO + ((uint32_t)(quarter * 32) << 16) + col0;
  uint32_t done = 0;
  // The place of a column's (row, head) among the call's, below 256 x 4 x 24 (past the last: the last's)
  auto place = [&](int first, int col) {
    const int rr = min(col, cols - 1) / kGroup;
    return (uint32_t)(first + min(col, cols - 1) + rr * (kHeads - kGroup));
  };
  // a segment's first, and the group's first column, formed anew where they are used: the rows of 20 columns
  // kept across the loops would not fit in the registers
  auto first_of = [&](const Seg& seg) { return seg.b * a.rows * kHeads + seg.head * kGroup; };
  auto anew = [](int x) {
    asm volatile("" : "+r"(x));
    return x;
  };
  // a segment's queries: four columns a warp, 8 dims a lane
  uint4 x[4];
  auto fetch = [&](const Seg& seg) {
    const int first = first_of(seg), at = anew(col0 + 4 * quarter);
#pragma unroll
    for (int i = 0; i < 4; ++i)
      x[i] = ld_input(reinterpret_cast<const uint4*>(a.q_prep + place(first, at + i) * kDim) + lane);
  };
  auto put_queries = [&]() {
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
      uint8_t* at = c.smem + Lay::q + (lane >> 4) * N * 128 +
                    sw128_offset((uint32_t)col, (uint32_t)(lane & 15) >> 1) + (lane & 1) * 8;
      *reinterpret_cast<uint2*>(at) = make_uint2(hi[0] | hi[1] << 16, hi[2] | hi[3] << 16);
      *reinterpret_cast<uint2*>(at + Lay::q_part) = make_uint2(lo[0] | lo[1] << 16, lo[2] | lo[3] << 16);
      if (lane < 4) c.smem[Lay::sf_q + (col & 31) * 16 + (col >> 5) * 4 + lane] = (uint8_t)(e + kSfBias);
    }
    fence_async_smem();
    __syncwarp();
    if (lane == 0) mbar_arrive(&c.ctl.q_full);
  };
  Walk<kTileN, kQ8Columns> walk(c.ctl.cut);
  Seg seg, next;
  bool more = walk.next(c.ctl.cut, a.n_seq, seg);
  if (more) {
    fetch(seg);
    put_queries();
  }
  for (; more; seg = next, ++done) {
    const uint32_t buf = done & 1u;
    more = walk.next(c.ctl.cut, a.n_seq, next);
    if (more) {
      fetch(next);
      warp_wait(&c.ctl.q_free, done & 1u, c.abort);   // every S of this segment is done
      put_queries();
    }
    // Steps of 8 columns of half of the dims, a dim a lane; gates are loaded a step ahead of their use.
    // Columns past the last are formed too and not stored: a branch for each would keep them from
    // overlapping.
    constexpr int kAtOnce = kCols / 2;
    uint32_t gate[kAtOnce];
    const int first = first_of(seg);
    auto load_gates = [&](int at) {
      const int d = 64 * (at & 2) + 32 * quarter + lane, c0 = anew(col0 + kAtOnce * (at & 1));
#pragma unroll
      for (int i = 0; i < kAtOnce; ++i) gate[i] = ld_input(a.qg + (place(first, c0 + i) * kQgStride + kDim + d));
    };
    if (seg.whole) load_gates(0);
    warp_wait(&c.ctl.sums_full[buf], (done >> 1) & 1u, c.abort);
    float inv;   // of column lane % 16
    {
      const int col = col0 + (lane & (kCols - 1));
      const float(&s)[4][kMaxCols] = c.ctl.sums[buf];
      const float sum = (s[0][col] + s[1][col]) + (s[2][col] + s[3][col]);
      inv = 1.0f / sum;
      if (!seg.whole && quarter == 0 && lane < kCols && col < cols)   // a NaN row's part weighs NaN, not nothing
        reinterpret_cast<float2*>(a.part_ml)[(size_t)seg.slot * kV4Lanes + col] =
            make_float2(sum != sum ? sum : sum == 0.f ? -INFINITY : c.ctl.refs[buf][col], sum);
    }
    warp_wait(&c.ctl.o_done[buf], (done >> 1) & 1u, c.abort);
    tc_fence_after();
#pragma unroll 1
    for (int at = 0; at < 4; ++at) {
      const int i0 = kAtOnce * (at & 1), c0 = anew(col0 + i0), d = 64 * (at & 2) + 32 * quarter + lane;
      uint32_t o[kAtOnce];
      tmem_ld8(o_at + buf * kTmemOBuf + ((at & 2) ? kTmemBuf : 0u) + i0, o);
      tmem_wait_ld(o);
      if (seg.whole) {
        float g[kAtOnce];
#pragma unroll
        for (int i = 0; i < kAtOnce; ++i) g[i] = lo_f(gate[i]);
        if (at < 3) load_gates(at + 1);
        uint16_t y[kAtOnce];
#pragma unroll
        for (int i = 0; i < kAtOnce; ++i) {
          const float scale = __shfl_sync(0xffffffffu, inv, i0 + i);
          y[i] = (uint16_t)(pack_bf16x2(__uint_as_float(o[i]) * scale * sigmoid_f(g[i]), 0.f) & 0xFFFFu);
        }
#pragma unroll
        for (int i = 0; i < kAtOnce; ++i)
          if (c0 + i < cols) a.out[place(first, c0 + i) * kDim + d] = y[i];
      } else {
        float* p = a.part_o + ((size_t)seg.slot * kV4Lanes + c0) * kDim + d;
#pragma unroll
        for (int i = 0; i < kAtOnce; ++i)
          if (c0 + i < cols) p[i * kDim] = __uint_as_float(o[i]);
      }
    }
    tc_fence_before();
    __syncwarp();
    if (lane == 0) mbar_arrive(&c.ctl.o_free[buf]);
  }
}

template <int kGroups>
__global__ void __launch_bounds__(128 + 256 * kGroups, 1)
    verify8_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                   const __grid_constant__ Verify8Args a, int box_keys) {
  using Lay = Layout<kGroups>;
  extern __shared__ __align__(1024) uint8_t smem[];
  if ((smem_u32(smem) & 1023u) != 0u) {
    if (threadIdx.x == 0) record(a.v.status, kDevBadLaunch);
    return;
  }
  Ctl& ctl = *reinterpret_cast<Ctl*>(smem + Lay::ctl);
  const int warp = threadIdx.x >> 5;
  if (threadIdx.x == 0) {
    const uint32_t warps = 4u * kGroups;
    ctl.abort = 0;
    for (int i = 0; i < kStages; ++i) {
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
      mbar_init(&ctl.sums_full[i], warps);
      mbar_init(&ctl.o_done[i], 1);
      mbar_init(&ctl.o_free[i], warps);
    }
    ctl.scales.init();
    mbar_init(&ctl.q_full, warps);
    mbar_init(&ctl.q_free, 1);
    mbar_init(&ctl.drain, 1);
    mbar_fence_init();
  }
  if (warp == 2 && (threadIdx.x & 31) == 0) {
    tma_prefetch_desc(&tm_k);
    tma_prefetch_desc(&tm_v);
  }
  // scales of columns past the groups are read by the copies and used by nothing
  for (int i = threadIdx.x; i < 3 * 512 / 4; i += blockDim.x) reinterpret_cast<uint32_t*>(smem + Lay::sf(0))[i] = 0u;
  grid_wait();
  grid_launch_dependents();
  if (warp == 1) {   // after the wait: the kernel before may still need tensor memory until it ends
    tmem_alloc(&ctl.tmem_base, kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  make_cut<kTileN, kQ8Columns>(a.v, ctl.cut, (int)gridDim.x, (int)blockIdx.x);   // two block barriers
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
  const Cta<kGroups> c = {smem, ctl, a, tmem, &ctl.abort};
  if (ctl.cut.run_tiles() > 0) {
    if (warp == 0) {
      issue_mma<kGroups>(c);
      umma_commit_warp(&ctl.drain);
      mbar_wait_quiet(&ctl.drain, 0, 100000000LL);
    } else if (warp == 2 || warp == 3) {
      const bool v = warp == 3;
      load_tiles<kQ8Columns>(a, ctl.cut, v ? &tm_v : &tm_k, v ? a.v_scales : a.k_scales, v,
                             smem + (v ? Lay::v(0) : Lay::k(0)), v ? Lay::v_stages : kStages, box_keys,
                             v ? ctl.v_full : ctl.k_full, v ? ctl.v_empty : ctl.k_empty, ctl.scales, &ctl.abort);
    } else if (warp >= 4 + 4 * kGroups) {
      segment_worker<kGroups>(c);
    } else if (warp >= 4) {
      softmax_worker<kGroups>(c);
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
  if (threadIdx.x == 0 && ctl.abort) record(a.v.status, ctl.abort);
}

}  // namespace

int verify8_box_keys(int page_size) {
  return page_size % kTileN == 0 ? kTileN : page_size % (kTileN / 2) == 0 ? kTileN / 2 : kQ8Block;
}

cudaError_t verify8_set_attributes() {
  constexpr auto kAttr = cudaFuncAttributeMaxDynamicSharedMemorySize;
  cudaError_t e = cudaFuncSetAttribute(verify8_kernel<1>, kAttr, Layout<1>::bytes);
  if (e == cudaSuccess) e = cudaFuncSetAttribute(verify8_kernel<2>, kAttr, Layout<2>::bytes);
  if (e == cudaSuccess) e = cudaFuncSetAttribute(verify8_kernel<3>, kAttr, Layout<3>::bytes);
  return e != cudaSuccess ? e : verify8_rows_set_attributes();
}

namespace {
template <int kGroups>
cudaError_t launch_groups(const CUtensorMap& k_codes, const CUtensorMap& v_codes, const Verify8Args& a, int ctas,
                          cudaStream_t s) {
  cudaLaunchAttribute attr[1];
  const cudaLaunchConfig_t cfg =
      overlapped_launch((unsigned)ctas, 128 + 256 * kGroups, (size_t)Layout<kGroups>::bytes, s, attr);
  return cudaLaunchKernelEx(&cfg, verify8_kernel<kGroups>, k_codes, v_codes, a, verify8_box_keys(a.v.page_size));
}
}  // namespace

cudaError_t launch_verify8(const CUtensorMap& k_codes, const CUtensorMap& v_codes, const Verify8Args& a,
                           int sm_count, cudaStream_t s) {
  const int ctas = sm_count < kV4MaxCtas ? sm_count : kV4MaxCtas;
  const int groups = (a.v.rows * kGroup + kCols - 1) / kCols;
  if (groups > kMaxGroups) return launch_verify8_rows(k_codes, v_codes, a, ctas, s);
  const cudaError_t e = groups == 1   ? launch_groups<1>(k_codes, v_codes, a, ctas, s)
                        : groups == 2 ? launch_groups<2>(k_codes, v_codes, a, ctas, s)
                                      : launch_groups<3>(k_codes, v_codes, a, ctas, s);
  return e != cudaSuccess ? e : launch_verify4_combine(a.v, ctas, kTileN, kQ8Columns, s);
}

}  // namespace ga

// Decode and verify attention over 4-bit paged caches (format: ga_q4.cuh).
//
// Per sequence with L cached tokens before the window, window row r (position L + r) sees keys
// 0 .. L + r; with s_j = q . k_j / 16, out = (sum_j e^(s_j) v_j / sum_j e^(s_j)) sigmoid(gate).
// Keys and values are widened from their codes without rounding; scores, maxima, sums and O are
// fp32; the weights e^(s - M) are rounded to bf16 for the tensor cores (and summed as rounded,
// so their normalisation is consistent); the output is rounded once.
//
// Work. A stream is (sequence, KV head), its keys in tiles of 128, its rows the window's rows of the
// 12 query heads of the group: one block when that makes at most 96 rows, else two of 6 heads, for
// two neighbouring CTAs. The streams' tiles, end to end, are cut into equal runs, one per CTA or two
// such (one CTA per SM), so any mix of lengths fills the device evenly (a stream counts for a few tiles
// more than it has, its fixed cost): a CTA may end one stream and begin another. The lengths are
// read on the device; every role of every CTA derives the same cut from them. A stream that one CTA
// runs whole is written out by it; a stream cut across CTAs leaves partial O, M, l per CTA (at most
// two per CTA: its first and its last segment), merged by the combine kernel.
//
// A tile of 128 keys moves 128 KiB of widened stores, 160 KiB of operand reads and 72 KiB of codes
// through shared memory, 2,800 cycles of the 2,975 that it takes. Whole calls from cold caches: 8 x 16
// rows over 65,536 keys in 194 us (this kernel alone 173 to 181, 1.14 to 1.19 PFLOP/s), 5 x 6 rows
// over up to 12,345 in 22.5, of which 5 are launch and fill.
//
// Structure (896 threads, 28 warps):
//   warp 0      issues S = Q K^T (tcgen05, M=128, N=128, K=256; Q dims 0..127 in tensor
//               memory, 128..255 in shared memory; lanes past the 96 rows hold whatever is there, and
//               nothing reads their results)
//   warp 1      issues O += P V (M=128, N=256, K=32 per piece of V; P in tensor memory)
//   warps 4-11  softmax: two warpgroups, one per 64-key half of a tile, a query row a thread
//               (warps without rows are idle); they also load Q and write the segment's result
//   warps 2, 3  load the codes and scales of K and V tiles by TMA, a granule of 32 keys a lane
//               (a page holds a multiple of that), through two stages each
//   warps 12-19 widen K, warps 20-27 widen V, four at even and four at odd pieces: a lane turns 64
//               codes of one row into a 128-byte row of the swizzled blocks that the tensor cores read
// K is handed over in four pieces of 64 dims and V in four of 32 keys (16 KiB each), so the
// tensor cores start on the first piece of a tile while the rest is being widened, and give
// its place back as soon as they have read it. The roles run different code at
// once and share the instruction cache: the widening loop is one short body for K and V (with
// the rows unrolled through registers the widening alone took 3,500 cycles a tile).
// Tensor memory: O [0, 256), S [256, 384), Q dims 0..127 [384, 448), P [448, 512).
// Every wait is bounded; a wait that gives up raises the CTA's abort flag, which the others see.
#include <cstddef>

#include "ga_v4.cuh"

namespace ga {
namespace {

constexpr int kThreads = 896;
constexpr int kBlockBytes = 128 * 128;    // 128 rows x 64 dims of bf16
constexpr int kGranule = 32;              // keys per TMA box
constexpr int kStages = 2;                // raw tiles in flight, for K and for V
constexpr int kRawBytes = kTileN * kQ4RowBytes, kRawScaleBytes = kTileN * kQ4ScaleBytes;
constexpr int kQBlockBytes = kV4Lanes * 128;      // 64 dims of the query rows
// Registers: launched at 72 a thread (896 x 72 = 64,512). The issuing warpgroup keeps 64, the
// softmax warpgroups take 120, the four widening ones keep 48: 128 x (64 + 2 x 120 + 4 x 48) =
// 63,488.
constexpr int kRegsIssue = 64, kRegsSoftmax = 120, kRegsWiden = 48;
static_assert(128 * (kRegsIssue + 2 * kRegsSoftmax + 4 * kRegsWiden) <= kThreads * 72,
              "register split");
constexpr uint32_t kTmemO = 0, kTmemS = 256, kTmemQ = 384, kTmemP = 448;
constexpr float kLog2eOver16 = 1.4426950408889634f / 16.0f;
constexpr float kLazyRescale = 8.0f;   // O and l are rescaled when the maximum grows by > 2^8

struct V4Smem {
  uint8_t kt[4][kBlockBytes];              // K tile: 64-dim blocks of 128 keys
  uint8_t vt[4][kBlockBytes];              // V tile: pieces of 32 keys, four 64-dim blocks each
  uint8_t qhi[2][kQBlockBytes];            // Q dims 128..255 (the MMA reads 32 rows past each block)
  uint8_t raw[2 * kStages][kRawBytes];     // code rows: K's stages, then V's
  uint8_t rsc[2 * kStages][kRawScaleBytes];
  V4Cut cut;
  float mx[2][2][kV4Lanes];                // exchange i: each half's row value, by i % 2
  uint64_t raw_full[2 * kStages], raw_empty[2 * kStages];
  uint64_t full[8], empty[8];              // pieces of the K tile, then of the V tile
  uint64_t q_full, s_full, s_free, p_full[2], p_empty[2], o_done, o_free, mx_bar;
  uint64_t drain_qk, drain_pv;
  uint32_t tmem_base;
  int abort;
};
static_assert(sizeof(V4Smem) <= 232448, "227 KiB of shared memory per CTA");
// What the copies, the descriptors and the barrier instructions need of the addresses.
static_assert(offsetof(V4Smem, kt) % 1024 == 0 && offsetof(V4Smem, vt) % 1024 == 0 &&
                  offsetof(V4Smem, qhi) % 1024 == 0 && kQBlockBytes % 1024 == 0 && kBlockBytes % 1024 == 0,
              "swizzled blocks begin at whole atoms");
static_assert(offsetof(V4Smem, raw) % 1024 == 0 && offsetof(V4Smem, rsc) % 128 == 0, "tiles of the copies");
static_assert(offsetof(V4Smem, raw_full) % 8 == 0 && offsetof(V4Smem, full) % 8 == 0 &&
                  offsetof(V4Smem, q_full) % 8 == 0 && offsetof(V4Smem, drain_pv) % 8 == 0,
              "every barrier at 8 bytes");
static_assert(offsetof(V4Smem, vt) + sizeof(V4Smem::vt) <= (1u << 18), "descriptor addresses have 18 bits");

// Two multiply-adds by one operation: a x + b for both x.
__device__ __forceinline__ void fma_f32x2(float& r0, float& r1, float x0, float x1, float a, float b) {
  asm("{\n\t.reg .b64 x, m, c, r;\n\t"
      "mov.b64 x, {%2, %3};\n\tmov.b64 m, {%4, %4};\n\tmov.b64 c, {%5, %5};\n\t"
      "fma.rn.f32x2 r, x, m, c;\n\tmov.b64 {%0, %1}, r;\n\t}"
      : "=f"(r0), "=f"(r1)
      : "f"(x0), "f"(x1), "f"(a), "f"(b));
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

// ------------------------------------------------------------------ loading codes
// Tiles of K (is_v 0) or V (1): four boxes of 32 code rows and four of 32 scale rows, by lanes
// 0 .. 3. A granule with no key of the sequence, or on a page outside the pool (recorded), is
// read past the pool's end, which gives zeros.
__device__ void raw_loader(V4Smem& sm, const CUtensorMap* tm_c, const CUtensorMap* tm_s, int is_v,
                           const Verify4Args& a, volatile int* abort) {
  const int lane = threadIdx.x & 31;
  const long long n_rows = (long long)a.n_pages * kKvHeads * a.page_size;
  uint32_t f = 0;   // tiles issued
  Walk<kTileN> walk(sm.cut);
  Seg seg;
  while (walk.next(sm.cut, a.n_seq, seg)) {
    const int end = cut_len<kTileN>(sm.cut, seg.b, a.rows) + a.rows;
    const int* table = a.page_table + (size_t)seg.b * a.max_pages;
    // this lane's granule of a tile, looked up a tile ahead (its page is in flight meanwhile)
    int page = 0, at = 0;
    bool in = false;
    auto look_up = [&](int kt) {
      const int key0 = kt * kTileN + kGranule * (lane & 3);
      in = key0 < end;
      if (!in) return;
      const int e = key0 / a.page_size;
      page = ld_input(table + e);
      at = seg.head * a.page_size + key0 - e * a.page_size;
    };
    look_up(seg.kt0);
    for (int j = 0; j < seg.n; ++j, ++f) {
      int row = (int)n_rows;
      if (in) {
        if (page >= 0 && page < a.n_pages) row = page * kKvHeads * a.page_size + at;
        else if (lane < 4) record(a.status, kDevBadPage);
      }
      const int st = kStages * is_v + (int)(f % kStages);
      if (!warp_wait(&sm.raw_empty[st], ((f / kStages) & 1) ^ 1, abort)) break;
      if (lane == 0) mbar_arrive_expect_tx(&sm.raw_full[st], kRawBytes + kRawScaleBytes);
      __syncwarp();
      if (lane < 4) {
        tma_load_2d(sm.raw[st] + lane * (kGranule * kQ4RowBytes), tm_c, &sm.raw_full[st], 0, row);
        tma_load_2d(sm.rsc[st] + lane * (kGranule * kQ4ScaleBytes), tm_s, &sm.raw_full[st], 0, row);
      }
      if (j + 1 < seg.n) look_up(seg.kt0 + j + 1);
    }
    if (*abort) break;
  }
  if (*abort) {   // the copies in flight land before the CTA leaves
    for (uint32_t i = f > kStages ? f - kStages : 0; i < f; ++i)
      mbar_wait_quiet(&sm.raw_full[kStages * is_v + (int)(i % kStages)], (i / kStages) & 1, 100000000LL);
  }
}

// ------------------------------------------------------------------ widening
// Warps 0 .. 3 take pieces 0 and 2 of every tile, 4 .. 7 pieces 1 and 3 (all eight at every piece
// cost a third more instructions for the same codes). Warp w of four. K, piece u (64-dim block u):
// keys 32w .. 32w+31, a key a lane. V, piece u (keys 32u ..): keys 32u + 8w .. + 7, four lanes a
// key, a 64-dim block each. Eight neighbouring lanes always hold eight neighbouring rows, so the
// swizzle keeps reads and writes free of bank conflicts.
__device__ void widen_worker(V4Smem& sm, int is_v, volatile int* abort) {
  const int lane = threadIdx.x & 31, w = ((int)(threadIdx.x >> 5) - 12) & 3;
  const int u0 = (((int)(threadIdx.x >> 5) - 12) >> 2) & 1;           // first piece
  const uint32_t row0 = is_v ? 8 * w + (lane & 7) : 32 * w + lane;   // the lane's row in piece 0
  const uint32_t blk = is_v ? (uint32_t)lane >> 3 : 0;               // and 64-dim block of it
  const uint32_t xr = row0 & 7;
  const uint32_t src_u = is_v ? kGranule * kQ4RowBytes : 0u;         // from piece to piece
  const uint32_t scs_u = is_v ? kGranule * kQ4ScaleBytes : 4u;
  const uint32_t ch_u = is_v ? 0u : 2u;                              // 16-byte chunks of the row
  // this lane's 128-byte row in its first piece, and the four 16-byte places of its first 32 codes in
  // it (the last 32 codes' are 64 bytes across)
  const uint32_t dst0 = smem_u32(is_v ? sm.vt[u0] : sm.kt[u0]) + (row0 >> 3) * 1024u + xr * 128u +
                        blk * (kGranule * 128u);
  uint32_t at[4];
#pragma unroll
  for (uint32_t j = 0; j < 4; ++j) at[j] = dst0 + ((j ^ xr) << 4);
  uint64_t* full = sm.full + 4 * is_v;
  uint64_t* empty = sm.empty + 4 * is_v;
  const int n = sm.cut.run_tiles();
  for (int g = 0; g < n; ++g) {
    const int st = kStages * is_v + g % kStages;
    if (!warp_wait(&sm.raw_full[st], (g / kStages) & 1, abort)) return;
    const uint32_t src = smem_u32(sm.raw[st]) + row0 * kQ4RowBytes;
    const uint32_t scs = smem_u32(sm.rsc[st]) + row0 * kQ4ScaleBytes + 4 * blk;
    uint32_t sc = lds_u32(scs + u0 * scs_u), ch = 2 * blk + u0 * ch_u;
    uint4 c0 = lds_v4(src + u0 * src_u + ((ch ^ xr) << 4)), c1 = lds_v4(src + u0 * src_u + (((ch + 1) ^ xr) << 4));
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int u = u0 + 2 * i;
      if (!warp_wait(&empty[u], (g & 1) ^ 1, abort)) return;
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const uint4 c = k ? c1 : c0;
        const uint32_t wd[4] = {c.x, c.y, c.z, c.w};
        const Q4Scale q0 = q4_scale((sc >> (16 * k)) & 0xFFu);
        const Q4Scale q1 = q4_scale((sc >> (16 * k + 8)) & 0xFFu);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          uint32_t o[4];
          q4_widen(wd[j], j < 2 ? q0 : q1, o);
          sts_v4((k ? at[j] ^ 64u : at[j]) + i * (2 * kBlockBytes), o);
        }
      }
      if (i == 0) {   // the next piece's codes, while the stores drain
        sc = lds_u32(scs + (u0 + 2) * scs_u);
        ch += 2 * ch_u;
        c0 = lds_v4(src + (u0 + 2) * src_u + ((ch ^ xr) << 4));
        c1 = lds_v4(src + (u0 + 2) * src_u + (((ch + 1) ^ xr) << 4));
      }
      fence_async_smem();   // the tensor cores read what the lanes wrote
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(&full[u]);
        if (i == 1) mbar_arrive(&sm.raw_empty[st]);
      }
    }
  }
}

// ------------------------------------------------------------------ MMA issue
__device__ void qk_issue(V4Smem& sm, const Verify4Args& a, uint32_t tmem, volatile int* abort) {
  constexpr uint32_t kId = idesc_bf16(128, kTileN, false, false);
  const uint64_t k_desc = sdesc_sw128(smem_u32(sm.kt[0]), 16, 1024);
  const uint64_t q_desc = sdesc_sw128(smem_u32(sm.qhi[0]), 16, 1024);
  Walk<kTileN> walk(sm.cut);
  Seg seg;
  uint32_t g = 0, done = 0;
  while (walk.next(sm.cut, a.n_seq, seg)) {
    if (!warp_wait(&sm.q_full, done & 1, abort)) return;
    for (int j = 0; j < seg.n; ++j, ++g) {
      if (g > 0 && !warp_wait(&sm.s_free, (g - 1) & 1, abort)) return;
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        if (!warp_wait(&sm.full[u], g & 1, abort)) return;
        tc_fence_after();
#pragma unroll
        for (int kk = 0; kk < 4; ++kk) {
          const uint64_t bd = k_desc + (uint64_t)(u * (kBlockBytes >> 4) + kk * 2);
          if (u < 2)
            umma_ts_warp(tmem + kTmemS, tmem + kTmemQ + 32 * u + 8 * kk, bd, kId,
                         (u > 0 || kk > 0) ? 1u : 0u);
          else
            umma_ss_warp(tmem + kTmemS, q_desc + (uint64_t)((u - 2) * (kQBlockBytes >> 4) + kk * 2),
                         bd, kId, 1u);
        }
        umma_commit_warp(&sm.empty[u]);
      }
      umma_commit_warp(&sm.s_full);
    }
    ++done;
  }
}

__device__ void pv_issue(V4Smem& sm, const Verify4Args& a, uint32_t tmem, volatile int* abort) {
  constexpr uint32_t kId = idesc_bf16(128, kDim, false, true);
  const uint64_t v_desc = sdesc_sw128(smem_u32(sm.vt[0]), kGranule * 128, 1024);
  Walk<kTileN> walk(sm.cut);
  Seg seg;
  uint32_t g = 0, done = 0;
  while (walk.next(sm.cut, a.n_seq, seg)) {
    if (done > 0 && !warp_wait(&sm.o_free, (done - 1) & 1, abort)) return;
    for (int j = 0; j < seg.n; ++j, ++g) {
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        if ((u & 1) == 0 && !warp_wait(&sm.p_full[u >> 1], g & 1, abort)) return;
        if (!warp_wait(&sm.full[4 + u], g & 1, abort)) return;
        tc_fence_after();
#pragma unroll
        for (int kk = 0; kk < 2; ++kk)
          umma_ts_warp(tmem + kTmemO, tmem + kTmemP + 16 * u + 8 * kk,
                       v_desc + (uint64_t)(u * (kBlockBytes >> 4) + kk * (2048 >> 4)), kId,
                       (j > 0 || u > 0 || kk > 0) ? 1u : 0u);
        umma_commit_warp(&sm.empty[4 + u]);
        if (u & 1) umma_commit_warp(&sm.p_empty[u >> 1]);   // [1]: O holds every P V so far
      }
    }
    umma_commit_warp(&sm.o_done);
    ++done;
  }
}

// ------------------------------------------------------------------ softmax
// Warpgroup hf takes keys 64 hf .. + 63 of every tile, and dims 128 hf .. + 127 of Q and O.
__device__ void softmax_worker(V4Smem& sm, const Verify4Args& a, uint32_t tmem, int hf,
                               volatile int* abort) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int r = (warp & 3) * 32 + lane;
  const uint32_t lane_off = (uint32_t)((warp & 3) * 32) << 16;
  const uint32_t s_taddr = tmem + kTmemS + lane_off + 64 * hf;
  const uint32_t o_taddr = tmem + kTmemO + lane_off + 128 * hf;
  const int heads = kGroup / row_blocks(a.rows);       // query heads of a row block
  const int rr = r / heads, hh = r - rr * heads;
  const bool valid = rr < a.rows;
  uint32_t g = 0, done = 0, mxn = 0;
  // one exchange of a value with the other warpgroup's thread of the same row (a buffer is
  // written again two exchanges on, after the reader has arrived at the next)
  auto exchange = [&](float mine, float& other) -> bool {
    sm.mx[mxn & 1][hf][r] = mine;
    __syncwarp();
    if (lane == 0) mbar_arrive(&sm.mx_bar);
    const bool ok = warp_wait(&sm.mx_bar, mxn & 1, abort);
    other = sm.mx[mxn & 1][hf ^ 1][r];
    ++mxn;
    return ok;
  };
  Walk<kTileN> walk(sm.cut);
  Seg seg;
  while (walk.next(sm.cut, a.n_seq, seg)) {
    const int L = cut_len<kTileN>(sm.cut, seg.b, a.rows);
    const int limit = L + min(rr, a.rows - 1);   // the row's last visible key
    const int h = seg.head * kGroup + (row_blocks(a.rows) == 2 ? heads * (int)(blockIdx.x & 1) : 0) + hh;
    const size_t row = (size_t)seg.b * a.rows + rr;
    {   // Q: dims 0..127 to tensor memory, 128..255 to shared memory. Both places are free: this
        // warp has seen the last S of the segment before, so its Q K^T are done.
      const uint4* qp = reinterpret_cast<const uint4*>(a.q_prep + (row * kHeads + h) * kDim) + 16 * hf;
      uint32_t x[64];   // all of it in flight at once
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const uint4 t = valid ? ld_input(qp + i) : make_uint4(0u, 0u, 0u, 0u);
        x[4 * i] = t.x; x[4 * i + 1] = t.y; x[4 * i + 2] = t.z; x[4 * i + 3] = t.w;
      }
      if (hf == 0) {
        tc_fence_after();
        tmem_st32(tmem + kTmemQ + lane_off, *reinterpret_cast<uint32_t(*)[32]>(x));
        tmem_st32(tmem + kTmemQ + lane_off + 32, *reinterpret_cast<uint32_t(*)[32]>(x + 32));
      } else {
#pragma unroll
        for (int i = 0; i < 16; ++i)
          *reinterpret_cast<uint4*>(sm.qhi[i >> 3] + sw128_offset((uint32_t)r, (uint32_t)(i & 7))) =
              make_uint4(x[4 * i], x[4 * i + 1], x[4 * i + 2], x[4 * i + 3]);
      }
      if (hf == 0) {
        tmem_wait_st();
        tc_fence_before();
      } else {
        fence_async_smem();
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm.q_full);
    }
    float M = -INFINITY, l = 0.f;
    for (int j = 0; j < seg.n; ++j, ++g) {
      const int key0 = (seg.kt0 + j) * kTileN + 64 * hf;
      if (!warp_wait(&sm.s_full, g & 1, abort)) return;
      tc_fence_after();
      uint32_t sb[64];
      tmem_ld32(s_taddr, *reinterpret_cast<uint32_t(*)[32]>(sb));
      tmem_ld32(s_taddr + 32, *reinterpret_cast<uint32_t(*)[32]>(sb + 32));
      tmem_wait_ld(sb);
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm.s_free);
      if (key0 + 63 > L) {   // some key of the half is hidden from some row
#pragma unroll
        for (int k = 0; k < 64; ++k)
          if (key0 + k > limit) sb[k] = 0xFF800000u;   // -inf: weight 0, never the maximum
      }
      auto f = [&](int k) { return __uint_as_float(sb[k]); };
      float m0 = f(0), m1 = f(1), m2 = f(2), m3 = f(3);
#pragma unroll
      for (int k = 4; k + 7 < 64; k += 8) {
        m0 = max3(m0, f(k), f(k + 1));
        m1 = max3(m1, f(k + 2), f(k + 3));
        m2 = max3(m2, f(k + 4), f(k + 5));
        m3 = max3(m3, f(k + 6), f(k + 7));
      }
      m0 = max3(m0, f(60), f(61));
      m1 = max3(m1, f(62), f(63));
      const float mine = fmaxf(fmaxf(m0, m1), fmaxf(m2, m3));
      float other;
      if (!exchange(mine, other)) return;
      const float top = fmaxf(mine, other) * kLog2eOver16;
      // M starts at the first visible tile's maximum and grows when that is passed by > 2^8
      const bool grow = top > M + kLazyRescale;
      const float newM = grow ? top : M;
      if (__any_sync(0xffffffffu, grow && M != -INFINITY)) {
        const float sc = (grow && M != -INFINITY) ? exp2f(M - newM) : 1.0f;
        // Half 0 scales all 256 columns of O: the next P V reads and writes every one of them and
        // starts when half 0's P is there (p_full[0]), not knowing how far the other half is. With a
        // half of the columns each, that P V could meet columns that half 1 was still scaling.
        if (hf == 0) {
          // O must hold every P V before it is scaled (the other half's last store waited for the
          // P V before the last, and the exchange came after it, so this phase is the next one)
          if (!warp_wait(&sm.p_empty[1], (g - 1) & 1, abort)) return;
          tc_fence_after();
#pragma unroll 1
          for (int c0 = 0; c0 < kDim; c0 += 32) {
            uint32_t o[32];
            tmem_ld32(tmem + kTmemO + lane_off + c0, o);
            tmem_wait_ld(o);
#pragma unroll
            for (int k = 0; k < 32; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * sc);
            tmem_st32(tmem + kTmemO + lane_off + c0, o);
          }
          tmem_wait_st();
        }
        l *= sc;
      }
      M = newM;
      const float mf = M == -INFINITY ? 0.f : M;
      float l0 = 0.f, l1 = 0.f, l2 = 0.f, l3 = 0.f;
#pragma unroll
      for (int k = 0; k < 32; ++k) {
        float t0, t1;
        fma_f32x2(t0, t1, f(2 * k), f(2 * k + 1), kLog2eOver16, -mf);
        sb[k] = pack_bf16x2(ex2_approx(t0), ex2_approx(t1));   // an index already read
        if (k & 1) add_bf16x2(l2, l3, sb[k]);
        else add_bf16x2(l0, l1, sb[k]);
      }
      l += (l0 + l2) + (l1 + l3);
      if (g > 0 && !warp_wait(&sm.p_empty[hf], (g - 1) & 1, abort)) return;
      tc_fence_after();
      tmem_st32(tmem + kTmemP + lane_off + 32 * hf, *reinterpret_cast<uint32_t(*)[32]>(sb));
      tmem_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm.p_full[hf]);
    }
    // the segment's result
    float other_l;
    if (!exchange(l, other_l)) return;
    l += other_l;
    if (!warp_wait(&sm.o_done, done & 1, abort)) return;
    tc_fence_after();
    const float inv = 1.0f / l;   // (every row sees a key: 0 only if all its scores are -inf, then NaN)
    const size_t prow = (size_t)seg.slot * kV4Lanes + r;
    const uint4* gp = reinterpret_cast<const uint4*>(a.qg + (row * kHeads + h) * kQgStride + kDim + 128 * hf);
    uint4* op = reinterpret_cast<uint4*>(a.out + (row * kHeads + h) * kDim + 128 * hf);
    if (seg.whole) {
      // 16 dims at a time, their gates loaded two steps ahead (loads do not pass the stores)
      uint4 g[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) g[i] = valid ? ld_input(gp + i) : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll 1
      for (int c = 0; c < 4; ++c) {
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          uint32_t o[16];
          tmem_ld16(o_taddr + 32 * c + 16 * k, o);
          tmem_wait_ld(o);
          const uint32_t gw[8] = {g[2 * k].x,     g[2 * k].y,     g[2 * k].z,     g[2 * k].w,
                                  g[2 * k + 1].x, g[2 * k + 1].y, g[2 * k + 1].z, g[2 * k + 1].w};
          uint32_t res[8];
#pragma unroll
          for (int q = 0; q < 8; ++q)
            res[q] = pack_bf16x2(__uint_as_float(o[2 * q]) * inv * sigmoid_f(lo_f(gw[q])),
                                 __uint_as_float(o[2 * q + 1]) * inv * sigmoid_f(hi_f(gw[q])));
          if (valid) {
            if (c < 3) {
              g[2 * k] = ld_input(gp + 4 * c + 2 * k + 4);
              g[2 * k + 1] = ld_input(gp + 4 * c + 2 * k + 5);
            }
            op[4 * c + 2 * k] = make_uint4(res[0], res[1], res[2], res[3]);
            op[4 * c + 2 * k + 1] = make_uint4(res[4], res[5], res[6], res[7]);
          }
        }
      }
    } else {
#pragma unroll 1
      for (int c = 0; c < 4; ++c) {
        uint32_t o[32];
        tmem_ld32(o_taddr + 32 * c, o);
        tmem_wait_ld(o);
        if (valid) {
#pragma unroll
          for (int i = 0; i < 8; ++i)
            *part_at(a.part_o, seg.slot, 32 * hf + 8 * c + i, r) = make_float4(__uint_as_float(o[4 * i]), __uint_as_float(o[4 * i + 1]),
                                        __uint_as_float(o[4 * i + 2]), __uint_as_float(o[4 * i + 3]));
        }
      }
    }
    if (valid && !seg.whole && hf == 0)
      reinterpret_cast<float2*>(a.part_ml)[prow] = make_float2(l != l ? l : M, l);   // a NaN row's part weighs NaN, not nothing
    tc_fence_before();
    __syncwarp();
    if (lane == 0) mbar_arrive(&sm.o_free);
    ++done;
  }
}

__global__ void __launch_bounds__(kThreads, 1)
    verify4_kernel(const __grid_constant__ CUtensorMap tm_kc, const __grid_constant__ CUtensorMap tm_vc,
                   const __grid_constant__ CUtensorMap tm_ks, const __grid_constant__ CUtensorMap tm_vs,
                   const __grid_constant__ Verify4Args a) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  if ((smem_u32(smem_raw) & 1023u) != 0u) {
    if (threadIdx.x == 0) record(a.status, kDevBadLaunch);
    return;
  }
  V4Smem& sm = *reinterpret_cast<V4Smem*>(smem_raw);
  const int warp = threadIdx.x >> 5;
  volatile int* abort = &sm.abort;
  // softmax warps with query rows, of each warpgroup's four
  const uint32_t act = (uint32_t)(a.rows * (kGroup / row_blocks(a.rows)) + 31) / 32;
  if (threadIdx.x == 0) {
    sm.abort = 0;
    for (int i = 0; i < 2 * kStages; ++i) {
      mbar_init(&sm.raw_full[i], 1);
      mbar_init(&sm.raw_empty[i], 8);   // one arrival per widening warp
    }
    for (int i = 0; i < 8; ++i) {
      mbar_init(&sm.full[i], 4);         // per widening warp of the piece
      mbar_init(&sm.empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sm.p_full[i], act);      // per softmax warp of the half
      mbar_init(&sm.p_empty[i], 1);
    }
    mbar_init(&sm.q_full, 2 * act);       // per softmax warp
    mbar_init(&sm.s_full, 1);
    mbar_init(&sm.s_free, 2 * act);
    mbar_init(&sm.o_done, 1);
    mbar_init(&sm.o_free, 2 * act);
    mbar_init(&sm.mx_bar, 2 * act);
    mbar_init(&sm.drain_qk, 1);
    mbar_init(&sm.drain_pv, 1);
    mbar_fence_init();
  }
  if (warp == 2 && (threadIdx.x & 31) == 0) {
    tma_prefetch_desc(&tm_kc);
    tma_prefetch_desc(&tm_vc);
    tma_prefetch_desc(&tm_ks);
    tma_prefetch_desc(&tm_vs);
  }
  grid_wait();
  grid_launch_dependents();
  if (warp == 1) {   // after the wait: the kernel before may still need tensor memory until it ends
    tmem_alloc(&sm.tmem_base, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  {   // two block barriers
    const int blocks = row_blocks(a.rows);
    make_cut<kTileN>(a, sm.cut, (int)gridDim.x / blocks, (int)blockIdx.x / blocks);
  }
  tc_fence_after();
  const uint32_t tmem = sm.tmem_base;
  if (warp < 4) {
    const int tiles = sm.cut.run_tiles();
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsIssue));
    if (warp == 0 && tiles > 0) {
      qk_issue(sm, a, tmem, abort);
      umma_commit_warp(&sm.drain_qk);
      mbar_wait_quiet(&sm.drain_qk, 0, 100000000LL);
    }
    if (warp == 1 && tiles > 0) {
      pv_issue(sm, a, tmem, abort);
      umma_commit_warp(&sm.drain_pv);
      mbar_wait_quiet(&sm.drain_pv, 0, 100000000LL);
    }
    if (warp >= 2)
      raw_loader(sm, warp == 2 ? &tm_kc : &tm_vc, warp == 2 ? &tm_ks : &tm_vs, warp - 2, a, abort);
  } else if (warp < 12) {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsSoftmax));
    if ((uint32_t)(warp & 3) < act) softmax_worker(sm, a, tmem, (warp - 4) >> 2, abort);
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsWiden));
    widen_worker(sm, warp >= 20 ? 1 : 0, abort);
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
  if (threadIdx.x == 0 && sm.abort) record(a.status, sm.abort);
}

// ------------------------------------------------------------------ combine
// The streams that the cut left in parts: o = sum_i 2^(M_i - M) O_i / sum_i 2^(M_i - M) l_i over a
// stream's parts, times the gate.
//
// A stream's items are (row, four dims), rows innermost, as the parts lie; a block takes an equal
// share of them. With few streams each has `slices` blocks, about twice the device's CTAs in all (32
// sequences of up to 4,096 keys, one row: a whole call of 22 us; with twice the blocks 25). With many
// (slices 0), most of them whole or of two parts, blocks go by the boundaries that cut streams, n - 1
// to a stream of n parts, kSplit to each, so that one long stream among many short ones is not left to
// few blocks (5 rows of one sequence of 65,536 keys and 63 of 200: 34 us, by streams 76). A thread merges eight parts of an item at
// a time, as they come; where a share has fewer items than the block has threads, a stream of more
// than eight parts is dealt to groups of threads, merged through shared memory. (With all (M, l)
// turned into weights in shared memory first, 76 parts of 96 rows took 28 us.)
constexpr int kCombineThreads = 384, kSplit = 2;
static_assert(kCombineThreads >= kV4MaxSeq, "a sequence a thread");
template <int kTile>
__global__ void __launch_bounds__(kCombineThreads) verify4_combine_kernel(
    const __grid_constant__ Verify4Args a, int workers, int slices) {
  __shared__ int warp_units[kV4MaxSeq / 32], warp_streams[kV4MaxSeq / 32];
  __shared__ int cut_b, cut_head, cut_u0, cut_n;
  __shared__ float4 join_o[kCombineThreads];
  __shared__ float2 join_ml[kCombineThreads];
  const int tid = threadIdx.x;
  const int blocks = row_blocks(a.rows), heads = kGroup / blocks, rows = heads * a.rows;
  // block `at` of a stream's `of`, or of a boundary's; the stream, or the boundary's first worker
  const int of = slices ? slices : kSplit, at = blockIdx.x % of, rest = blockIdx.x / of;
  const int block = slices ? rest / (kKvHeads * a.n_seq) : rest % blocks, w = rest / blocks;
  int tiles = 0;
  if (tid < a.n_seq) {
    bool refused;
    tiles = seq_tiles<kTile>(a, ld_len(a.seq_len + tid), refused);
  }
  if (tid == 0) cut_n = 0;
  const Units q = scan_units<kTile>(tiles, warp_units, warp_streams);
  const int total = q.per_head * kKvHeads, share = v4_share(total, workers);
  if (slices) {
    if (tid == rest % a.n_seq) {
      cut_b = tid;
      cut_head = rest / a.n_seq % kKvHeads;
      cut_u0 = cut_head * q.per_head + q.before;
      cut_n = q.n;
    }
  } else if (const int u = share * (w + 1); u < total) {   // the stream that the boundary cuts, if any
    const int head = u / q.per_head, rem = u - head * q.per_head - q.before;
    if (uncut<kTile>(share) <= rem && rem < q.n) {
      cut_b = tid;
      cut_head = head;
      cut_u0 = u - rem;
      cut_n = q.n;
    }
  }
  __syncthreads();
  // (every block waits, so that the grid's end stands for the attention kernel's too)
  if (cut_n == 0) {   // no stream here
    grid_wait();
    return;
  }
  // its parts: worker c0 has its first tile; boundaries cut it from u0 + uncut on
  const int b = cut_b, head = cut_head, u0 = cut_u0, u1 = u0 + cut_n;
  const int c0 = (min(u0 + uncut<kTile>(share), u1) - 1) / share;
  const int n = (u1 - 1) / share - c0 + 1;
  // part i is of worker c0 + i: its first segment unless the stream began inside the worker's run
  const bool inside = c0 * share < u0;
  auto slot = [&](int i) { return 2 * (blocks * (c0 + i) + block) + (i == 0 && inside ? 1 : 0); };
  // this block's items
  const long long items = rows * (kDim / 4);
  const int shares = slices ? of : of * max(n - 1, 1), share_at = slices ? at : of * (w - c0) + at;
  const int lo = (int)(items * share_at / shares), hi = (int)(items * (share_at + 1) / shares);
  const int count = hi - lo;
  const int groups = max(1, min((n + 7) / 8, kCombineThreads / max(count, 1)));
  const int group = groups > 1 ? tid / count : 0;   // (from `groups` on: idle)
  grid_wait();
  if (n == 1 || count == 0) return;   // (one CTA ran the whole stream and wrote it)
  for (int item = lo + tid - group * count; item < hi; item += kCombineThreads) {
    const int d4 = item / rows, r = item - d4 * rows;
    float M = -INFINITY, L = 0.f;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    auto scale = [&](float top) {   // to a new maximum
      const float f = M == -INFINITY ? 0.f : exp2f(M - top);
      M = top;
      L *= f;
      o.x *= f;
      o.y *= f;
      o.z *= f;
      o.w *= f;
    };
    auto add = [&](float2 x, float4 v) {
      if (x.x == -INFINITY) return;   // no such part, or no key of it is visible
      const float f = exp2f(x.x - M);
      L = fmaf(f, x.y, L);
      o.x = fmaf(f, v.x, o.x);
      o.y = fmaf(f, v.y, o.y);
      o.z = fmaf(f, v.z, o.z);
      o.w = fmaf(f, v.w, o.w);
    };
    for (int i0 = group < groups ? group : n; i0 < n; i0 += 8 * groups) {
      float2 x[8];
      float4 v[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const int i = i0 + k * groups;
        x[k] = make_float2(-INFINITY, 0.f);
        if (i < n) {
          x[k] = reinterpret_cast<const float2*>(a.part_ml)[(size_t)slot(i) * kV4Lanes + r];
          v[k] = *part_at(a.part_o, slot(i), d4, r);
        }
      }
      float top = M;
#pragma unroll
      for (int k = 0; k < 8; ++k) top = fmaxf(top, x[k].x);
      scale(top);
#pragma unroll
      for (int k = 0; k < 8; ++k) add(x[k], v[k]);
    }
    if (groups > 1) {   // every thread has one item: the loop runs once
      join_ml[tid] = make_float2(L != L ? L : M, L);
      join_o[tid] = o;
      __syncthreads();
      if (group > 0) return;
      float top = M;
      for (int k = 1; k < groups; ++k) top = fmaxf(top, join_ml[k * count + tid].x);
      scale(top);
      for (int k = 1; k < groups; ++k) add(join_ml[k * count + tid], join_o[k * count + tid]);
    }
    // times the gate, to the output
    const float inv = 1.0f / L;
    const int rr = r / heads, h = head * kGroup + block * heads + r - rr * heads, p = 4 * d4;
    const size_t row = ((size_t)b * a.rows + rr) * kHeads + h;
    const uint16_t* gates = a.qg + row * kQgStride + kDim;
    uint16_t* out = a.out + row * kDim;
    if (kTile != kTileN) {   // place p + k is dim 32 (p % 8 + k) + p / 8
      const int d = 32 * (p & 7) + (p >> 3);
      const float x[4] = {o.x, o.y, o.z, o.w};
#pragma unroll
      for (int k = 0; k < 4; ++k)
        out[d + 32 * k] = (uint16_t)(pack_bf16x2(x[k] * inv * sigmoid_f(lo_f(ld_input(gates + d + 32 * k))), 0.f) & 0xFFFFu);
    } else {
      const uint2 g = ld_input(reinterpret_cast<const uint2*>(gates + p));
      *reinterpret_cast<uint2*>(out + p) =
          make_uint2(pack_bf16x2(o.x * inv * sigmoid_f(lo_f(g.x)), o.y * inv * sigmoid_f(hi_f(g.x))),
                     pack_bf16x2(o.z * inv * sigmoid_f(lo_f(g.y)), o.w * inv * sigmoid_f(hi_f(g.y))));
    }
  }
}

}  // namespace

size_t verify4_ws_bytes() {
  return (size_t)2 * kV4MaxCtas * kV4Lanes * (kDim + 2) * sizeof(float);
}

cudaError_t verify4_set_attributes() {
  const cudaError_t e = cudaFuncSetAttribute(verify4_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             (int)sizeof(V4Smem));
  return e != cudaSuccess ? e : decode4_set_attributes();
}

cudaError_t launch_verify4_combine(const Verify4Args& a, int workers, int tile, cudaStream_t s) {
  const int blocks = row_blocks(a.rows), streams = a.n_seq * kKvHeads * blocks;
  const int ctas = workers * blocks, slices = streams * 2 >= ctas ? 0 : 2 * ctas / streams < 64 ? 2 * ctas / streams : 64;
  cudaLaunchAttribute attr[1];
  const cudaLaunchConfig_t cfg = overlapped_launch(
      (unsigned)(slices ? streams * slices : (workers - 1) * blocks * kSplit), kCombineThreads, 0, s, attr);
  return tile == kTileN ? cudaLaunchKernelEx(&cfg, verify4_combine_kernel<kTileN>, a, workers, slices)
                        : cudaLaunchKernelEx(&cfg, verify4_combine_kernel<32>, a, workers, slices);
}

cudaError_t launch_verify4(const CUtensorMap& k_codes, const CUtensorMap& v_codes,
                           const CUtensorMap& k_scales, const CUtensorMap& v_scales,
                           const Verify4Args& a, int sm_count, cudaStream_t s) {
  const int ctas = sm_count < kV4MaxCtas ? sm_count : kV4MaxCtas;
  if (a.rows == 1) return launch_decode4(k_codes, v_codes, k_scales, v_scales, a, ctas, s);
  cudaLaunchAttribute attr[1];
  const int blocks = row_blocks(a.rows), workers = ctas / blocks;
  const cudaLaunchConfig_t cfg = overlapped_launch((unsigned)(workers * blocks), kThreads, sizeof(V4Smem), s, attr);
  const cudaError_t e = cudaLaunchKernelEx(&cfg, verify4_kernel, k_codes, v_codes, k_scales, v_scales, a);
  return e != cudaSuccess ? e : launch_verify4_combine(a, workers, kTileN, s);
}

}  // namespace ga

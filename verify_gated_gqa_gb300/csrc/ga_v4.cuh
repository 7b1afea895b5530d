// The attention kernels over 4-bit paged caches (ga_verify4.cu, ga_decode4.cu): how the work is
// cut among the CTAs, and small helpers.
#pragma once
#include "ga_internal.h"
#include "ga_q4.cuh"
#include "ga_sm100.cuh"

namespace ga {

__device__ __forceinline__ void record(int* status, int code) {
  if (code) atomicCAS(status, 0, code);
}
// mbar_wait with a time hint on every try after the first, so that a waiting warp is suspended by
// the hardware: most warps of these kernels wait most of the time, and spinning they took a third of
// the SM's issue slots.
__device__ __forceinline__ bool v4_wait(uint32_t bar, uint32_t parity, volatile int* abort) {
  if (mbar_try_wait(bar, parity)) return true;
  const long long t0 = clock64();
  while (true) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}\n"
        : "=r"(ok)
        : "r"(bar), "r"(parity), "r"(20000u)   // ns
        : "memory");
    if (ok) return true;
    if (*abort) return false;
    if (clock64() - t0 > kWaitCycles) {
      *abort = kDevWaitTimeout;
      return false;
    }
  }
}
// The same in all 32 lanes, which agree on the outcome.
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, volatile int* abort) {
  const bool ok = v4_wait(bar, parity, abort);
  return __all_sync(0xffffffffu, ok);
}
__device__ __forceinline__ bool v4_wait(uint64_t* bar, uint32_t parity, volatile int* abort) {
  return v4_wait(smem_u32(bar), parity, abort);
}
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, volatile int* abort) {
  return warp_wait(smem_u32(bar), parity, abort);
}
__device__ __forceinline__ uint32_t lds_u32(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ uint32_t lds_u16(uint32_t addr) {
  uint16_t v;
  asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ uint4 lds_v4(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}
__device__ __forceinline__ void sts_v4(uint32_t addr, const uint32_t (&v)[4]) {
  asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(v[0]), "r"(v[1]),
               "r"(v[2]), "r"(v[3])
               : "memory");
}
// A tensor load by the calling thread alone.
__device__ __forceinline__ void tma_load_2d(void* dst, const CUtensorMap* map, uint64_t* bar, int c0, int c1) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4}], [%2];" ::"r"(
          smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(c0), "r"(c1)
      : "memory");
}
// The merge reads the lengths before its wait (the attention kernel waited for their writer before it
// let the merge begin): from L2, where they are current.
__device__ __forceinline__ int ld_len(const int* p) {
  int v;
  asm volatile("ld.relaxed.gpu.global.s32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
  return v;
}
__device__ __forceinline__ float sigmoid_f(float g) { return __fdividef(1.0f, 1.0f + __expf(-g)); }
__device__ __forceinline__ float lo_f(uint32_t u) { return __uint_as_float(u << 16); }
__device__ __forceinline__ float hi_f(uint32_t u) { return __uint_as_float(u & 0xFFFF0000u); }


// ------------------------------------------------------------------ the cut of the work
// Key tiles (of kTile keys) of a sequence with L cached tokens and a window of `rows`: none when its
// slot is unused (negative length) or the window passes the end of its page-table row.
template <int kTile>
__device__ __forceinline__ int seq_tiles(const Verify4Args& a, int L, bool& refused) {
  const long long keys = (long long)L + a.rows;
  refused = L >= 0 && (keys > (long long)a.max_pages * a.page_size || keys > GA_MAX_TOKENS);
  return L < 0 || refused ? 0 : (int)((keys + kTile - 1) / kTile);
}
// Query-row blocks of a (sequence, KV head), of 12 or 6 heads each: one while all heads' rows fit in
// kV4Lanes. Two blocks go to two neighbouring CTAs, which run the same share of the tiles at the
// same time (a worker is a CTA, or these two) and so read them from memory once: 8 x 16 rows over
// 65,536 keys read 607 MB when the blocks were streams of their own.
__host__ __device__ __forceinline__ int row_blocks(int rows) {
  return rows * kGroup > kV4Lanes ? 2 : 1;
}

// Forms over the 8-bit cache: query rows on the columns of the MMAs, or on their rows.
constexpr int kQ8Columns = 1, kQ8Rows = 2;

// A stream's units in the cut: its tiles after kLead units of no work, which stand for what a
// segment costs beside its tiles (its queries, the first loads, its result). A boundary inside them,
// or fewer than kFront tiles past them, moves to the stream's beginning: the CTA before is spared a
// segment. Cut by tiles alone, a CTA that meets several short streams takes longer than one inside a
// long one: 64 ragged sequences of up to 8,192 keys, one row: 60 us against 54; of up to 300 keys
// 24 against 18; 5 x 5 rows over up to 12,345 keys 25 against 21; 200 x 5 rows over up to 2,047 93
// against 85. (Equal long streams take the same: 64 x 4,095 keys 53 us.)
// Over the 8-bit cache segments cost less beside their tiles. kQ8Columns: 64 ragged sequences of up to 8,192
// keys 53.5 us with a lead of 3, 54.6 with 4; 256 of up to 1,000 keys 51.4, with 2 52.5 and with 4 54.2.
// kQ8Rows: 64 x 16 rows over up to 4,096 keys 84.0 us with 5, 88.0 with 3 and 86.8 with 8; 64 x 8 rows 62.7,
// with 3 65.2; 20 x 12 rows over up to 3,000 35.4, with 3 37.3.
template <int kTile, int kQ8 = 0>
constexpr int kLead = kTile == 32 ? 16 : kQ8 == kQ8Rows ? 5 : kQ8 ? 3 : 6;
template <int kTile, int kQ8 = 0>
constexpr int kFront = kTile == 32 ? 8 : kQ8 ? 1 : 2;
template <int kTile, int kQ8 = 0>
__device__ __forceinline__ int stream_units(int tiles) {
  return tiles ? tiles + kLead<kTile, kQ8> : 0;
}
// A stream's units that no boundary cuts off from its beginning (few streams are cut finely).
template <int kTile, int kQ8 = 0>
__device__ __forceinline__ int uncut(int share) {
  return kLead<kTile, kQ8> + min(kFront<kTile, kQ8>, share);
}

// A worker's share of the streams' units: `left` units from unit `at` of stream (head, b) on.
// Streams are ordered by KV head, then sequence.
struct Seg {
  int head, b, kt0, n;    // tiles kt0 .. kt0 + n - 1 of the stream
  bool whole;             // all of the stream's tiles
  int slot;               // partial slot of a segment that is not whole
};
// What every role of a CTA derives its share from, in shared memory.
struct V4Cut {
  uint16_t tiles[kV4MaxSeq];   // key tiles of each sequence
  uint8_t spare[kV4MaxSeq];    // and what its keys lack of filling the last
  int warp_units[kV4MaxSeq / 32], warp_streams[kV4MaxSeq / 32];   // of 32 sequences, one head
  int at[2], tiles_at[2];      // the worker's run of units, and the tiles before its ends
  int head0, b0, at0;          // the stream that it begins in
  __device__ __forceinline__ int run_tiles() const { return tiles_at[1] - tiles_at[0]; }
};
static_assert((long long)kKvHeads * kV4MaxSeq * (GA_MAX_TOKENS / 32 + kLead<32>) + (1 << 20) < (1LL << 31),
              "unit counts of a launch fit in 32 bits");
// Units per worker of a cut of `total` units.
__device__ __forceinline__ int v4_share(int total, int workers) { return (total + workers - 1) / workers; }

// The units of sequence threadIdx.x's streams, and sums over the sequences, for one KV head.
struct Units {
  int n, before, per_head;    // its units, those of the sequences before it, all
  int streams, all_streams;   // streams before it, all
};
// By a whole block of at least kV4MaxSeq threads, a sequence each (`tiles` is 0 past the last); one
// block barrier. Short on purpose: this code runs once, from a cold instruction cache, before
// anything can be loaded (a warp's search over the sequences took 2.5 us here).
template <int kTile, int kQ8 = 0>
__device__ __forceinline__ Units scan_units(int tiles, int (&warp_units)[kV4MaxSeq / 32],
                                            int (&warp_streams)[kV4MaxSeq / 32]) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int n = stream_units<kTile, kQ8>(tiles);
  int sum = n, streams = 0;
  if (threadIdx.x < kV4MaxSeq) {
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const int o = __shfl_up_sync(0xffffffffu, sum, off);
      if (lane >= off) sum += o;
    }
    streams = __popc(__ballot_sync(0xffffffffu, n > 0) & (0xffffffffu >> (31 - lane)));
    if (lane == 31) {
      warp_units[warp] = sum;
      warp_streams[warp] = streams;
    }
  }
  __syncthreads();
  Units u = {n, sum - n, 0, n ? streams - 1 : streams, 0};
#pragma unroll
  for (int w = 0; w < kV4MaxSeq / 32; ++w) {
    const int x = warp_units[w], y = warp_streams[w];
    u.per_head += x;
    u.all_streams += y;
    if (w < warp) {
      u.before += x;
      u.streams += y;
    }
  }
  return u;
}

// The sequences' tiles and the part of the cut of worker `me` of `workers`: both heads' sequences,
// end to end. A refused length is recorded by the first block. Two block barriers.
template <int kTile, int kQ8 = 0>
__device__ __forceinline__ void make_cut(const Verify4Args& a, V4Cut& c, int workers, int me) {
  const int b = threadIdx.x;
  int tiles = 0;
  if (b < kV4MaxSeq && b < a.n_seq) {
    const int L = ld_len(a.seq_len + b);
    bool refused;
    tiles = seq_tiles<kTile>(a, L, refused);
    if (refused && blockIdx.x == 0) record(a.status, kDevBadPosition);
    c.tiles[b] = (uint16_t)tiles;
    c.spare[b] = (uint8_t)(tiles * kTile - L - a.rows);
  }
  const Units q = scan_units<kTile, kQ8>(tiles, c.warp_units, c.warp_streams);
  const int total = q.per_head * kKvHeads, share = v4_share(total, workers);
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int u = share * (me + i);
    if (u >= total) {
      if (b == 0) {
        c.at[i] = total;
        c.tiles_at[i] = total - kLead<kTile, kQ8> * kKvHeads * q.all_streams;
      }
      continue;
    }
    const int head = u / q.per_head, rem = u - head * q.per_head - q.before;
    if (0 <= rem && rem < q.n) {   // one sequence's thread (n is 0 past the last)
      const int rel = rem < uncut<kTile, kQ8>(share) ? 0 : rem;
      const int at = head * q.per_head + q.before + rel;
      c.at[i] = at;
      c.tiles_at[i] = at - kLead<kTile, kQ8> * (head * q.all_streams + q.streams) - min(rel, kLead<kTile, kQ8>);
      if (i == 0) {
        c.head0 = head;
        c.b0 = b;
        c.at0 = rel;
      }
    }
  }
  __syncthreads();
}
// Cached tokens of a sequence that has tiles.
template <int kTile>
__device__ __forceinline__ int cut_len(const V4Cut& c, int b, int rows) {
  return (int)c.tiles[b] * kTile - (int)c.spare[b] - rows;
}
template <int kTile, int kQ8 = 0>
struct Walk {
  int head, b, at, left, seen;
  __device__ __forceinline__ explicit Walk(const V4Cut& c)
      : head(c.head0), b(c.b0), at(c.at0), left(c.at[1] - c.at[0]), seen(0) {}
  __device__ __forceinline__ bool next(const V4Cut& c, int n_seq, Seg& s) {
    if (left <= 0) return false;
    int total = stream_units<kTile, kQ8>(c.tiles[b]);
    while (at >= total) {   // the next stream with tiles
      at = 0;
      if (++b == n_seq) {
        b = 0;
        ++head;
      }
      total = stream_units<kTile, kQ8>(c.tiles[b]);
    }
    const int n = min(left, total - at);   // past the lead: no boundary lies in one
    s.kt0 = max(at - kLead<kTile, kQ8>, 0);
    s.n = at + n - kLead<kTile, kQ8> - s.kt0;
    s.whole = n == total;
    s.head = head;
    s.b = b;
    // of a worker's segments only the first and the last can be parts of a stream
    s.slot = 2 * (int)blockIdx.x + (seen ? 1 : 0);
    ++seen;
    at += n;
    left -= n;
    return true;
  }
};

// A part's O in the workspace: float4 of four dims at (slot, dims / 4, row), rows innermost, so that
// the attention kernel, whose threads hold a row each, writes whole sectors (row after row of 1
// KiB it wrote half sectors, 32 rows an instruction: 3 us a segment). The decode form keeps dims in
// the order that its fragments leave them in: place p is dim 32 (p % 8) + p / 8.
__device__ __forceinline__ float4* part_at(float* part_o, int slot, int d4, int row) {
  return reinterpret_cast<float4*>(part_o) + ((size_t)slot * (kDim / 4) + d4) * kV4Lanes + row;
}

// The log-sum-exp merge of the streams that the cut over `workers` left in parts, after a kernel with
// tiles of `tile` keys (128 or 32), or of a form over the 8-bit cache (q8, or 0).
cudaError_t launch_verify4_combine(const Verify4Args& a, int workers, int tile, int q8, cudaStream_t s);

}  // namespace ga

// The bookkeeping of one serving step, on the device: from each sequence's cached length and
// the tokens it adds, the pages it needs (popped from a stack of free pages and appended to
// its page-table row), the packed row starts, and every new token's cache slot and position.
//
// All of it follows from three exclusive sums over the sequences (tokens, pages taken, pages
// given back), which one CTA forms in shared memory: n_seq <= 2048 is two sequences a thread.
// The lists that follow (pages, tokens) are then dealt to the threads entry by entry, each
// finding its sequence by a binary search of the sums, so that one long prompt among short
// ones costs no more than the same tokens spread evenly. The call is bound by latency (one
// trip for the lengths, one for the pages, one for the table rows), not by bytes.
// Up to kPlanFusedTokens slots the same CTA writes the slots; past that a second launch of
// many CTAs does. 256 sequences of a token: 4.6 us of GPU time; 48 of 2,700: 9.8, of which the first
// launch, whose one CTA deals 4,050 pages, takes 8.5.
#include "ga_internal.h"
#include "ga_sm100.cuh"

namespace ga {
namespace {

constexpr int kThreads = 1024;
constexpr int kSeqPerThread = GA_PLAN_MAX_SEQ / kThreads;
static_assert(kSeqPerThread == 2 && kSeqPerThread * kThreads == GA_PLAN_MAX_SEQ,
              "two sequences per thread");
constexpr int kSlotThreads = 256;
constexpr int kSlotsPerThread = 4;

// Slot and position of packed token t; padding past the last token is -1 and 0.
__device__ __forceinline__ void write_slot(const PlanArgs& a, const unsigned* start, int t,
                                           unsigned tokens) {
  int slot = -1, pos = 0;
  if ((unsigned)t < tokens) {
    const int b = find_seq(start, a.n_seq, (unsigned)t);
    const int p = a.seq_len[b] + (int)((unsigned)t - start[b]);
    const int e = p / a.page_size;
    const int page = a.page_table[(long long)b * a.max_pages + e];
    slot = page * a.page_size + (p - e * a.page_size);
    pos = p + (a.pos_delta ? a.pos_delta[b] : 0);
  }
  a.slot_map[t] = slot;
  if (a.positions) a.positions[t] = pos;
}

struct Triple {
  unsigned tok, need, rel;
};
// (tok and need are at most 2^20 a sequence; what rows claim to hold is only bounded by the table's
// width, so its sum stops at the largest value, which is then refused)
__device__ __forceinline__ Triple add(Triple x, Triple y) {
  const unsigned rel = x.rel + y.rel;
  return Triple{x.tok + y.tok, x.need + y.need, rel < x.rel ? 0xFFFFFFFFu : rel};
}
// Inclusive sums over the lanes of a warp.
__device__ __forceinline__ Triple warp_scan(Triple x, int lane) {
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const Triple o = {__shfl_up_sync(0xFFFFFFFFu, x.tok, off),
                      __shfl_up_sync(0xFFFFFFFFu, x.need, off),
                      __shfl_up_sync(0xFFFFFFFFu, x.rel, off)};
    if (lane >= off) x = add(x, o);
  }
  return x;
}
__device__ __forceinline__ Triple warp_get(Triple x, int from) {
  return Triple{__shfl_sync(0xFFFFFFFFu, x.tok, from), __shfl_sync(0xFFFFFFFFu, x.need, from),
                __shfl_sync(0xFFFFFFFFu, x.rel, from)};
}

__global__ void __launch_bounds__(kThreads) plan_kernel(const __grid_constant__ PlanArgs a,
                                                        int fused) {
  __shared__ unsigned start[GA_PLAN_MAX_SEQ], need0[GA_PLAN_MAX_SEQ], rel0[GA_PLAN_MAX_SEQ];
  __shared__ Triple warp_sum[kThreads / 32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int n = a.n_seq;
  const int count = *a.free_count;
  // this thread's sequences: 2 tid and 2 tid + 1
  Triple mine[kSeqPerThread];
  int held[kSeqPerThread];
  int err = 0;   // one bit per kind
  if (count < 0 || count > a.n_free) err |= 8;
#pragma unroll
  for (int k = 0; k < kSeqPerThread; ++k) {
    const int b = kSeqPerThread * tid + k;
    mine[k] = Triple{0u, 0u, 0u};
    held[k] = 0;
    if (b >= n) continue;
    const int L = a.seq_len[b], add_tok = a.new_len[b];
    held[k] = a.held[b];
    if (held[k] < 0 || held[k] > a.max_pages) {
      err |= 8;
    } else if (add_tok < 0) {
      mine[k].rel = (unsigned)held[k];      // finished: every page goes back
    } else if (L >= 0) {
      const long long end = (long long)L + add_tok;
      if (end > (long long)a.max_pages * a.page_size || end > GA_MAX_TOKENS) {
        err |= 2;
      } else {
        const int pages = (int)((end + a.page_size - 1) / a.page_size);
        mine[k].tok = (unsigned)add_tok;    // at most 2^20 each: the sums stay below 2^32
        mine[k].need = pages > held[k] ? (unsigned)(pages - held[k]) : 0u;
      }
    }
  }
  // exclusive sums: in the thread, over the warp, over the warps
  const Triple sum = add(mine[0], mine[1]);
  const Triple inc = warp_scan(sum, lane);
  if (lane == 31) warp_sum[warp] = inc;
  __syncthreads();
  const Triple w = warp_sum[lane];   // 32 warps
  const Triple winc = warp_scan(w, lane);
  const Triple before =
      warp_get(Triple{winc.tok - w.tok, winc.need - w.need, winc.rel - w.rel}, warp);
  Triple total = warp_get(winc, 31);
  // every thread agrees on the outcome before anything is written
  if (total.tok > (unsigned)a.max_tokens) err |= 1;
  if (count >= 0 && total.need > (unsigned)count) err |= 4;
  if (count >= 0 && (long long)count - total.need + total.rel > a.n_free) err |= 16;
  int any = 0;
  if (__syncthreads_or(err))
    for (int bit = 1; bit <= 16; bit <<= 1) any |= __syncthreads_or(err & bit) ? bit : 0;
  // a sequence past its table (2) comes before the sums' refusals: its pages are not in them
  const int status = any & 8 ? 4 : any & 2 ? 2 : any & 16 ? 4 : any & 1 ? 1 : any & 4 ? 3 : 0;
  if (status) total = Triple{0u, 0u, 0u};
  Triple at = {before.tok + inc.tok - sum.tok, before.need + inc.need - sum.need,
               before.rel + inc.rel - sum.rel};
#pragma unroll
  for (int k = 0; k < kSeqPerThread; ++k) {
    const int b = kSeqPerThread * tid + k;
    if (b >= n) continue;
    start[b] = at.tok;
    need0[b] = at.need;
    rel0[b] = at.rel;
    a.row_start[b] = status ? 0 : (int)at.tok;
    a.held_out[b] = status ? held[k] : mine[k].rel ? 0 : held[k] + (int)mine[k].need;
    at = add(at, mine[k]);
  }
  if (tid == 0) {
    a.row_start[n] = (int)total.tok;
    *a.free_count_out = count - (int)total.need + (int)total.rel;
    a.info[0] = status;
    a.info[1] = (int)total.tok;
    a.info[2] = (int)total.need;
    a.info[3] = (int)total.rel;
  }
  __syncthreads();
  // page i taken (in order of sequence, then of page): the stack's entry count - 1 - i. The
  // first column is the row's pages held before, which held_out still tells.
  for (unsigned i = tid; i < total.need; i += kThreads) {
    const int b = find_seq(need0, n, i);
    const unsigned row_need = (b + 1 < n ? need0[b + 1] : total.need) - need0[b];
    const int col = a.held_out[b] - (int)row_need + (int)(i - need0[b]);
    a.page_table[(long long)b * a.max_pages + col] = a.free_pages[count - 1 - (int)i];
  }
  __syncthreads();
  // pages given back go on top of what is left, in order of sequence, then of page
  for (unsigned i = tid; i < total.rel; i += kThreads) {
    const int b = find_seq(rel0, n, i);
    a.free_pages[count - (int)total.need + (int)i] =
        a.page_table[(long long)b * a.max_pages + (int)(i - rel0[b])];
  }
  if (!fused) return;
  for (int t = tid; t < a.max_tokens; t += kThreads) write_slot(a, start, t, total.tok);
}

// The slots of a large step: a CTA per kSlotThreads * kSlotsPerThread tokens, after plan_kernel.
__global__ void __launch_bounds__(kSlotThreads) plan_slots_kernel(
    const __grid_constant__ PlanArgs a) {
  __shared__ unsigned start[GA_PLAN_MAX_SEQ];
  for (int b = threadIdx.x; b < a.n_seq; b += kSlotThreads) start[b] = (unsigned)a.row_start[b];
  const unsigned tokens = (unsigned)a.info[1];
  __syncthreads();
#pragma unroll
  for (int k = 0; k < kSlotsPerThread; ++k) {
    const int t = (blockIdx.x * kSlotsPerThread + k) * kSlotThreads + threadIdx.x;
    if (t < a.max_tokens) write_slot(a, start, t, tokens);
  }
}

}  // namespace

cudaError_t launch_plan(const PlanArgs& a, cudaStream_t s) {
  const int fused = a.max_tokens <= kPlanFusedTokens ? 1 : 0;
  plan_kernel<<<1, kThreads, 0, s>>>(a, fused);
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess || fused) return e;
  constexpr int kPerCta = kSlotThreads * kSlotsPerThread;
  plan_slots_kernel<<<(a.max_tokens + kPerCta - 1) / kPerCta, kSlotThreads, 0, s>>>(a);
  return cudaGetLastError();
}

}  // namespace ga

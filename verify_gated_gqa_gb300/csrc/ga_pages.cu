// Pages that several sequences hold: forks, pages given back, compaction, and the copies of pages
// that forks and compactions ask for.
//
// The first three are bookkeeping over page tables, a stack of free pages and a count of further
// holders a page. They move a few kilobytes and are bound by latency: a chain of dependent loads
// (a length, an entry, a count) and the barriers between the steps that read and the ones that
// write. Each is one launch of a team, one CTA of 1,024 threads or a cluster of eight, which every
// step deals its entries to; the cluster's hardware barrier stands between the steps.
// The order of what they write is fixed by the inputs alone: sums and counts, no race, decide
// every place.
#include <climits>

#include "ga_internal.h"
#include "ga_sm100.cuh"

namespace ga {
namespace {

constexpr int kThreads = 1024;
constexpr int kTeamCtas = 8;
constexpr int kExchanges = 2;
static_assert(GA_PLAN_MAX_SEQ == 2 * kThreads, "two rows a thread");

__device__ __forceinline__ void record_page(int* status) { atomicCAS(status, 0, (int)kDevBadPage); }

struct Pair {
  unsigned a, b;
};
struct TeamSmem {
  Pair warp_sum[kThreads / 32];
  Pair sums[kExchanges][kTeamCtas];
};

template <int kCtas>
struct Team {
  TeamSmem& sm;
  int rank, gid, size;
  __device__ __forceinline__ explicit Team(TeamSmem& s)
      : sm(s), rank(kCtas > 1 ? (int)cluster_ctarank() : 0), gid(rank * kThreads + (int)threadIdx.x),
        size(kCtas * kThreads) {}
  // All of the team; what was written before is seen after.
  __device__ __forceinline__ void sync() const {
    if (kCtas == 1) {
      __syncthreads();
    } else {
      asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
    }
  }
  // Sums over the threads of this CTA before this one, and over all of it.
  __device__ __forceinline__ Pair block_scan(Pair v, Pair& total) const {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const Pair inc = warp_scan(v, lane);
    if (lane == 31) sm.warp_sum[warp] = inc;
    __syncthreads();
    const Pair w = sm.warp_sum[lane];
    const Pair winc = warp_scan(w, lane);
    const Pair before = {__shfl_sync(~0u, winc.a - w.a, warp) + inc.a - v.a,
                         __shfl_sync(~0u, winc.b - w.b, warp) + inc.b - v.b};
    total = {__shfl_sync(~0u, winc.a, 31), __shfl_sync(~0u, winc.b, 31)};
    __syncthreads();   // warp_sum may be written again
    return before;
  }
  // The same over the team; a sync. Exchange x is used once in a kernel (a CTA may still be reading
  // its copy while another is past it).
  __device__ __forceinline__ Pair scan(int x, Pair v, Pair& total) const {
    Pair before = block_scan(v, total);
    if (kCtas == 1) return before;
    publish(x, total);
    sync();
    total = {0u, 0u};
#pragma unroll
    for (int r = 0; r < kCtas; ++r) {
      const Pair o = sm.sums[x][r];
      if (r < rank) before = {before.a + o.a, before.b + o.b};
      total = {total.a + o.a, total.b + o.b};
    }
    return before;
  }
  // Whether v is set anywhere in the team; a sync.
  __device__ __forceinline__ bool any(int x, bool v) const {
    int r = __syncthreads_or(v);
    if (kCtas == 1) return r != 0;
    publish(x, Pair{(unsigned)r, 0u});
    sync();
#pragma unroll
    for (int i = 0; i < kCtas; ++i) r |= (int)sm.sums[x][i].a;
    return r != 0;
  }

 private:
  __device__ __forceinline__ static Pair warp_scan(Pair v, int lane) {
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const unsigned a = __shfl_up_sync(~0u, v.a, off), b = __shfl_up_sync(~0u, v.b, off);
      if (lane >= off) v = {v.a + a, v.b + b};
    }
    return v;
  }
  // This CTA's value into every CTA's copy.
  __device__ __forceinline__ void publish(int x, Pair v) const {
    if (threadIdx.x < kCtas) {
      const uint32_t at = mapa_shared(smem_u32(&sm.sums[x][rank]), threadIdx.x);
      asm volatile("st.shared::cluster.v2.u32 [%0], {%1, %2};" ::"r"(at), "r"(v.a), "r"(v.b) : "memory");
    }
  }
};

// n entries of one array to another, unless they are the same.
template <int kCtas>
__device__ __forceinline__ void copy_array(const Team<kCtas>& t, const int* from, int* to, int n) {
  if (from == to) return;
  for (int i = t.gid; i < n; i += t.size) to[i] = from[i];
}

// ------------------------------------------------------------------ forks
// Every CTA checks all forks (two a thread) and forms the same sums; the whole pages of all forks,
// end to end, are then dealt to the team's threads.
template <int kCtas>
__global__ void __launch_bounds__(kThreads) fork_kernel(const __grid_constant__ ForkArgs a) {
  __shared__ TeamSmem tsm;
  __shared__ unsigned start[GA_PLAN_MAX_SEQ], named[GA_PLAN_MAX_SEQ / 32];
  const Team<kCtas> team(tsm);
  const int tid = threadIdx.x;
  grid_wait();
  grid_launch_dependents();
  if (tid < GA_PLAN_MAX_SEQ / 32) named[tid] = 0u;
  copy_array(team, a.shared, a.shared_out, a.n_free);
  const int count = *a.free_count;
  int err = count < 0 || count > a.n_free ? 8 : 0;
  __syncthreads();
  int parent[2], child[2], len[2], held_c[2] = {0, 0};
  Pair need[2];   // whole pages, a page begun
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const int i = 2 * tid + k;
    parent[k] = -1;
    need[k] = {0u, 0u};
    if (i >= a.n_fork) continue;
    parent[k] = a.parent[i];
    child[k] = a.child[i];
    len[k] = a.len[i];
    if (parent[k] < 0) continue;
    if (parent[k] >= a.n_seq || child[k] < 0 || child[k] >= a.n_seq || parent[k] == child[k]) {
      err |= 1;
      continue;
    }
    const int held_p = a.held[parent[k]];
    held_c[k] = a.held[child[k]];
    if (held_p < 0 || held_p > a.max_pages || held_c[k] < 0 || held_c[k] > a.max_pages) err |= 8;
    if (held_c[k] != 0 || (atomicOr(&named[child[k] >> 5], 1u << (child[k] & 31)) >> (child[k] & 31) & 1u))
      err |= 1;
    if (len[k] < 0 || (long long)len[k] > (long long)held_p * a.page_size) {
      err |= 2;
      continue;
    }
    need[k] = {(unsigned)(len[k] / a.page_size), len[k] % a.page_size ? 1u : 0u};
  }
  Pair total;
  const Pair before = team.block_scan(Pair{need[0].a + need[1].a, need[0].b + need[1].b}, total);
  if (count >= 0 && total.b > (unsigned)count) err |= 4;
  for (int b = tid; b < a.n_seq; b += kThreads)   // rows that no fork names count too
    if (a.held[b] < 0 || a.held[b] > a.max_pages) err |= 8;
  int all = 0;
  for (int bit = 1; bit <= 8; bit <<= 1) all |= __syncthreads_or(err & bit) ? bit : 0;
  const int status = all & 8 ? 4 : all & 1 ? 1 : all & 2 ? 2 : all & 4 ? 3 : 0;
  int forks = 0;
  if (status) total = {0u, 0u};
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    start[2 * tid + k] = k ? before.a + need[0].a : before.a;
    forks += parent[k] >= 0 && !status;
  }
  const int made = __syncthreads_count(forks > 0) + __syncthreads_count(forks > 1);
  copy_array(team, a.held, a.held_out, a.n_seq);
  team.sync();   // every CTA has read what is written from here on
  if (team.rank == 0) {
    if (tid == 0) {
      *a.free_count_out = count - (int)total.b;
      a.info[0] = status;
      a.info[1] = made;
      a.info[2] = (int)total.b;
      a.info[3] = (int)total.a;
    }
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const int i = 2 * tid + k;
      if (i >= a.n_fork) continue;
      int src = -1, dst = -1;
      if (parent[k] >= 0 && !status) {
        a.held_out[child[k]] = (int)(need[k].a + need[k].b);
        if (need[k].b) {
          src = a.page_table[(long long)parent[k] * a.max_pages + need[k].a];
          dst = a.free_pages[count - 1 - (int)(k ? before.b + need[0].b : before.b)];
          a.page_table[(long long)child[k] * a.max_pages + need[k].a] = dst;
          if (src < 0 || src >= a.n_free || dst < 0 || dst >= a.n_free) {
            record_page(a.status);
            src = dst = -1;
          }
        }
      }
      a.copy_src[i] = src;
      a.copy_dst[i] = dst;
    }
  }
  for (unsigned i = team.gid; i < total.a; i += team.size) {
    const int f = find_seq(start, a.n_fork, i);
    const unsigned col = i - start[f];
    const int page = a.page_table[(long long)a.parent[f] * a.max_pages + col];
    a.page_table[(long long)a.child[f] * a.max_pages + col] = page;
    if (page < 0 || page >= a.n_free) record_page(a.status);
    else atomicAdd(a.shared_out + page, 1);
  }
}

// ------------------------------------------------------------------ pages given back
// The pages that the rows let go, end to end in order of row and column, are dealt to the team's
// threads in runs. `shared` counts a page's holders less one, so once each place has taken one off,
// a page is free where -1 is left, and one that found less than 0 was let go too often. A free page's
// first place is found by a minimum over its places' numbers in the same word, from INT_MIN up.
template <int kCtas>
__global__ void __launch_bounds__(kThreads) release_kernel(const __grid_constant__ ReleaseArgs a) {
  __shared__ TeamSmem tsm;
  __shared__ unsigned start[GA_PLAN_MAX_SEQ];
  __shared__ int kept[GA_PLAN_MAX_SEQ];
  const Team<kCtas> team(tsm);
  const int tid = threadIdx.x;
  grid_wait();
  grid_launch_dependents();
  copy_array(team, a.shared, a.shared_out, a.n_free);
  const int count = *a.free_count;
  int err = count < 0 || count > a.n_free ? 8 : 0;
  unsigned gone[2], rows = 0;
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const int b = 2 * tid + k;
    gone[k] = 0u;
    if (b >= a.n_seq) continue;
    const int held = a.held[b], keep = a.keep[b];
    int left = held;
    if (held < 0 || held > a.max_pages) {
      err |= 8;
    } else if (keep >= 0) {
      left = min(held, (int)(((long long)keep + a.page_size - 1) / a.page_size));
      gone[k] = (unsigned)(held - left);   // n_seq * max_pages < 2^30
    }
    kept[b] = left;
    rows += gone[k] > 0;
  }
  Pair total;
  const Pair before = team.block_scan(Pair{gone[0] + gone[1], rows}, total);
  start[2 * tid] = before.a;
  start[2 * tid + 1] = before.a + gone[0];
  const bool range = __syncthreads_or(err) != 0;   // the same in every CTA
  team.sync();   // every CTA has read what is written from here on
  int status = range ? 4 : 0;
  unsigned freed = 0;
  if (!status && total.a > 0u) {
    // this thread's places; as many of their pages as fit stay in registers, so that the loads of a step
    // are all in flight at once (one by one, 27,714 pages took 21 us)
    constexpr unsigned kKeep = 8;
    const unsigned per = (total.a + team.size - 1) / team.size;
    const unsigned lo = min(total.a, per * team.gid), hi = min(total.a, lo + per);
    const int row0 = lo < hi ? find_seq(start, a.n_seq, lo) : 0;
    auto page_at = [&](unsigned i, int& b) {
      while (b + 1 < a.n_seq && start[b + 1] <= i) ++b;
      return a.page_table[(long long)b * a.max_pages + kept[b] + (int)(i - start[b])];
    };
    int pages[kKeep], b1 = row0;
#pragma unroll
    for (unsigned k = 0; k < kKeep; ++k) pages[k] = lo + k < hi ? page_at(lo + k, b1) : -1;
#pragma unroll
    for (unsigned k = 0; k < kKeep; ++k)
      if (lo + k < hi && (unsigned)pages[k] >= (unsigned)a.n_free) {   // passed over
        record_page(a.status);
        pages[k] = -1;
      }
    // f(place, page) over them, load(page) first for a batch
    auto each = [&](auto load, auto f) {
      int got[kKeep];
#pragma unroll
      for (unsigned k = 0; k < kKeep; ++k)
        if (pages[k] >= 0) got[k] = load(pages[k]);
#pragma unroll
      for (unsigned k = 0; k < kKeep; ++k)
        if (pages[k] >= 0) f(lo + k, pages[k], got[k]);
      int b = b1;
      for (unsigned i = lo + kKeep; i < hi; ++i) {
        const int page = page_at(i, b);
        if ((unsigned)page < (unsigned)a.n_free) f(i, page, load(page));
        else record_page(a.status);
      }
    };
    volatile int* left = a.shared_out;
    auto read = [&](int page) { return left[page]; };
    auto nothing = [](int) { return 0; };
    auto put_back = [&]() {   // as it was
      each(nothing, [&](unsigned, int page, int) { atomicAdd(a.shared_out + page, 1); });
    };
    bool bad = false;
    each([&](int page) { return atomicSub(a.shared_out + page, 1); }, [&](unsigned, int, int was) { bad |= was < 0; });
    if (team.any(0, bad)) {
      status = 5;
      put_back();
    } else {
      each(read, [&](unsigned i, int page, int v) {
        if (v < 0) atomicMin(a.shared_out + page, INT_MIN + (int)i);
      });
      team.sync();
      // first places: those in registers are remembered, later ones read again
      Pair own = {0u, 0u}, sum;
      uint32_t firsts = 0u;
      each(read, [&](unsigned i, int, int v) {
        const bool is = v == INT_MIN + (int)i;
        own.a += is;
        if (i - lo < kKeep) firsts |= (uint32_t)is << (i - lo);
      });
      unsigned to = team.scan(1, own, sum).a;
      if ((long long)count + sum.a > a.n_free) {
        status = 4;
        each(read, [&](unsigned i, int page, int v) {
          if (v == INT_MIN + (int)i) left[page] = -1;
        });
        team.sync();
        put_back();
      } else {
        freed = sum.a;
        const auto again = [&](int page) { return hi - lo > kKeep ? left[page] : 0; };
        each(again, [&](unsigned i, int page, int v) {
          if (i - lo < kKeep ? !(firsts >> (i - lo) & 1u) : v != INT_MIN + (int)i) return;
          a.free_pages[count + (int)to++] = page;
          left[page] = 0;
        });
      }
    }
  }
  for (int b = team.gid; b < a.n_seq; b += team.size)
    if (status == 0) a.held_out[b] = kept[b];
    else if (a.held_out != a.held) a.held_out[b] = a.held[b];
  if (team.gid == 0) {
    *a.free_count_out = count + (int)freed;
    a.info[0] = status;
    a.info[1] = status ? 0 : (int)total.b;
    a.info[2] = (int)freed;
    a.info[3] = status ? 0 : (int)total.a;
  }
}

// ------------------------------------------------------------------ compaction
// map[p] first tells whether page p is free, then where its contents go. Each warp has a run of pages,
// in order, so that its loads are whole lines (with a run a thread 262,144 pages took 197 us, so they take
// 61; 1,024 pages 5.0 and 6.0). Sums of free pages below n_live and of pages in use from it on give the
// moves their numbers, and those give every place on the new stack.
// Batches of 32 pages loaded together (1: 262,144 pages 66 us; 4: 59, but 2,048 7.5 for 7.1).
constexpr int kMapBatch = 2;
template <int kCtas>
__global__ void __launch_bounds__(kThreads) compact_kernel(const __grid_constant__ CompactArgs a, int remap) {
  __shared__ TeamSmem tsm;
  const Team<kCtas> team(tsm);
  grid_wait();
  grid_launch_dependents();
  const int n = a.n_free, count = *a.free_count;
  bool err = count < 0 || count > n;
  for (int b = team.gid; b < a.n_seq; b += team.size) err |= a.held[b] < 0 || a.held[b] > a.max_pages;
  for (int p = team.gid; p < n; p += team.size) a.map[p] = 0;
  team.sync();
  if (count >= 0 && count <= n) {
    for (int i = team.gid; i < count; i += team.size) {
      const int p = a.free_pages[i];
      if (p < 0 || p >= n || atomicExch(a.map + p, 1) != 0) err = true;
    }
  }
  const long long entries = (long long)a.n_seq * a.max_pages;
  if (team.any(0, err)) {
    if (a.page_table != a.page_table_out && remap)
      for (long long i = team.gid; i < entries; i += team.size) a.page_table_out[i] = a.page_table[i];
    copy_array(team, a.free_pages, a.free_pages_out, n);
    copy_array(team, a.shared, a.shared_out, n);
    for (int i = team.gid; i < a.max_moves; i += team.size) a.move_src[i] = a.move_dst[i] = -1;
    if (team.gid < 4) a.info[team.gid] = team.gid == 0 ? 4 : 0;
    return;
  }
  volatile int* map = a.map;
  const int live = n - count;
  const int lane = threadIdx.x & 31;
  const uint32_t before_lane = (1u << lane) - 1u;
  const int warps = team.size / 32, per = (n + warps - 1) / warps;
  const int lo = (int)min((long long)n, (long long)per * (team.gid / 32)), hi = min(n, lo + per);
  // f(page or -1, whether it is free) in order of the warp's run; all lanes call it
  auto each = [&](auto f) {
    for (int p0 = lo; p0 < hi; p0 += 32 * kMapBatch) {
      int free[kMapBatch];
#pragma unroll
      for (int k = 0; k < kMapBatch; ++k) free[k] = p0 + 32 * k + lane < hi ? map[p0 + 32 * k + lane] : 0;
#pragma unroll
      for (int k = 0; k < kMapBatch; ++k) {
        const int p = p0 + 32 * k + lane;
        if (p - lane < hi) f(p < hi ? p : -1, free[k] != 0);
      }
    }
  };
  // free pages below live, and pages in use from it on: as many of each
  auto is_hole = [&](int p, bool free) { return p >= 0 && p < live && free; };
  auto is_mover = [&](int p, bool free) { return p >= live && !free; };
  Pair own = {0u, 0u}, sum;
  each([&](int p, bool free) {
    own.a += is_hole(p, free);
    own.b += is_mover(p, free);
  });
  own = {__reduce_add_sync(~0u, own.a), __reduce_add_sync(~0u, own.b)};
  if (lane != 0) own = {0u, 0u};
  Pair at = team.scan(1, own, sum);
  at = {__shfl_sync(~0u, at.a, 0), __shfl_sync(~0u, at.b, 0)};
  const int all = (int)sum.b, moves = min(a.max_moves, all);
  // f(page or -1, free, holes before it, movers before it)
  auto each_numbered = [&](auto f) {
    int holes = (int)at.a, movers = (int)at.b;
    each([&](int p, bool free) {
      const uint32_t h = __ballot_sync(~0u, is_hole(p, free)), m = __ballot_sync(~0u, is_mover(p, free));
      if (p >= 0) f(p, free, holes + __popc(h & before_lane), movers + __popc(m & before_lane));
      holes += __popc(h);
      movers += __popc(m);
    });
  };
  // the lowest holes take the highest movers, highest first
  each_numbered([&](int p, bool free, int holes, int movers) {
    if (is_hole(p, free) && holes < moves) a.move_dst[holes] = p;
    if (is_mover(p, free) && all - 1 - movers < moves) a.move_src[all - 1 - movers] = p;
  });
  for (int i = moves + team.gid; i < a.max_moves; i += team.size) a.move_src[i] = a.move_dst[i] = -1;
  team.sync();
  volatile int* dst = a.move_dst;
  each_numbered([&](int p, bool free, int holes, int movers) {
    // free pages before p afterwards: the holes left, and past live every page but those still in use
    const int rank = max(holes - moves, 0) + max(p - live, 0) - movers + max(0, movers - (all - moves));
    int to = p;
    bool free_after = free;
    const int number = all - 1 - movers;
    if (is_hole(p, free) && holes < moves) {
      free_after = false;   // its count comes with its contents
    } else if (is_mover(p, free) && number < moves) {
      to = dst[number];
      free_after = true;
      a.shared_out[to] = a.shared[p];
      a.shared_out[p] = 0;
    } else if (a.shared != a.shared_out) {
      a.shared_out[p] = a.shared[p];
    }
    map[p] = to;
    if (free_after) a.free_pages_out[count - 1 - rank] = p;
  });
  if (a.free_pages != a.free_pages_out)
    for (int i = count + team.gid; i < n; i += team.size) a.free_pages_out[i] = a.free_pages[i];
  if (team.gid == 0) {
    a.info[0] = 0;
    a.info[1] = moves;
    a.info[2] = live;
    a.info[3] = all - moves;
  }
  if (!remap) return;
  team.sync();
  for (long long i = team.gid; i < entries; i += team.size) {
    const int b = (int)(i / a.max_pages), col = (int)(i - (long long)b * a.max_pages);
    int p = a.page_table[i];
    if (col < a.held[b]) {
      if (p >= 0 && p < n) p = map[p];
      else record_page(a.status);
    }
    a.page_table_out[i] = p;
  }
}

// The table of a large batch: a CTA per kRemapEntries of it, after compact_kernel, whose cluster would take
// longer over it than a launch costs: 65,536 entries 10.8 us for 13.2 within, a million 35 for 96, but 8,192
// 12.5 for 11.0.
constexpr long long kRemapInside = 32768;
constexpr int kRemapThreads = 256, kRemapEntries = 1024;
__global__ void __launch_bounds__(kRemapThreads) remap_kernel(const __grid_constant__ CompactArgs a) {
  const long long entries = (long long)a.n_seq * a.max_pages;
  const bool refused = a.info[0] != 0;
#pragma unroll
  for (int k = 0; k < kRemapEntries / kRemapThreads; ++k) {
    const long long i = (long long)blockIdx.x * kRemapEntries + k * kRemapThreads + threadIdx.x;
    if (i >= entries) return;
    const int b = (int)(i / a.max_pages), col = (int)(i - (long long)b * a.max_pages);
    int p = a.page_table[i];
    if (!refused && col < a.held[b]) {
      if (p >= 0 && p < a.n_free) p = a.map[p];
      else record_page(a.status);
    }
    a.page_table_out[i] = p;
  }
}

// ------------------------------------------------------------------ copies of pages
// An item is a piece of a copied page of one pool. Pools whose pages are 16-byte aligned and not small
// go in pieces of up to 32 KiB through shared memory by bulk copies, three loads and three stores in
// flight from one thread of each CTA; the others (scales, odd sizes) through registers by the other
// warps, a page an item. Bound by the bytes, in and out.
constexpr int kCopyThreads = 256, kCopyLoads = 4;
constexpr int kPieceBytes = 32768, kCopyStages = 6, kCopyAhead = 3;
// Smaller pages go through registers: 512 pages of 2 KiB take 2.3 us there, 4.0 by bulk copies (one thread
// issues a CTA's), 8 of 4 KiB 2.8 against 2.1.
constexpr int kBulkLeast = 4096;

template <typename T>
__device__ __forceinline__ void copy_page(const uint8_t* from, uint8_t* to, long long bytes, int tid, int threads) {
  for (long long off = 0; off < bytes; off += (long long)kCopyLoads * threads * sizeof(T)) {
    T v[kCopyLoads];
#pragma unroll
    for (int k = 0; k < kCopyLoads; ++k) {
      const long long at = off + ((long long)k * threads + tid) * sizeof(T);
      if (at < bytes) v[k] = *reinterpret_cast<const T*>(from + at);
    }
#pragma unroll
    for (int k = 0; k < kCopyLoads; ++k) {
      const long long at = off + ((long long)k * threads + tid) * sizeof(T);
      if (at < bytes) *reinterpret_cast<T*>(to + at) = v[k];
    }
  }
}

// Copy i's pages, or src -1: an entry to pass over (a page outside the pool is recorded).
__device__ __forceinline__ int2 copy_entry(const PageCopyArgs& a, long long i) {
  int2 e = make_int2(a.src[i], a.dst[i]);
  if (e.x < 0 || e.y < 0) {
    e.x = -1;
  } else if (e.x >= a.n_pages || e.y >= a.n_pages) {
    record_page(a.status);
    e.x = -1;
  }
  return e;
}

struct CopySmem {
  uint8_t stages[kCopyStages][kPieceBytes];
  uint64_t full[kCopyStages];
  uint8_t* to[kCopyStages];   // of the loads in flight
  int bytes[kCopyStages], abort;
};

// The bulk pieces of this CTA, by one warp: items blockIdx.x, + gridDim.x, ...
__device__ void copy_bulk(const PageCopyArgs& a, CopySmem& sm) {
  const int lane = threadIdx.x & 31;
  const long long items = (long long)a.n_copies * a.pieces;
  long long next = blockIdx.x;
  // 32 items at a time, an item a lane; those to be done are gathered in the lanes 0 .. have - 1
  const uint8_t* from = nullptr;
  uint8_t* to = nullptr;
  int bytes = 0, have = 0, at = 0;
  auto fetch = [&]() {   // whether there is another item: lane `at`'s
    while (at == have && next < items) {
      const long long w = next + (long long)lane * gridDim.x;
      bytes = 0;
      if (w < items) {
        const long long i = w / a.pieces;
        const int piece = (int)(w - i * a.pieces);
        int j = 0;
        while (piece < a.pool[j].first || piece >= a.pool[j].first + a.pool[j].pieces) ++j;
        const PageCopyArgs::Pool& p = a.pool[j];
        const int2 e = copy_entry(a, i);
        if (e.x >= 0) {
          const long long off = (long long)(piece - p.first) * a.piece_bytes;
          from = p.base + e.x * p.bytes + off;
          to = p.base + e.y * p.bytes + off;
          bytes = (int)min((long long)a.piece_bytes, p.bytes - off);
        }
      }
      next += 32LL * gridDim.x;
      const uint32_t live = __ballot_sync(~0u, bytes > 0);
      have = __popc(live);
      at = 0;
      const int pick = lane < have ? (int)__fns(live, 0, lane + 1) : 0;
      from = (const uint8_t*)__shfl_sync(~0u, (unsigned long long)from, pick);
      to = (uint8_t*)__shfl_sync(~0u, (unsigned long long)to, pick);
      bytes = __shfl_sync(~0u, bytes, pick);
    }
    return at < have;
  };
  unsigned n = 0, m = 0;   // loaded, stored
  volatile int* abort = &sm.abort;
  while (true) {
    while (n - m < kCopyAhead && fetch()) {
      const unsigned st = n % kCopyStages;
      const uint8_t* src = (const uint8_t*)__shfl_sync(~0u, (unsigned long long)from, at);
      uint8_t* dst = (uint8_t*)__shfl_sync(~0u, (unsigned long long)to, at);
      const int size = __shfl_sync(~0u, bytes, at);
      if (lane == 0) {
        // the stage's last store, one of those before the last kCopyStages - kCopyAhead, has read it
        asm volatile("cp.async.bulk.wait_group.read %0;" ::"n"(kCopyStages - kCopyAhead) : "memory");
        sm.to[st] = dst;
        sm.bytes[st] = size;
        mbar_arrive_expect_tx(&sm.full[st], (uint32_t)size);
        asm volatile(
            "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                smem_u32(sm.stages[st])),
            "l"(src), "r"(size), "r"(smem_u32(&sm.full[st]))
            : "memory");
      }
      ++at;
      ++n;
      __syncwarp();
    }
    if (m == n) break;
    const unsigned st = m % kCopyStages;
    if (!__all_sync(~0u, mbar_wait(&sm.full[st], (m / kCopyStages) & 1u, abort))) {
      for (unsigned k = m; k < n; ++k)   // the loads in flight land before the CTA leaves
        mbar_wait_quiet(&sm.full[k % kCopyStages], (k / kCopyStages) & 1u, 100000000LL);
      if (lane == 0) atomicCAS(a.status, 0, *abort);
      break;
    }
    if (lane == 0) {
      asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(sm.to[st]),
                   "r"(smem_u32(sm.stages[st])), "r"(sm.bytes[st])
                   : "memory");
      bulk_commit_group();
    }
    ++m;
    __syncwarp();
  }
  if (lane == 0) bulk_wait_group0();
}

__global__ void __launch_bounds__(kCopyThreads) copy_kernel(const __grid_constant__ PageCopyArgs a) {
  extern __shared__ __align__(128) uint8_t raw[];
  CopySmem& sm = *reinterpret_cast<CopySmem*>(raw);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    sm.abort = 0;
    for (int i = 0; i < kCopyStages; ++i) mbar_init(&sm.full[i], 1);
    mbar_fence_init();
  }
  __syncthreads();
  grid_wait();
  grid_launch_dependents();
  if (warp == 0) {
    if (a.pieces > 0) copy_bulk(a, sm);
    return;
  }
  if (!a.small) return;
  constexpr int kWarps = kCopyThreads / 32 - 1;
  for (long long i = (long long)blockIdx.x * kWarps + warp - 1; i < a.n_copies; i += (long long)gridDim.x * kWarps) {
    const int2 e = copy_entry(a, i);
    if (e.x < 0) continue;
    for (int j = 0; j < a.n_pools; ++j) {
      const PageCopyArgs::Pool& p = a.pool[j];
      if (p.pieces > 0) continue;
      const uint8_t* from = p.base + e.x * p.bytes;
      uint8_t* to = p.base + e.y * p.bytes;
      switch (p.width) {
        case 16: copy_page<uint4>(from, to, p.bytes, lane, 32); break;
        case 8: copy_page<uint2>(from, to, p.bytes, lane, 32); break;
        case 4: copy_page<uint32_t>(from, to, p.bytes, lane, 32); break;
        case 2: copy_page<uint16_t>(from, to, p.bytes, lane, 32); break;
        default: copy_page<uint8_t>(from, to, p.bytes, lane, 32);
      }
    }
  }
}

// One CTA while a step's entries are few (its barriers are cheaper), else the cluster of eight: 1,024 table
// entries let go 7.8 us against 10.0, 2,048 10.7 against 10.2 and 4,096 17.3 against 10.5; forks of 1,008
// entries 5.1 against 5.4, of 2,016 6.3 against 5.5. Copying an array of 8,192 pages costs one CTA as much
// as its barriers save (forks of 252 entries 5.4 against 4.8), and a compaction of 2,048 pages takes 6.9
// against 9.0, of 4,096 11.6 against 9.2. All may be placed while the kernel before them ends.
constexpr long long kOneCtaEntries = 1024, kOneCtaCopies = 8192, kOneCtaPages = 2048;
template <typename K1, typename K8, typename... A>
cudaError_t launch_team(K1 one, K8 eight, bool large, cudaStream_t s, A... args) {
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = kTeamCtas;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(large ? kTeamCtas : 1);
  cfg.blockDim = dim3(kThreads);
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = large ? 2 : 1;
  return large ? cudaLaunchKernelEx(&cfg, eight, args...) : cudaLaunchKernelEx(&cfg, one, args...);
}

}  // namespace

cudaError_t pages_set_attributes() {
  return cudaFuncSetAttribute(copy_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)sizeof(CopySmem));
}

cudaError_t launch_page_fork(const ForkArgs& a, cudaStream_t s) {
  const bool large = (long long)a.n_fork * a.max_pages > kOneCtaEntries || a.n_free >= kOneCtaCopies;
  return launch_team(fork_kernel<1>, fork_kernel<kTeamCtas>, large, s, a);
}

cudaError_t launch_page_release(const ReleaseArgs& a, cudaStream_t s) {
  const bool large = (long long)a.n_seq * a.max_pages > kOneCtaEntries || a.n_free >= kOneCtaCopies;
  return launch_team(release_kernel<1>, release_kernel<kTeamCtas>, large, s, a);
}

cudaError_t launch_page_compact(const CompactArgs& a, cudaStream_t s) {
  const long long entries = (long long)a.n_seq * a.max_pages;
  const int remap = entries <= kRemapInside ? 1 : 0;
  const bool large = a.n_free > kOneCtaPages || (remap && entries > kOneCtaPages);
  const cudaError_t e = launch_team(compact_kernel<1>, compact_kernel<kTeamCtas>, large, s, a, remap);
  if (e != cudaSuccess || remap) return e;
  remap_kernel<<<(unsigned)((entries + kRemapEntries - 1) / kRemapEntries), kRemapThreads, 0, s>>>(a);
  return cudaGetLastError();
}

cudaError_t launch_page_copy(PageCopyArgs a, int sm_count, cudaStream_t s) {
  // pieces of 32 KiB when there is one for every other SM, else of 8 KiB, which more SMs share: 64 pieces of
  // 32 KiB take 2.7 us whole and 2.5 as quarters, 128 2.8 against 3.1, 256 3.5 against 4.2
  for (a.piece_bytes = kPieceBytes;; a.piece_bytes = kPieceBytes / 4) {
    a.pieces = 0;
    a.small = false;
    for (int j = 0; j < a.n_pools; ++j) {
      PageCopyArgs::Pool& p = a.pool[j];
      const size_t both = reinterpret_cast<size_t>(p.base) | (size_t)p.bytes;
      p.width = both % 16 == 0 ? 16 : both % 8 == 0 ? 8 : both % 4 == 0 ? 4 : both % 2 == 0 ? 2 : 1;
      p.first = a.pieces;
      p.pieces = p.width < 16 || p.bytes < kBulkLeast ? 0 : (int)((p.bytes + a.piece_bytes - 1) / a.piece_bytes);
      a.pieces += p.pieces;
      a.small |= p.pieces == 0;
    }
    if (a.piece_bytes < kPieceBytes || 2LL * a.n_copies * a.pieces >= sm_count) break;
  }
  const long long bulk = (long long)a.n_copies * a.pieces, small = a.small ? (a.n_copies + 6LL) / 7 : 0;
  const long long ctas = bulk > small ? bulk : small;
  cudaLaunchAttribute attr[1];
  const cudaLaunchConfig_t cfg = overlapped_launch((unsigned)(ctas < sm_count ? ctas : sm_count), kCopyThreads,
                                                   sizeof(CopySmem), s, attr);
  return cudaLaunchKernelEx(&cfg, copy_kernel, a);
}

}  // namespace ga

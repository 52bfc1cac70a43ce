// Pages of a batch's pools: branching requests (release, share, copy), pages for the next round,
// compaction.  include/treeverify.h gives the rules; here is how they run.
//
// The state is small and its steps depend on one another (who still holds a page decides which
// pages are free, that decides who gets which), so a call is a chain of round trips, and what it
// takes is latency.  It is planned by one CTA with the counts in shared memory, or, for pools and
// batches that are too large for that, by a cluster of eight on the arrays in global memory, with a
// cluster barrier between the steps; requests and pages are split over the CTAs in contiguous
// ranges, so that counts in range order give the order of requests and pages, and with it results
// that do not depend on timing.  The reference counts change by integer atomics only.  The plan
// leaves a list of copies in the workspace; a second kernel, its programmatic dependent, moves the
// rows.
#include <cooperative_groups.h>

#include "tv_common.cuh"

namespace tv {
namespace cg = cooperative_groups;

constexpr int kPlanRanks = 8;         // CTAs of a cluster plan
constexpr int kPlanThreads = 1024;
// A single CTA plans up to this many pages and steps (table entries; requests for a reserve).
constexpr int kOnePages = 8192, kOneSteps = 4096;
constexpr int kPlanWarps = kPlanThreads / 32;
constexpr int kCopyThreads = 256;
constexpr int kCopyUnroll = 8;
constexpr int kCopyChunk = kCopyThreads * kCopyUnroll * 16;   // bytes of one copy unit

// A page copy: the rows that `tokens` valid tokens fill, in all layers.
struct PageJob {
  int32_t src, dst, tokens, pad;
};

// What a request does in a fork.
enum { kKeep = 0, kRelease = 1, kTruncate = 2, kFork = 3 };

struct PageWorkspace {
  int32_t* n_jobs;     // [1] copies in jobs
  int32_t* rank_sum;   // [3 * kPlanRanks] per-CTA counts
  PageJob* jobs;       // [n_pool]
  int32_t* list;       // [n_pool] free pages, or holes
  int32_t* tokens;     // [n_pool] valid tokens of a page
  int32_t* holders;    // [n_pool] table entries that name a page
  int32_t* act;        // [B]
  int32_t* len;        // [B] new length
  int32_t* pages;      // [B] pages to allocate
  int32_t* from;       // [B] page the partial last page is copied from
};

static size_t page_workspace(const tv_shape* s, void* base, PageWorkspace* w) {
  const size_t n = (size_t)s->n_pool_pages, B = (size_t)s->B;
  char* p = (char*)base;
  size_t at = 0;
  auto take = [&](size_t bytes) {
    char* q = p + at;
    at += (bytes + 255) / 256 * 256;
    return q;
  };
  PageWorkspace x;
  x.n_jobs = (int32_t*)take(256);
  x.rank_sum = x.n_jobs + 16;
  x.jobs = (PageJob*)take(n * sizeof(PageJob));
  x.list = (int32_t*)take(n * 4);
  x.tokens = (int32_t*)take(n * 4);
  x.holders = (int32_t*)take(n * 4);
  x.act = (int32_t*)take(B * 4);
  x.len = (int32_t*)take(B * 4);
  x.pages = (int32_t*)take(B * 4);
  x.from = (int32_t*)take(B * 4);
  if (w) *w = x;
  return at;
}

struct PlanArgs {
  int B, max_pages, n_pool, page_tokens;
  int64_t raw_cap;
  int32_t* table;
  int32_t* refs;
  const int32_t* L;
  int32_t* status;
  PageWorkspace w;
};

__device__ __forceinline__ bool in_pool(const PlanArgs& a, int page) {
  return page >= 0 && page < a.n_pool;
}

// Contiguous share of [0, n) of a CTA.
struct Range {
  int lo, hi;
};
template <int kRanks>
__device__ __forceinline__ Range share_of(int n, int rank) {
  const int per = (n + kRanks - 1) / kRanks;
  const int lo = min(n, rank * per);
  return {lo, min(n, lo + per)};
}

template <int kRanks>
__device__ __forceinline__ int plan_rank() {
  return kRanks == 1 ? 0 : (int)cg::this_cluster().block_rank();
}
template <int kRanks>
__device__ __forceinline__ void plan_sync() {
  if constexpr (kRanks == 1)
    __syncthreads();
  else
    cg::this_cluster().sync();
}

// Index of a table entry: 32 bits where a single CTA plans (at most kOneSteps).
template <int kRanks>
struct EntryIndex {
  using type = int64_t;
};
template <>
struct EntryIndex<1> {
  using type = int32_t;
};

// The plan's arrays: a single CTA's in shared memory (n ints each, in order), a cluster's the
// global ones.
struct SharedInts {
  int32_t* next;
  template <int kRanks>
  __device__ __forceinline__ int32_t* take(int32_t* global, int n) {
    if constexpr (kRanks != 1) return global;
    int32_t* p = next;
    next += n;
    return p;
  }
};

// Exclusive prefix of v over the CTA's threads; *total: the sum.
__device__ __forceinline__ int block_prefix(int v, int* total) {
  __shared__ int s_warp[kPlanWarps];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  __syncthreads();   // the last call's readers are done
  if (lane == 31) s_warp[warp] = x;
  __syncthreads();
  // every warp scans the warps' sums
  const int c = lane < kPlanWarps ? s_warp[lane] : 0;
  int y = c;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int z = __shfl_up_sync(0xffffffffu, y, o);
    if (lane >= o) y += z;
  }
  *total = __shfl_sync(0xffffffffu, y, 31);
  return __shfl_sync(0xffffffffu, y - c, warp) + x - v;
}

// Sum of f(i) over the CTA's share r, by all its threads.
template <typename F>
__device__ __forceinline__ int block_count(Range r, F f) {
  int n = 0, total;
  for (int i = r.lo + threadIdx.x; i < r.hi; i += kPlanThreads) n += f(i);
  block_prefix(n, &total);
  return total;
}

// Calls g(i, position) for every i of the share with f(i) = n > 0, position being `start` plus the
// sum of f over the share before i.
template <typename F, typename G>
__device__ __forceinline__ void block_place(Range r, int start, F f, G g) {
  for (int i0 = r.lo; i0 < r.hi; i0 += kPlanThreads) {
    const int i = i0 + threadIdx.x;
    const int n = i < r.hi ? f(i) : 0;
    int total;
    const int at = start + block_prefix(n, &total);
    if (n > 0) g(i, at);
    start += total;
  }
}

// The sums of s0 and s1 over the CTAs before this one and over all of them (with several CTAs: left
// in the workspace, and a wait for the cluster).
struct Sums {
  int before[2], all[2];
};
template <int kRanks>
__device__ __forceinline__ Sums plan_sums(const PlanArgs& a, int rank, int s0, int s1) {
  if constexpr (kRanks == 1) return {{0, 0}, {s0, s1}};
  if (threadIdx.x == 0) {
    a.w.rank_sum[2 * rank] = s0;
    a.w.rank_sum[2 * rank + 1] = s1;
  }
  plan_sync<kRanks>();
  Sums s = {{0, 0}, {0, 0}};
  for (int q = 0; q < kRanks; ++q)
    for (int k = 0; k < 2; ++k) {
      const int c = a.w.rank_sum[2 * q + k];
      if (q < rank) s.before[k] += c;
      s.all[k] += c;
    }
  return s;
}

// Whether the call's requests can all have their pages; if so, the lowest free pages are listed in
// order (complete after the closing barrier).  `want`: pages that the CTA's requests need; *start:
// the list position of the CTA's first one; *total: all CTAs' together.
template <int kRanks>
__device__ __forceinline__ bool list_free_pages(const PlanArgs& a, int rank, const int32_t* refs,
                                                int32_t* list, int want, int* start, int* total) {
  const Range pages = share_of<kRanks>(a.n_pool, rank);
  auto is_free = [&](int p) { return refs[p] == 0 ? 1 : 0; };
  const Sums s = plan_sums<kRanks>(a, rank, want, block_count(pages, is_free));
  *start = s.before[0];
  *total = s.all[0];
  const bool ok = s.all[0] <= s.all[1];
  if (ok && s.before[1] < s.all[0])
    block_place(pages, s.before[1], is_free, [&](int p, int at) {
      if (at < s.all[0]) list[at] = p;
    });
  plan_sync<kRanks>();
  if (!ok && rank == 0 && threadIdx.x == 0) record_error(a.status, TV_ERR_CAPACITY);
  return ok;
}

// ---- fork: release, truncate, share ------------------------------------------------------------
// Shared memory of a single CTA: counts and free list of the pages, four numbers per request.
static size_t fork_smem(int n_pool, int B) { return ((size_t)2 * n_pool + (size_t)4 * B) * 4; }

template <int kRanks>
__global__ void __launch_bounds__(kPlanThreads)
    fork_plan_kernel(const PlanArgs a, int32_t* L, const int32_t* source,
                     const int32_t* keep) {
  pdl_wait();
  // the copy kernel waits for this grid before it reads the plan; its CTAs come early only where the
  // plan takes one SM: placed around a cluster plan they fill the SMs unevenly (compacting 1.3 GB
  // 430 us, 410 us without)
  if constexpr (kRanks == 1) pdl_launch_dependents();
  extern __shared__ __align__(16) int32_t smem_ints[];
  const int rank = plan_rank<kRanks>(), tid = threadIdx.x;
  const Range mine = share_of<kRanks>(a.B, rank);
  const int P = a.page_tokens, G = a.max_pages;
  SharedInts ints = {smem_ints};
  int32_t* refs = ints.take<kRanks>(a.refs, a.n_pool);
  int32_t* list = ints.take<kRanks>(a.w.list, a.n_pool);
  int32_t* act = ints.take<kRanks>(a.w.act, a.B);
  int32_t* new_len = ints.take<kRanks>(a.w.len, a.B);
  int32_t* pages = ints.take<kRanks>(a.w.pages, a.B);
  int32_t* from = ints.take<kRanks>(a.w.from, a.B);
  // f(request, position) over the table entries of the CTA's requests that change
  using Entry = typename EntryIndex<kRanks>::type;
  auto entries = [&](auto f) {
    const Entry hi = (Entry)mine.hi * G;
    for (Entry e = (Entry)mine.lo * G + tid; e < hi; e += kPlanThreads) {
      const int b = (int)(e / G);
      if (act[b] != kKeep) f(b, (int)(e - (Entry)b * G), e);
    }
  };

  // 1. what every request does and its new length
  if constexpr (kRanks == 1)
    for (int p = tid; p < a.n_pool; p += kPlanThreads) refs[p] = a.refs[p];
  for (int b = mine.lo + tid; b < mine.hi; b += kPlanThreads) {
    const int s = source[b];
    int what = kKeep, len = 0;
    if (s == -1) {
      what = kRelease;
    } else if (s < 0 || s >= a.B || source[s] != s) {
      record_error(a.status, TV_ERR_ARG);
    } else {
      const int Ls = L[s];
      len = Ls;
      if (keep) {
        const int ks = keep[s], kb = keep[b];
        if (ks >= 0) len = min(len, ks);
        if (kb >= 0) len = min(len, kb);
      }
      if (s != b || len < Ls) what = s != b ? kFork : kTruncate;
      if (what != kKeep && (Ls < 0 || Ls > a.raw_cap)) {
        record_error(a.status, TV_ERR_CAPACITY);
        what = kKeep;
      }
    }
    act[b] = what;
    new_len[b] = len;
    pages[b] = 0;   // here: whether a page is missing among the source's
  }
  __syncthreads();
  entries([&](int b, int g, Entry) {
    if (act[b] != kRelease && (int64_t)g * P < new_len[b] &&
        !in_pool(a, a.table[(int64_t)source[b] * G + g]))
      pages[b] = 1;
  });
  __syncthreads();
  for (int b = mine.lo + tid; b < mine.hi; b += kPlanThreads) {
    const int len = new_len[b];
    int need = 0, src = -1;
    if (pages[b]) {
      record_error(a.status, TV_ERR_ARG);
      act[b] = kKeep;
    } else if ((act[b] == kTruncate || act[b] == kFork) && len % P != 0) {
      // the partial last page: a fork gets a copy, a truncated request does if others hold it
      src = a.table[(int64_t)source[b] * G + len / P];
      need = act[b] == kFork || refs[src] > 1 ? 1 : 0;
    }
    pages[b] = need;
    from[b] = src;
  }
  plan_sync<kRanks>();

  // 2. the reference counts: entries that go, full pages that gain a holder (sign -1: undone)
  auto count = [&](int sign) {
    entries([&](int b, int g, Entry e) {
      const int len = new_len[b];
      if (act[b] != kTruncate || (int64_t)g * P >= len) {
        const int p = a.table[e];
        if (in_pool(a, p)) atomicAdd(&refs[p], -sign);
      }
      if (act[b] == kFork && g < len / P)
        atomicAdd(&refs[a.table[(int64_t)source[b] * G + g]], sign);
    });
  };
  count(1);
  plan_sync<kRanks>();

  // 3. new pages for the partial last pages, in the order of the requests
  auto pages_of = [&](int b) { return pages[b]; };
  int start, total;
  const bool ok = list_free_pages<kRanks>(a, rank, refs, list, block_count(mine, pages_of), &start,
                                          &total);
  if (rank == 0 && tid == 0) a.w.n_jobs[0] = ok ? total : 0;
  if (!ok) {   // nothing changes (a single CTA has only changed its own copy of the counts)
    if constexpr (kRanks != 1) count(-1);
    __syncthreads();
    for (int b = mine.lo + tid; b < mine.hi; b += kPlanThreads) a.w.act[b] = kKeep;
    return;
  }
  block_place(mine, start, pages_of, [&](int b, int at) {
    const int page = list[at], src = from[b];
    a.w.jobs[at] = {src, page, new_len[b] % P, 0};
    refs[page] = 1;
    if (act[b] == kTruncate) atomicAdd(&refs[src], -1);
    from[b] = page;
  });
  __syncthreads();   // the new pages of this CTA's requests are in from

  // 4. the table, the lengths, the counts.  A fork reads full pages of its source, which no other
  //    request writes: a source changes at most its last partial page and what lies behind it.
  entries([&](int b, int g, Entry e) {
    const int len = new_len[b], full = len / P;
    if (act[b] != kRelease && g < full) {
      if (act[b] == kFork) a.table[e] = a.table[(int64_t)source[b] * G + g];
    } else if (act[b] != kRelease && g == full && len % P != 0) {
      if (pages[b]) a.table[e] = from[b];
    } else {
      a.table[e] = -1;
    }
  });
  for (int b = mine.lo + tid; b < mine.hi; b += kPlanThreads) {
    if (act[b] != kKeep) L[b] = new_len[b];
    if constexpr (kRanks == 1) {   // for the copies of the indexer keys
      a.w.act[b] = act[b];
      a.w.len[b] = new_len[b];
    }
  }
  if constexpr (kRanks == 1)
    for (int p = tid; p < a.n_pool; p += kPlanThreads) a.refs[p] = refs[p];
}

// ---- reserve: the pages of the next tokens -------------------------------------------------------
static size_t reserve_smem(int n_pool, int B) { return ((size_t)2 * n_pool + (size_t)2 * B) * 4; }

// A round needs a page or two per request, which its thread looks at; a prompt's pages are looked at
// by the thread's warp.
constexpr int kShortWindow = 4;

template <int kRanks>
__global__ void __launch_bounds__(kPlanThreads)
    reserve_kernel(const PlanArgs a, const int32_t* need) {
  pdl_wait();
  extern __shared__ __align__(16) int32_t smem_ints[];
  const int rank = plan_rank<kRanks>(), tid = threadIdx.x, lane = tid & 31;
  const Range mine = share_of<kRanks>(a.B, rank);
  const int P = a.page_tokens, G = a.max_pages;
  SharedInts ints = {smem_ints};
  int32_t* refs = ints.take<kRanks>(a.refs, a.n_pool);
  int32_t* list = ints.take<kRanks>(a.w.list, a.n_pool);
  int32_t* pages = ints.take<kRanks>(a.w.pages, a.B);
  int32_t* first = ints.take<kRanks>(a.w.from, a.B);
  if constexpr (kRanks == 1)
    for (int p = tid; p < a.n_pool; p += kPlanThreads) refs[p] = a.refs[p];
  // f(request, first page, last page, whole warp) for the CTA's requests; a warp's lanes pass their own
  // windows (lo > hi: none), which are called one by one for the whole warp where they are long
  auto windows = [&](int b, int lo, int hi, auto f) {
    const bool is_long = hi - lo >= kShortWindow;
    if (lo <= hi && !is_long) f(b, lo, hi, false);
    for (unsigned m = __ballot_sync(0xffffffffu, is_long); m; m &= m - 1) {
      const int q = __ffs(m) - 1;
      f(__shfl_sync(0xffffffffu, b, q), __shfl_sync(0xffffffffu, lo, q),
        __shfl_sync(0xffffffffu, hi, q), true);
    }
  };
  // 1. unmapped pages of the positions L .. L + need - 1
  const int steps = (mine.hi - mine.lo + kPlanThreads - 1) / kPlanThreads;
  for (int k = 0; k < steps; ++k) {
    const int b = mine.lo + k * kPlanThreads + tid;
    int lo = 0, hi = -1;
    if (b < mine.hi) {
      const int n = need[b], L = a.L[b];
      if (n > 0) {
        if (L < 0) {
          record_error(a.status, TV_ERR_ARG);
        } else if ((int64_t)L + n > a.raw_cap) {
          record_error(a.status, TV_ERR_CAPACITY);
        } else {
          lo = L / P;
          hi = (L + n - 1) / P;
        }
      }
      pages[b] = 0;
    }
    windows(b, lo, hi, [&](int q, int g0, int g1, bool warp) {
      int missing = 0;
      for (int g = g0 + (warp ? lane : 0); g <= g1; g += warp ? 32 : 1) {
        const int p = a.table[(int64_t)q * G + g];
        if (p == -1)
          ++missing;
        else if (!in_pool(a, p))
          record_error(a.status, TV_ERR_ARG);
      }
      if (warp) missing = __reduce_add_sync(0xffffffffu, missing);
      if (b == q) pages[q] = missing;   // (the request's own thread)
    });
  }
  __syncthreads();
  // 2. the lowest free pages, in the order of requests and positions
  auto pages_of = [&](int b) { return pages[b]; };
  int start, total;
  if (!list_free_pages<kRanks>(a, rank, refs, list, block_count(mine, pages_of), &start, &total))
    return;
  if (total == 0) return;
  block_place(mine, start, pages_of, [&](int b, int at) { first[b] = at; });
  __syncthreads();
  for (int k = 0; k < steps; ++k) {
    const int b = mine.lo + k * kPlanThreads + tid;
    int lo = 0, hi = -1;
    if (b < mine.hi && pages[b] > 0) {
      const int L = a.L[b];
      lo = L / P;
      hi = (L + need[b] - 1) / P;
    }
    windows(b, lo, hi, [&](int q, int g0, int g1, bool warp) {
      int at = first[q];
      for (int g = g0; g <= g1; g += warp ? 32 : 1) {
        const int mine_g = warp ? g + lane : g;
        int32_t* e = &a.table[(int64_t)q * G + mine_g];
        const bool missing = mine_g <= g1 && *e == -1;
        const unsigned m = warp ? __ballot_sync(0xffffffffu, missing) : 0u;
        if (missing) {
          const int page = list[at + __popc(m & ((1u << lane) - 1u))];
          *e = page;
          a.refs[page] = 1;
        }
        at += warp ? __popc(m) : missing ? 1 : 0;
      }
    });
  }
}

// ---- compaction ----------------------------------------------------------------------------------
static size_t compact_smem(int n_pool, int) { return (size_t)5 * n_pool * 4; }

template <int kRanks>
__global__ void __launch_bounds__(kPlanThreads)
    compact_plan_kernel(const PlanArgs a, int32_t* remap_out, int32_t* n_live_out) {
  pdl_wait();
  if constexpr (kRanks == 1) pdl_launch_dependents();   // (see fork_plan_kernel)
  extern __shared__ __align__(16) int32_t smem_ints[];
  const int rank = plan_rank<kRanks>();
  const int tid = threadIdx.x, all = rank * kPlanThreads + tid;
  constexpr int kAll = kRanks * kPlanThreads;
  const Range mine = share_of<kRanks>(a.n_pool, rank);
  const int P = a.page_tokens, G = a.max_pages;
  using Entry = typename EntryIndex<kRanks>::type;
  const Entry entries = (Entry)a.B * G;
  SharedInts ints = {smem_ints};
  const int32_t* refs = a.refs;
  int32_t* tokens = ints.take<kRanks>(a.w.tokens, a.n_pool);
  int32_t* holders = ints.take<kRanks>(a.w.holders, a.n_pool);
  int32_t* list = ints.take<kRanks>(a.w.list, a.n_pool);
  int32_t* remap = ints.take<kRanks>(remap_out, a.n_pool);
  if constexpr (kRanks == 1) {
    int32_t* copy = ints.take<1>(nullptr, a.n_pool);
    for (int p = tid; p < a.n_pool; p += kPlanThreads) copy[p] = a.refs[p];
    refs = copy;
  }

  // 1. every page's holders in the table and the most tokens that one of them has in it
  for (int p = mine.lo + tid; p < mine.hi; p += kPlanThreads) tokens[p] = holders[p] = 0;
  plan_sync<kRanks>();
  for (Entry e = all; e < entries; e += kAll) {
    const int p = a.table[e];
    if (p == -1) continue;
    if (!in_pool(a, p)) {
      record_error(a.status, TV_ERR_ARG);
      continue;
    }
    const int b = (int)(e / G), g = (int)(e - (Entry)b * G);
    const int64_t left = (int64_t)a.L[b] - (int64_t)g * P;
    atomicMax(&tokens[p], (int)(left < 0 ? 0 : left > P ? P : left));
    atomicAdd(&holders[p], 1);
  }
  plan_sync<kRanks>();

  // 2. live pages in order; those at n_live and above take the holes below it, in order
  auto live = [&](int p) { return refs[p] > 0 || holders[p] > 0 ? 1 : 0; };
  const Sums s = plan_sums<kRanks>(a, rank, block_count(mine, live), 0);
  const int n_live = s.all[0];
  int low_live;   // live pages below n_live
  {
    int low = 0;
    for (int p = mine.lo + tid; p < min(mine.hi, n_live); p += kPlanThreads) low += live(p);
    block_prefix(low, &low_live);
    if constexpr (kRanks != 1) {
      int32_t* sums = a.w.rank_sum + 2 * kRanks;
      if (tid == 0) sums[rank] = low_live;
      plan_sync<kRanks>();
      low_live = 0;
      for (int q = 0; q < kRanks; ++q) low_live += sums[q];
    }
  }
  const int moves = n_live - low_live;
  int before = s.before[0];
  for (int p0 = mine.lo; p0 < mine.hi; p0 += kPlanThreads) {
    const int p = p0 + tid;
    const int is = p < mine.hi ? live(p) : 0;
    int total;
    const int at = before + block_prefix(is, &total);   // live pages before p
    before += total;
    if (p >= mine.hi) continue;
    if (refs[p] < holders[p]) record_error(a.status, TV_ERR_ARG);
    if (p < n_live) {
      remap[p] = is ? p : -1;
      if (!is) list[p - at] = p;
    } else if (is) {
      // a page that somebody besides the table holds moves whole
      a.w.jobs[at - low_live] = {p, -1, refs[p] > holders[p] ? P : tokens[p], 0};
    } else {
      remap[p] = -1;
    }
  }
  plan_sync<kRanks>();
  for (int i = all; i < moves; i += kAll) {
    const int src = a.w.jobs[i].src, dst = list[i];
    a.w.jobs[i].dst = dst;
    remap[src] = dst;
    a.refs[dst] = refs[src];
    a.refs[src] = 0;
  }
  if (all == 0) {
    n_live_out[0] = n_live;
    a.w.n_jobs[0] = moves;
  }
  plan_sync<kRanks>();

  // 3. the table follows
  for (Entry e = all; e < entries; e += kAll) {
    const int p = a.table[e];
    if (in_pool(a, p) && remap[p] != p) a.table[e] = remap[p];
  }
  if constexpr (kRanks == 1)
    for (int p = tid; p < a.n_pool; p += kPlanThreads) remap_out[p] = remap[p];
}

// ---- the copies ------------------------------------------------------------------------------------
struct CopyArgs {
  char* pool[6];         // rawK, rawV, c4K, c4V, c128K, c128V (nullptr: inactive)
  int64_t row_bytes;
  int page_tokens;
  int units[3];          // copy units of one page of a raw, C4, C128 pool
  const int32_t* n_jobs;
  const PageJob* jobs;
  // indexer keys of forked slots
  char* keys;            // nullptr: none
  int64_t key_row, key_slot;   // bytes of a row, of a slot
  int key_units, B;
  const int32_t* act;
  const int32_t* len;
  const int32_t* source;
};

// One unit: up to kCopyChunk bytes, every load of a thread in flight before its stores.
__device__ __forceinline__ void copy_unit(const char* src, char* dst, int64_t bytes) {
  const uint4* s = reinterpret_cast<const uint4*>(src);
  uint4* d = reinterpret_cast<uint4*>(dst);
  const int n = (int)((bytes < kCopyChunk ? bytes : kCopyChunk) / 16);
  uint4 v[kCopyUnroll];
#pragma unroll
  for (int u = 0; u < kCopyUnroll; ++u) {
    const int i = u * kCopyThreads + threadIdx.x;
    if (i < n) v[u] = s[i];
  }
#pragma unroll
  for (int u = 0; u < kCopyUnroll; ++u) {
    const int i = u * kCopyThreads + threadIdx.x;
    if (i < n) d[i] = v[u];
  }
}

__global__ void __launch_bounds__(kCopyThreads) page_copy_kernel(const CopyArgs a) {
  pdl_wait();
  const int per_page = 2 * (a.units[0] + a.units[1] + a.units[2]);
  const int64_t total = (int64_t)a.n_jobs[0] * per_page;
  for (int64_t t = blockIdx.x; t < total; t += gridDim.x) {
    const int64_t j = t / per_page;
    int u = (int)(t - j * per_page);
    const PageJob job = a.jobs[j];
    int layer = 0;
    while (u >= 2 * a.units[layer]) u -= 2 * a.units[layer++];
    const int kv = u >= a.units[layer] ? 1 : 0;
    u -= kv * a.units[layer];
    const int per_row = layer == 0 ? 1 : layer == 1 ? 4 : 128;   // tokens of a row
    const int64_t off = (int64_t)u * kCopyChunk;
    const int64_t left = (int64_t)(job.tokens / per_row) * a.row_bytes - off;
    if (left <= 0) continue;
    char* pool = a.pool[2 * layer + kv];
    const int64_t page = (int64_t)(a.page_tokens / per_row) * a.row_bytes;
    copy_unit(pool + job.src * page + off, pool + job.dst * page + off, left);
  }
  if (a.keys == nullptr) return;
  const int64_t keys = (int64_t)a.B * a.key_units;
  for (int64_t t = blockIdx.x; t < keys; t += gridDim.x) {
    const int b = (int)(t / a.key_units);
    if (a.act[b] != kFork) continue;
    const int64_t off = (t - (int64_t)b * a.key_units) * kCopyChunk;
    const int64_t left = (int64_t)(a.len[b] / 4) * a.key_row - off;
    if (left <= 0) continue;
    copy_unit(a.keys + a.source[b] * a.key_slot + off, a.keys + b * a.key_slot + off, left);
  }
}

static int launch_error(const char* fn, cudaError_t e) {
  cudaGetLastError();
  return tv_set_error(TV_ERR_CUDA, "%s: launch failed: %s", fn, cudaGetErrorString(e));
}

static PlanArgs plan_args(const tv_shape* s, const int32_t* L, int32_t* refs, void* workspace,
                          int32_t* status) {
  PlanArgs a;
  a.B = s->B;
  a.max_pages = s->max_pages;
  a.n_pool = s->n_pool_pages;
  a.page_tokens = s->page_tokens;
  a.raw_cap = s->raw_cap;
  a.table = const_cast<int32_t*>(s->page_table);
  a.refs = refs;
  a.L = L;
  a.status = status;
  page_workspace(s, workspace, &a.w);
  return a;
}

static int launch_copy(const char* fn, const tv_shape* s, const PlanArgs& p, void* const pools[6],
                       void* keys, int d_idx, const int32_t* source, cudaStream_t stream) {
  CopyArgs a = {};
  for (int i = 0; i < 6; ++i) a.pool[i] = (char*)pools[i];
  a.row_bytes = (int64_t)s->d * (s->dtype == TV_BF16 ? 2 : 4);
  a.page_tokens = s->page_tokens;
  const int per_row[3] = {1, 4, 128};
  for (int i = 0; i < 3; ++i) {
    const int64_t bytes = s->page_tokens / per_row[i] * a.row_bytes;
    a.units[i] = pools[2 * i] ? (int)((bytes + kCopyChunk - 1) / kCopyChunk) : 0;
  }
  a.n_jobs = p.w.n_jobs;
  a.jobs = p.w.jobs;
  a.B = s->B;
  if (keys) {
    a.keys = (char*)keys;
    a.key_row = (int64_t)d_idx * 2;
    a.key_slot = s->c4_cap * a.key_row;
    a.key_units = (int)((a.key_slot + kCopyChunk - 1) / kCopyChunk);
    a.act = p.w.act;
    a.len = p.w.len;
    a.source = source;
  }
  const cudaError_t e = launch_pdl(page_copy_kernel, dim3(152 * 2), dim3(kCopyThreads), 0, stream, a);
  return e == cudaSuccess ? tv_check_launch(fn) : launch_error(fn, e);
}

// Launches a plan: one CTA where the state is small, else the cluster.  Measured (us, one CTA and
// cluster; slots x pages per slot, pool): fork 64 x 9, 400: 6.8 and 11.3; 64 x 32, 2048: 9.0 and 11.0;
// 256 x 32, 4096: 18.2 and 11.8.  compact 64 x 32, 2048: 6.3 and 10.6; 256 x 32, 4096: 10.9 and 10.4.
// reserve 64 slots, 400 pages: 3.0 and 4.4; 1024 slots, 8192 pages: 3.9 and 4.5.
template <typename... KArgs, typename... Args>
static int launch_plan(const char* fn, const tv_shape* s, int64_t steps, void (*one)(KArgs...),
                       void (*cluster)(KArgs...), size_t (*smem_of)(int, int), cudaStream_t stream,
                       Args... args) {
  const bool single = s->n_pool_pages <= kOnePages && steps <= kOneSteps;
  const size_t smem = smem_of(s->n_pool_pages, s->B);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(single ? 1 : kPlanRanks);
  cfg.blockDim = dim3(kPlanThreads);
  cfg.dynamicSmemBytes = single ? smem : 0;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = kPlanRanks;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = single ? 1 : 2;
  cudaError_t e = cudaSuccess;
  if (single && smem > 48 * 1024)   // always the most that any call takes (a request has a step or
                                    // more): another host thread may be launching the same kernel
    e = cudaFuncSetAttribute(one, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             (int)smem_of(kOnePages, kOneSteps));
  if (e == cudaSuccess) e = cudaLaunchKernelEx(&cfg, single ? one : cluster, KArgs(args)...);
  return e == cudaSuccess ? tv_check_launch(fn) : launch_error(fn, e);
}

}  // namespace tv

size_t tv_pages_workspace(const tv_shape* s) { return tv::page_workspace(s, nullptr, nullptr); }

int tv_launch_fork(const tv_shape* s, const int32_t* source, const int32_t* keep, int32_t* L,
                   int32_t* refs, void* const pools[6], void* keys, int d_idx, void* workspace,
                   int32_t* status, cudaStream_t stream) {
  const char* fn = "tv_pages_fork";
  const tv::PlanArgs a = tv::plan_args(s, L, refs, workspace, status);
  if (int rc = tv::launch_plan(fn, s, (int64_t)s->B * s->max_pages, tv::fork_plan_kernel<1>,
                               tv::fork_plan_kernel<tv::kPlanRanks>, tv::fork_smem, stream, a, L, source, keep))
    return rc;
  return tv::launch_copy(fn, s, a, pools, keys, d_idx, source, stream);
}

int tv_launch_reserve(const tv_shape* s, const int32_t* need, const int32_t* L, int32_t* refs,
                      void* workspace, int32_t* status, cudaStream_t stream) {
  const tv::PlanArgs a = tv::plan_args(s, L, refs, workspace, status);
  return tv::launch_plan("tv_pages_reserve", s, s->B, tv::reserve_kernel<1>,
                         tv::reserve_kernel<tv::kPlanRanks>, tv::reserve_smem, stream, a, need);
}

int tv_launch_compact(const tv_shape* s, const int32_t* L, int32_t* refs, void* const pools[6],
                      int32_t* remap, int32_t* n_live, void* workspace, int32_t* status,
                      cudaStream_t stream) {
  const char* fn = "tv_pages_compact";
  const tv::PlanArgs a = tv::plan_args(s, L, refs, workspace, status);
  if (int rc = tv::launch_plan(fn, s, (int64_t)s->B * s->max_pages, tv::compact_plan_kernel<1>,
                               tv::compact_plan_kernel<tv::kPlanRanks>, tv::compact_smem, stream,
                               a, remap, n_live))
    return rc;
  return tv::launch_copy(fn, s, a, pools, nullptr, 0, nullptr, stream);
}

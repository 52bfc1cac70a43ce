// Pages of a batch's pools: branching requests (release, share, copy), pages for the next round,
// compaction.  include/treeverify.h gives the rules; here is how they run.
//
// The state is small and its steps depend on one another (who still holds a page decides which
// pages are free, that decides who gets which), so each call plans on one cluster of eight CTAs,
// with a cluster barrier between the steps; requests and pages are split over the CTAs in
// contiguous ranges, so that counts in range order give the order of requests and pages, and with
// it results that do not depend on timing.  The reference counts change by integer atomics only.
// The plan leaves a list of copies in the workspace; a second kernel, its programmatic dependent,
// moves the rows.
#include <cooperative_groups.h>

#include "tv_common.cuh"

namespace tv {
namespace cg = cooperative_groups;

constexpr int kPlanRanks = 8;
constexpr int kPlanThreads = 512;
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
__device__ __forceinline__ Range share_of(int n, int rank) {
  const int per = (n + kPlanRanks - 1) / kPlanRanks;
  const int lo = min(n, rank * per);
  return {lo, min(n, lo + per)};
}

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
  int before = 0, sum = 0;
#pragma unroll
  for (int w = 0; w < kPlanWarps; ++w) {
    const int c = s_warp[w];
    before += w < warp ? c : 0;
    sum += c;
  }
  *total = sum;
  return before + x - v;
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

// Leaves the CTA's sums in the workspace, waits for the cluster, and returns the sums over the
// CTAs before this one and over all of them.
struct Sums {
  int before[2], all[2];
};
__device__ __forceinline__ Sums cluster_sums(const PlanArgs& a, int rank, int s0, int s1) {
  if (threadIdx.x == 0) {
    a.w.rank_sum[2 * rank] = s0;
    a.w.rank_sum[2 * rank + 1] = s1;
  }
  cg::this_cluster().sync();
  Sums s = {{0, 0}, {0, 0}};
  for (int q = 0; q < kPlanRanks; ++q)
    for (int k = 0; k < 2; ++k) {
      const int c = a.w.rank_sum[2 * q + k];
      if (q < rank) s.before[k] += c;
      s.all[k] += c;
    }
  return s;
}

// Whether the call's requests can all have their pages; if so, the lowest free pages are listed in
// order (cluster-wide: the list is complete after the closing barrier).  `want`: pages that the
// CTA's requests need; *start: the list position of the CTA's first one.
__device__ __forceinline__ bool list_free_pages(const PlanArgs& a, int rank, int want, int* start) {
  const Range pages = share_of(a.n_pool, rank);
  auto is_free = [&](int p) { return a.refs[p] == 0 ? 1 : 0; };
  const Sums s = cluster_sums(a, rank, want, block_count(pages, is_free));
  *start = s.before[0];
  const int total = s.all[0];
  const bool ok = total <= s.all[1];
  if (ok && s.before[1] < total)
    block_place(pages, s.before[1], is_free, [&](int p, int at) {
      if (at < total) a.w.list[at] = p;
    });
  cg::this_cluster().sync();
  if (!ok && rank == 0 && threadIdx.x == 0) record_error(a.status, TV_ERR_CAPACITY);
  return ok;
}

// ---- fork: release, truncate, share ------------------------------------------------------------
__global__ void __cluster_dims__(kPlanRanks, 1, 1) __launch_bounds__(kPlanThreads)
    fork_plan_kernel(const PlanArgs a, int32_t* L, const int32_t* __restrict__ source,
                     const int32_t* __restrict__ keep) {
  pdl_launch_dependents();   // the copy kernel waits for this grid before it reads the plan
  const int rank = (int)cg::this_cluster().block_rank();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const Range mine = share_of(a.B, rank);
  const int P = a.page_tokens, G = a.max_pages;
  const PageWorkspace& w = a.w;

  // 1. what every request does, its new length, whether the source has the pages for it
  for (int b = mine.lo + warp; b < mine.hi; b += kPlanWarps) {
    const int s = source[b];
    int act = kKeep, len = 0, pages = 0, from = -1;
    if (s == -1) {
      act = kRelease;
    } else if (s < 0 || s >= a.B || source[s] != s) {
      if (lane == 0) record_error(a.status, TV_ERR_ARG);
    } else {
      const int Ls = L[s];
      len = Ls;
      if (keep) {
        const int ks = keep[s], kb = keep[b];
        if (ks >= 0) len = min(len, ks);
        if (kb >= 0) len = min(len, kb);
      }
      if (s != b || len < Ls) act = s != b ? kFork : kTruncate;
      if (act != kKeep) {
        bool ok = Ls >= 0 && Ls <= a.raw_cap;
        if (!ok && lane == 0) record_error(a.status, TV_ERR_CAPACITY);
        if (ok) {
          const int n = (len + P - 1) / P;
          bool mapped = true;
          for (int g = lane; g < n; g += 32) mapped &= in_pool(a, a.table[(int64_t)s * G + g]);
          ok = __all_sync(0xffffffffu, mapped);
          if (!ok && lane == 0) record_error(a.status, TV_ERR_ARG);
        }
        if (!ok) {
          act = kKeep;
        } else if (len % P != 0) {
          // the partial last page: a fork gets a copy, a truncated request does if others hold it
          from = a.table[(int64_t)s * G + len / P];
          pages = act == kFork || a.refs[from] > 1 ? 1 : 0;
        }
      }
    }
    if (lane == 0) {
      w.act[b] = act;
      w.len[b] = len;
      w.pages[b] = pages;
      w.from[b] = from;
    }
  }
  cg::this_cluster().sync();

  // 2. the reference counts: entries that go, full pages that gain a holder (sign -1: undone)
  auto count = [&](int sign) {
    for (int b = mine.lo + warp; b < mine.hi; b += kPlanWarps) {
      const int act = w.act[b];
      if (act == kKeep) continue;
      const int len = w.len[b], full = len / P, held = (len + P - 1) / P;
      const int s = source[b];
      for (int g = lane; g < G; g += 32) {
        if (act != kTruncate || g >= held) {
          const int p = a.table[(int64_t)b * G + g];
          if (in_pool(a, p)) atomicAdd(&a.refs[p], -sign);
        }
        if (act == kFork && g < full) atomicAdd(&a.refs[a.table[(int64_t)s * G + g]], sign);
      }
    }
  };
  count(1);
  cg::this_cluster().sync();

  // 3. new pages for the partial last pages, in the order of the requests
  auto pages_of = [&](int b) { return w.pages[b]; };
  int start;
  const bool ok = list_free_pages(a, rank, block_count(mine, pages_of), &start);
  if (!ok) {   // nothing changes
    if (rank == 0 && tid == 0) w.n_jobs[0] = 0;
    count(-1);
    __syncthreads();
    for (int b = mine.lo + tid; b < mine.hi; b += kPlanThreads) w.act[b] = kKeep;
    return;
  }
  block_place(mine, start, pages_of, [&](int b, int at) {
    const int page = w.list[at], src = w.from[b];
    w.jobs[at] = {src, page, w.len[b] % P, 0};
    a.refs[page] = 1;
    if (w.act[b] == kTruncate) atomicAdd(&a.refs[src], -1);
    w.from[b] = page;
  });
  __syncthreads();   // the new pages of this CTA's requests are in w.from

  // 4. the table and the lengths.  A fork reads full pages of its source, which no other request
  //    writes: a source changes at most its last partial page and what lies behind it.
  for (int b = mine.lo + warp; b < mine.hi; b += kPlanWarps) {
    const int act = w.act[b];
    if (act == kKeep) continue;
    const int len = w.len[b], full = len / P, tail = len % P != 0 ? full : -1;
    const int s = source[b], pages = w.pages[b], page = w.from[b];
    for (int g = lane; g < G; g += 32) {
      int32_t* e = &a.table[(int64_t)b * G + g];
      if (act == kRelease)
        *e = -1;
      else if (g < full) {
        if (act == kFork) *e = a.table[(int64_t)s * G + g];
      } else if (g == tail) {
        if (pages) *e = page;
      } else {
        *e = -1;
      }
    }
    if (lane == 0) L[b] = len;
  }
  // the number of copies: the last CTA's list position after its own
  int total;
  {
    int n = 0;
    for (int b = mine.lo + tid; b < mine.hi; b += kPlanThreads) n += w.pages[b];
    block_prefix(n, &total);
  }
  if (rank == kPlanRanks - 1 && tid == 0) w.n_jobs[0] = start + total;
}

// ---- reserve: the pages of the next tokens -------------------------------------------------------
__global__ void __cluster_dims__(kPlanRanks, 1, 1) __launch_bounds__(kPlanThreads)
    reserve_kernel(const PlanArgs a, const int32_t* __restrict__ need) {
  const int rank = (int)cg::this_cluster().block_rank();
  const Range mine = share_of(a.B, rank);
  const int P = a.page_tokens, G = a.max_pages;
  // unmapped pages of the positions L .. L + need - 1
  for (int b = mine.lo + threadIdx.x; b < mine.hi; b += kPlanThreads) {
    const int n = need[b], L = a.L[b];
    int pages = 0;
    if (n > 0) {
      if (L < 0) {
        record_error(a.status, TV_ERR_ARG);
      } else if ((int64_t)L + n > a.raw_cap) {
        record_error(a.status, TV_ERR_CAPACITY);
      } else {
        for (int g = L / P; g <= (L + n - 1) / P; ++g) {
          const int p = a.table[(int64_t)b * G + g];
          if (p == -1)
            ++pages;
          else if (!in_pool(a, p))
            record_error(a.status, TV_ERR_ARG);
        }
      }
    }
    a.w.pages[b] = pages;
  }
  __syncthreads();
  auto pages_of = [&](int b) { return a.w.pages[b]; };
  int start;
  if (!list_free_pages(a, rank, block_count(mine, pages_of), &start)) return;
  block_place(mine, start, pages_of, [&](int b, int at) {
    const int L = a.L[b], n = need[b];
    for (int g = L / P; g <= (L + n - 1) / P; ++g) {
      int32_t* e = &a.table[(int64_t)b * G + g];
      if (*e != -1) continue;
      const int page = a.w.list[at++];
      *e = page;
      a.refs[page] = 1;
    }
  });
}

// ---- compaction ----------------------------------------------------------------------------------
__global__ void __cluster_dims__(kPlanRanks, 1, 1) __launch_bounds__(kPlanThreads)
    compact_plan_kernel(const PlanArgs a, int32_t* __restrict__ remap,
                        int32_t* __restrict__ n_live_out) {
  pdl_launch_dependents();
  auto cluster = cg::this_cluster();
  const int rank = (int)cluster.block_rank();
  const int tid = threadIdx.x, all = rank * kPlanThreads + tid;
  constexpr int kAll = kPlanRanks * kPlanThreads;
  const Range mine = share_of(a.n_pool, rank);
  const int P = a.page_tokens, G = a.max_pages;
  const int64_t entries = (int64_t)a.B * G;
  const PageWorkspace& w = a.w;

  // 1. every page's holders in the table and the most tokens that one of them has in it
  for (int p = mine.lo + tid; p < mine.hi; p += kPlanThreads) w.tokens[p] = w.holders[p] = 0;
  cluster.sync();
  for (int64_t e = all; e < entries; e += kAll) {
    const int p = a.table[e];
    if (p == -1) continue;
    if (!in_pool(a, p)) {
      record_error(a.status, TV_ERR_ARG);
      continue;
    }
    const int b = (int)(e / G), g = (int)(e - (int64_t)b * G);
    const int64_t left = (int64_t)a.L[b] - (int64_t)g * P;
    atomicMax(&w.tokens[p], (int)(left < 0 ? 0 : left > P ? P : left));
    atomicAdd(&w.holders[p], 1);
  }
  cluster.sync();

  // 2. live pages in order; those at n_live and above take the holes below it, in order
  auto live = [&](int p) { return a.refs[p] > 0 || w.holders[p] > 0 ? 1 : 0; };
  const Sums s = cluster_sums(a, rank, block_count(mine, live), 0);
  const int n_live = s.all[0];
  // live pages below n_live: complete in the shares before the one that holds n_live
  int before = s.before[0];
  {
    int low = 0, total;
    for (int p = mine.lo + tid; p < min(mine.hi, n_live); p += kPlanThreads) low += live(p);
    block_prefix(low, &total);
    if (tid == 0) w.rank_sum[2 * kPlanRanks + rank] = total;
  }
  cluster.sync();
  int low_live = 0;
  for (int q = 0; q < kPlanRanks; ++q) low_live += w.rank_sum[2 * kPlanRanks + q];
  const int moves = n_live - low_live;
  for (int p0 = mine.lo; p0 < mine.hi; p0 += kPlanThreads) {
    const int p = p0 + tid;
    const int is = p < mine.hi ? live(p) : 0;
    int total;
    const int at = before + block_prefix(is, &total);   // live pages before p
    before += total;
    if (p >= mine.hi) continue;
    const int refs = a.refs[p];
    if (refs < w.holders[p]) record_error(a.status, TV_ERR_ARG);
    if (p < n_live) {
      remap[p] = is ? p : -1;
      if (!is) w.list[p - at] = p;
    } else if (is) {
      // a page that somebody besides the table holds moves whole
      w.jobs[at - low_live] = {p, -1, refs > w.holders[p] ? P : w.tokens[p], 0};
    } else {
      remap[p] = -1;
    }
  }
  cluster.sync();
  for (int i = all; i < moves; i += kAll) {
    const int src = w.jobs[i].src, dst = w.list[i];
    w.jobs[i].dst = dst;
    remap[src] = dst;
    a.refs[dst] = a.refs[src];
    a.refs[src] = 0;
  }
  if (all == 0) {
    n_live_out[0] = n_live;
    w.n_jobs[0] = moves;
  }
  cluster.sync();

  // 3. the table follows
  for (int64_t e = all; e < entries; e += kAll) {
    const int p = a.table[e];
    if (in_pool(a, p)) a.table[e] = remap[p];
  }
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
  const cudaError_t e = launch_pdl(page_copy_kernel, dim3(152 * 4), dim3(kCopyThreads), 0, stream, a);
  return e == cudaSuccess ? tv_check_launch(fn) : launch_error(fn, e);
}

}  // namespace tv

size_t tv_pages_workspace(const tv_shape* s) { return tv::page_workspace(s, nullptr, nullptr); }

int tv_launch_fork(const tv_shape* s, const int32_t* source, const int32_t* keep, int32_t* L,
                   int32_t* refs, void* const pools[6], void* keys, int d_idx, void* workspace,
                   int32_t* status, cudaStream_t stream) {
  const char* fn = "tv_pages_fork";
  const tv::PlanArgs a = tv::plan_args(s, L, refs, workspace, status);
  tv::fork_plan_kernel<<<tv::kPlanRanks, tv::kPlanThreads, 0, stream>>>(a, L, source, keep);
  if (int rc = tv_check_launch(fn)) return rc;
  return tv::launch_copy(fn, s, a, pools, keys, d_idx, source, stream);
}

int tv_launch_reserve(const tv_shape* s, const int32_t* need, const int32_t* L, int32_t* refs,
                      void* workspace, int32_t* status, cudaStream_t stream) {
  const tv::PlanArgs a = tv::plan_args(s, L, refs, workspace, status);
  tv::reserve_kernel<<<tv::kPlanRanks, tv::kPlanThreads, 0, stream>>>(a, need);
  return tv_check_launch("tv_pages_reserve");
}

int tv_launch_compact(const tv_shape* s, const int32_t* L, int32_t* refs, void* const pools[6],
                      int32_t* remap, int32_t* n_live, void* workspace, int32_t* status,
                      cudaStream_t stream) {
  const char* fn = "tv_pages_compact";
  const tv::PlanArgs a = tv::plan_args(s, L, refs, workspace, status);
  tv::compact_plan_kernel<<<tv::kPlanRanks, tv::kPlanThreads, 0, stream>>>(a, remap, n_live);
  if (int rc = tv_check_launch(fn)) return rc;
  return tv::launch_copy(fn, s, a, pools, nullptr, 0, nullptr, stream);
}

// From logits to the integers and log probabilities a tree round works with: per (request, node)
// row the log-sum-exp, the entropy, the target token, the best alternatives, and the log
// probabilities of given tokens (a draft tree's tokens under their parents).
//
// With m = max x, d_i = x_i - m, S = sum e^{scale d_i} and T = sum d_i e^{scale d_i}:
//   lse = scale m + ln S,  entropy = ln S - scale T / S,  log p_i = scale d_i - ln S.
// The row is read once.  A thread keeps its own running (m, S, T) and rescales when its maximum
// grows; the partial triples are joined over the CTA, and over the CTAs of a cluster that share a
// row when there are few rows.
//
// The alternatives.  K distinct threads whose largest logits are >= t show that the K-th largest
// logit is >= t, so a logit below t is no alternative.  In the pass a thread only notes its largest
// logit, the tile that holds it, and the largest of its other tiles; at the end t is taken from
// the threads' largest logits, the few threads at or above t look at that one tile again, and where
// a second tile reaches t a warp looks at all of the thread's vectors.  The logits found, little
// more than K, are ranked by counting: a key's place is the number of larger keys (a key is the
// logit's order, then the lower id, so keys differ).  Rows of so many equal logits that the list
// overflows take one scan per alternative instead.
#include <cooperative_groups.h>
#include <float.h>

#include "tv_common.cuh"
#include "tv_sm100.cuh"

namespace tv {
namespace cg = cooperative_groups;
using sm100::add_f32x2;
using sm100::fma_f32x2;
using sm100::pack_f32x2;
using sm100::unpack_f32x2;

constexpr int kLpThreads = 128;
constexpr int kLpWarps = kLpThreads / 32;
constexpr int kLpUnroll = 4;                        // 16-byte vectors per thread and tile
constexpr int kLpTile = kLpThreads * kLpUnroll;     // vectors per tile
constexpr int kLpStages = 4;                        // tiles in flight
constexpr int kLpMaxTop = 32;
constexpr int kLpCand = 1024;                       // candidate list
constexpr int kLpMaxRanks = 16;
constexpr float kLog2e = 1.4426950408889634f;

struct LogprobArgs {
  int D, vocab, n_tok, n_top;
  int64_t ld;
  float scale;
  const int32_t* tokens;
  const int32_t* nodes;
  float* lse;
  float* entropy;
  float* logprobs;
  int32_t* top_ids;
  float* top_logprobs;
  int32_t* target;
  int32_t* status;
};

// Partial sums of a set of logits: their maximum (-inf: none above -inf yet), and S and T relative
// to it.  A NaN or +inf logit makes S NaN.
struct Partial {
  float m, s, t;
};

// Exponent scale, and the difference below which e^{scale d} is taken as 0 (2^-256; it also keeps
// -inf out of the products d e^{scale d}).
struct ExpScale {
  float c, dmin;
};

__device__ __forceinline__ float exp2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float max_nan(float a, float b) {   // NaN if either is
  float y;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(a), "f"(b));
  return y;
}
__device__ __forceinline__ uint64_t mul_f32x2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}

// p relative to a maximum m >= p.m
__device__ __forceinline__ void rebase(Partial& p, float m, ExpScale k) {
  if (m > p.m) {
    const float d = fmaxf(p.m - m, k.dmin);
    const float f = exp2_approx(d * k.c);
    p.t = (p.t + d * p.s) * f;
    p.s *= f;
    p.m = m;
  }
}

__device__ __forceinline__ Partial join(Partial a, Partial b, ExpScale k) {
  const float m = fmaxf(a.m, b.m);
  rebase(a, m, k);
  rebase(b, m, k);
  return {m, a.s + b.s, a.t + b.t};
}

// Order of a logit as an unsigned number; equal logits (and -0, +0) give equal numbers.
__device__ __forceinline__ uint32_t order_of(float x) {
  const uint32_t u = __float_as_uint(x + 0.f);
  return u ^ ((u >> 31) ? 0xffffffffu : 0x80000000u);
}
__device__ __forceinline__ float logit_of_order(uint32_t o) {
  return __uint_as_float(o ^ ((o >> 31) ? 0x80000000u : 0xffffffffu));
}
constexpr uint32_t kOrderLowest = 0x00800000u;   // order_of(-FLT_MAX), one above -inf's

// Selection key: larger logits first, then lower ids.  0: not a candidate (-inf or NaN).
__device__ __forceinline__ uint64_t key_of(float x, int id) {
  return x > -INFINITY ? ((uint64_t)order_of(x) << 32) | (uint32_t)~id : 0ull;
}

// A row as 16-byte vectors: vector i holds the elements i * kVec - skew + (0 .. kVec-1).  Rows
// may start at any element; only the first and the last vector can reach past the row.
template <typename T>
struct Row {
  static constexpr int kVec = 16 / sizeof(T);
  const T* p;
  int vocab, skew, n_vec;
  __device__ Row(const T* row, int v) : p(row), vocab(v) {
    skew = (int)(((uintptr_t)row & 15u) / sizeof(T));
    n_vec = (skew + v + kVec - 1) / kVec;
  }
  __device__ __forceinline__ int id(int i, int j) const { return i * kVec - skew + j; }
  __device__ __forceinline__ uint4 whole(int i) const {
    return *reinterpret_cast<const uint4*>(p + (i * kVec - skew));
  }
  // -inf where the vector reaches past the row or `hi`
  __device__ __forceinline__ uint4 edge(int i, int hi) const {
    const int e0 = i * kVec - skew;
    if (i < hi && e0 >= 0 && e0 + kVec <= vocab) return whole(i);
    uint32_t u[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      if constexpr (sizeof(T) == 2) {
        const int e = e0 + 2 * q;
        const uint32_t lo = i < hi && e >= 0 && e < vocab ? bits(e) : 0xff80u;
        const uint32_t up = i < hi && e + 1 >= 0 && e + 1 < vocab ? bits(e + 1) : 0xff80u;
        u[q] = lo | up << 16;
      } else {
        const int e = e0 + q;
        u[q] = i < hi && e >= 0 && e < vocab ? bits(e) : 0xff800000u;
      }
    }
    return make_uint4(u[0], u[1], u[2], u[3]);
  }
  __device__ __forceinline__ uint32_t bits(int e) const {
    if constexpr (sizeof(T) == 2)
      return reinterpret_cast<const uint16_t*>(p)[e];
    else
      return reinterpret_cast<const uint32_t*>(p)[e];
  }
  __device__ static __forceinline__ void unpack(const uint4& w, float (&x)[kVec]) {
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if constexpr (sizeof(T) == 2) {
        x[2 * j] = __uint_as_float(u[j] << 16);
        x[2 * j + 1] = __uint_as_float(u[j] & 0xffff0000u);
      } else {
        x[j] = __uint_as_float(u[j]);
      }
    }
  }
  // largest value (NaN ignored)
  __device__ static __forceinline__ float largest(const uint4& w) {
    if constexpr (sizeof(T) == 2) {
      auto h = [](uint32_t u) { return *reinterpret_cast<const __nv_bfloat162*>(&u); };
      const __nv_bfloat162 m = __hmax2(__hmax2(h(w.x), h(w.y)), __hmax2(h(w.z), h(w.w)));
      return fmaxf(__low2float(m), __high2float(m));
    } else {
      return fmaxf(fmaxf(__uint_as_float(w.x), __uint_as_float(w.y)),
                   fmaxf(__uint_as_float(w.z), __uint_as_float(w.w)));
    }
  }
};

__device__ __forceinline__ uint64_t max_u64(uint64_t a, uint64_t b) { return a > b ? a : b; }

// Shared memory of one CTA.  Of rank 0's, the other CTAs of the cluster write part and peer.
struct LpShared {
  uint4 ring[kLpStages][kLpUnroll][kLpThreads];   // tiles in flight; a thread reads only its own
  Partial warp_part[kLpWarps];
  Partial part[kLpMaxRanks];       // the CTAs' shares of the row
  uint64_t top[kLpMaxTop];         // largest keys, descending (0: none)
  uint32_t bound[kLpWarps][2];
  int count, columns;
  uint64_t scan[kLpWarps];
  uint64_t cand[kLpCand];
  uint64_t peer[kLpMaxRanks * kLpMaxTop];   // the CTAs' top lists
  uint64_t peer_bound;
  uint8_t column[kLpThreads];      // threads with more than one tile to look at again
};
static_assert(kLpMaxRanks * kLpMaxTop <= kLpCand, "every CTA's keys fit into cand");

// Lower bound (as an order) of the K-th largest logit that the CTA has seen, from the threads'
// largest ones m: either K threads of one warp are at or above it, or ceil(K / warps) of every
// warp.  The order of the lowest finite value where there are fewer.
__device__ __forceinline__ uint32_t kth_bound(LpShared& sm, float m, int K) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int r = (K + kLpWarps - 1) / kLpWarps;
  uint32_t o = order_of(m);
  uint32_t kth = 0u, rth = 0u;
  const int rounds = K <= kLpWarps ? K : r;
#pragma unroll 1
  for (int i = 1; i <= rounds; ++i) {
    const uint32_t w = __reduce_max_sync(0xffffffffu, o);
    if (i == r) rth = w;
    if (i == K) kth = w;
    const uint32_t at = __ballot_sync(0xffffffffu, o == w);
    if (lane == __ffs(at) - 1) o = 0u;
  }
  if (lane == 0) {
    sm.bound[warp][0] = kth;
    sm.bound[warp][1] = rth;
  }
  __syncthreads();
  uint32_t one = 0u, every = 0xffffffffu;
#pragma unroll
  for (int w = 0; w < kLpWarps; ++w) {
    one = max(one, sm.bound[w][0]);
    every = min(every, sm.bound[w][1]);
  }
  uint32_t t = max(one, every);
  if (t < kOrderLowest && K > kLpWarps) {
    // some warp has too few logits (a short or masked row): the K-th of one warp after all
    o = order_of(m);
#pragma unroll 1
    for (int i = 1; i < K; ++i) {
      const uint32_t w = __reduce_max_sync(0xffffffffu, o);
      if (w < kOrderLowest) break;
      const uint32_t at = __ballot_sync(0xffffffffu, o == w);
      if (lane == __ffs(at) - 1) o = 0u;
    }
    o = __reduce_max_sync(0xffffffffu, o);
    __syncthreads();
    if (lane == 0) sm.bound[warp][0] = o;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kLpWarps; ++w) t = max(t, sm.bound[w][0]);
  }
  return max(t, kOrderLowest);
}

// Appends the logits of vector i that are >= bound to the candidate list.
template <typename T>
__device__ __forceinline__ void list_vector(LpShared& sm, const Row<T>& row, int i, int hi,
                                            float bound) {
  const uint4 q = row.edge(i, hi);
  if (Row<T>::largest(q) < bound) return;
  float x[Row<T>::kVec];
  Row<T>::unpack(q, x);
#pragma unroll
  for (int j = 0; j < Row<T>::kVec; ++j)
    if (x[j] >= bound) {
      const int at = atomicAdd(&sm.count, 1);
      if (at < kLpCand) sm.cand[at] = key_of(x[j], row.id(i, j));
    }
}

// The CTA's K largest keys by one scan of its vectors [lo, hi) per key, into sm.top.
template <typename T>
__device__ __noinline__ void scan_top(LpShared& sm, const Row<T>& row, int lo, int hi, int K) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  uint64_t last = ~0ull;
  for (int k = 0; k < K; ++k) {
    uint64_t best = 0ull;
    for (int i = lo + threadIdx.x; i < hi; i += kLpThreads) {
      float x[Row<T>::kVec];
      Row<T>::unpack(row.edge(i, hi), x);
#pragma unroll
      for (int j = 0; j < Row<T>::kVec; ++j) {
        const uint64_t key = key_of(x[j], row.id(i, j));
        if (key < last) best = max_u64(best, key);
      }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) best = max_u64(best, __shfl_xor_sync(0xffffffffu, best, o));
    __syncthreads();
    if (lane == 0) sm.scan[warp] = best;
    __syncthreads();
    for (int w = 0; w < kLpWarps; ++w) best = max_u64(best, sm.scan[w]);
    if (threadIdx.x == 0) sm.top[k] = best;
    last = best;
  }
}

// Places of the n keys of `list` among each other: out[place] = key for the places below K.
__device__ __noinline__ void rank_keys(const uint64_t* list, int n, int K, uint64_t* out) {
  for (int i = threadIdx.x; i < n; i += kLpThreads) {
    const uint64_t key = list[i];
    int place = 0;
#pragma unroll 8
    for (int j = 0; j < n; ++j) place += list[j] > key ? 1 : 0;
    if (place < K) out[place] = key;
  }
}

__device__ __forceinline__ void cp_async_16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}

// Joins the partials held by the lanes of a warp (every lane gets the result).
template <int kLanes>
__device__ __forceinline__ Partial warp_join(Partial p, ExpScale k) {
  const uint32_t top = __reduce_max_sync(0xffffffffu, order_of(p.m));
  rebase(p, logit_of_order(top), k);
#pragma unroll
  for (int o = kLanes / 2; o > 0; o >>= 1) {
    p.s += __shfl_xor_sync(0xffffffffu, p.s, o);
    p.t += __shfl_xor_sync(0xffffffffu, p.t, o);
  }
  return p;
}

template <typename T, bool kCluster>
__global__ void __launch_bounds__(kLpThreads) logprobs_kernel(const T* __restrict__ logits,
                                                              const LogprobArgs a, int ranks) {
  extern __shared__ __align__(16) unsigned char smem_raw[];
  LpShared& sm = *reinterpret_cast<LpShared*>(smem_raw);
  const int rank = kCluster ? (int)cg::this_cluster().block_rank() : 0;
  const int64_t r = kCluster ? blockIdx.x / ranks : blockIdx.x;
  const int b = (int)(r / a.D), v = (int)(r - (int64_t)b * a.D);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const Row<T> row(logits + r * a.ld, a.vocab);
  constexpr int kVec = Row<T>::kVec;
  const ExpScale ks = {a.scale * kLog2e, -256.f / (a.scale * kLog2e)};
  const int K = a.n_top > 1 ? a.n_top : 1;
  // the CTA's vectors
  const int per = kCluster ? (row.n_vec + ranks - 1) / ranks : row.n_vec;
  const int lo = min(row.n_vec, rank * per), hi = min(row.n_vec, lo + per);

  // a tile's copies: whole vectors asynchronously, the row's ends and what lies past hi at once
  const T* src = row.p + ((lo + tid) * kVec - row.skew);
  const uint32_t ring = sm100::smem_u32(&sm.ring[0][0][tid]);
  constexpr uint32_t kStageBytes = sizeof(sm.ring[0]);
  const int inner_hi = min(hi, row.n_vec - 1);
  auto fetch = [&](int t) {
    const int i0 = lo + t * kLpTile;
    const uint32_t slot = ring + t % kLpStages * kStageBytes;
    const T* at = src + (int64_t)t * (kLpTile * kVec);
    if (i0 > 0 && i0 + kLpTile <= inner_hi) {
#pragma unroll
      for (int u = 0; u < kLpUnroll; ++u)
        cp_async_16(slot + u * kLpThreads * 16, at + u * kLpThreads * kVec);
    } else {
#pragma unroll 1
      for (int u = 0; u < kLpUnroll; ++u) {
        const int i = i0 + u * kLpThreads + tid;
        if (i > 0 && i < inner_hi)
          cp_async_16(slot + u * kLpThreads * 16, at + u * kLpThreads * kVec);
        else
          sm.ring[t % kLpStages][u][tid] = row.edge(i, hi);
      }
    }
  };
  const int tiles = (hi - lo + kLpTile - 1) / kLpTile;
#pragma unroll 1
  for (int t = 0; t < kLpStages - 1; ++t) {
    if (t < tiles) fetch(t);
    asm volatile("cp.async.commit_group;" ::: "memory");
  }
  if constexpr (kCluster) asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
  // the first given tokens of this row, so that their logits arrive under the others
  const bool first = rank == 0 && tid < a.n_tok;
  int given_node = -1, given_tok = -1;
  float given = 0.f;
  if (first) {
    const int64_t at = (int64_t)b * a.n_tok + tid;
    given_node = a.nodes ? a.nodes[at] : tid;
    given_tok = a.tokens[at];
    if (given_node == v && given_tok >= 0 && given_tok < a.vocab) given = load_f(row.p + given_tok);
  }
  if (tid == 0) sm.count = sm.columns = 0;
  if (tid < K) sm.top[tid] = 0ull;

  Partial p = {-INFINITY, 0.f, 0.f};
  float second = -INFINITY;   // largest logit outside the tile of the largest
  int at_tile = 0;
#pragma unroll 1
  for (int t = 0; t < tiles; ++t) {
    if (t + kLpStages - 1 < tiles) fetch(t + kLpStages - 1);
    asm volatile("cp.async.commit_group;" ::: "memory");
    asm volatile("cp.async.wait_group %0;" ::"n"(kLpStages - 1) : "memory");
    const uint4(*tile)[kLpThreads] = sm.ring[t % kLpStages];
    uint4 w[kLpUnroll];
    float m = -INFINITY;
#pragma unroll
    for (int u = 0; u < kLpUnroll; ++u) {
      w[u] = tile[u][tid];
      m = fmaxf(m, Row<T>::largest(w[u]));
    }
    if (m > p.m) {
      second = p.m;
      at_tile = t;
      rebase(p, m, ks);
    } else {
      second = fmaxf(second, m);
    }
    const float base = p.m == -INFINITY ? 0.f : p.m;
    const uint64_t neg = pack_f32x2(-base, -base), c2 = pack_f32x2(ks.c, ks.c);
    uint64_t s2 = pack_f32x2(0.f, 0.f), t2 = s2;
#pragma unroll
    for (int u = 0; u < kLpUnroll; ++u) {
      float x[kVec];
      Row<T>::unpack(w[u], x);
#pragma unroll
      for (int j = 0; j < kVec; j += 2) {
        const uint64_t d = add_f32x2(pack_f32x2(x[j], x[j + 1]), neg);
        float y0, y1;
        unpack_f32x2(mul_f32x2(d, c2), y0, y1);
        const uint64_t e = pack_f32x2(exp2_approx(y0), exp2_approx(y1));
        s2 = add_f32x2(s2, e);
        t2 = fma_f32x2(d, e, t2);
      }
    }
    float s0, s1, t0, t1;
    unpack_f32x2(s2, s0, s1);
    unpack_f32x2(t2, t0, t1);
    p.s += s0 + s1;
    float dt = t0 + t1;
    if (!(dt == dt)) {   // a masked logit: -inf times 0; the differences are bounded below instead
      dt = 0.f;
#pragma unroll 1
      for (int u = 0; u < kLpUnroll; ++u) {
        float x[kVec];
        Row<T>::unpack(tile[u][tid], x);
#pragma unroll
        for (int j = 0; j < kVec; ++j) {
          const float d = max_nan(x[j] - base, ks.dmin);
          dt += d * exp2_approx(d * ks.c);
        }
      }
    }
    p.t += dt;
  }
  // the CTA's sums
  const float largest = p.m;
  p = warp_join<32>(p, ks);
  if (lane == 0) sm.warp_part[warp] = p;
  const float bound = logit_of_order(kth_bound(sm, largest, K));   // (its barrier: warp_part)
  p = warp_join<kLpWarps>(sm.warp_part[lane % kLpWarps], ks);
  if (second >= bound) {
    sm.column[atomicAdd(&sm.columns, 1)] = (uint8_t)tid;
  } else if (largest >= bound) {
#pragma unroll 1
    for (int u = 0; u < kLpUnroll; ++u)
      list_vector(sm, row, lo + at_tile * kLpTile + u * kLpThreads + tid, hi, bound);
  }
  __syncthreads();
  const int columns = sm.columns;
#pragma unroll 1
  for (int k = warp; k < columns; k += kLpWarps) {
    if (*(volatile int*)&sm.count > kLpCand) break;   // too many equal logits
    for (int i = lo + sm.column[k] + lane * kLpThreads; i < hi; i += 32 * kLpThreads)
      list_vector(sm, row, i, hi, bound);
  }
  __syncthreads();
  const int n = sm.count;
  if (n > kLpCand)
    scan_top(sm, row, lo, hi, K);
  else
    rank_keys(sm.cand, n, K, sm.top);
  __syncthreads();
  if constexpr (kCluster) {
    // every CTA leaves its sums and keys in rank 0's shared memory, which joins them
    auto cluster = cg::this_cluster();
    asm volatile("barrier.cluster.wait.aligned;" ::: "memory");   // rank 0 has started
    LpShared* to = cluster.map_shared_rank(&sm, 0);
    if (tid == 0) to->part[rank] = p;
    if (tid < K) to->peer[rank * K + tid] = sm.top[tid];
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
    if (rank != 0) return;
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
    const Partial q = {-INFINITY, 0.f, 0.f};
    p = warp_join<kLpMaxRanks>(lane % kLpMaxRanks < ranks ? sm.part[lane % kLpMaxRanks] : q, ks);
    // the K-th largest of all keys is at least any CTA's K-th, and at least the least of the CTAs'
    // ceil(K / ranks)-th
    if (warp == 0) {
      const int r_th = (K + ranks - 1) / ranks;
      uint64_t one = lane < ranks ? sm.peer[lane * K + K - 1] : 0ull;
      uint64_t every = lane < ranks ? sm.peer[lane * K + r_th - 1] : ~0ull;
#pragma unroll
      for (int o = 8; o > 0; o >>= 1) {
        const uint64_t x = __shfl_xor_sync(0xffffffffu, one, o);
        const uint64_t y = __shfl_xor_sync(0xffffffffu, every, o);
        one = x > one ? x : one;
        every = y < every ? y : every;
      }
      if (lane == 0) {
        sm.peer_bound = one > every ? one : every;
        sm.count = 0;
      }
    }
    __syncthreads();
    if (tid < K) sm.top[tid] = 0ull;
    const uint64_t least = sm.peer_bound;
    for (int i = tid; i < ranks * K; i += kLpThreads) {
      const uint64_t key = sm.peer[i];
      if (key != 0ull && key >= least) sm.cand[atomicAdd(&sm.count, 1)] = key;
    }
    __syncthreads();
    rank_keys(sm.cand, sm.count, K, sm.top);
    __syncthreads();
  }

  const bool bad = !(p.s == p.s) || p.m == INFINITY;   // a NaN or +inf among the logits
  const bool none = !bad && p.m == -INFINITY;
  const float nan = __int_as_float(0x7fffffff);
  const float log_s = logf(p.s);   // -inf for an empty row
  auto log_prob = [&](float x) {
    return bad ? nan : x == -INFINITY ? x : (x - p.m) * a.scale - log_s;
  };
  if (tid == 0) {
    if (bad) record_error(a.status, TV_ERR_VALUE);
    if (a.lse) a.lse[r] = bad ? nan : none ? -INFINITY : p.m * a.scale + log_s;
    if (a.entropy)
      a.entropy[r] = bad ? nan : none ? 0.f : fmaxf(log_s - a.scale * (p.t / p.s), 0.f);
  }
  if (tid < K) {
    const uint64_t key = bad ? 0ull : sm.top[tid];
    const int id = key ? (int)~(uint32_t)key : -1;
    if (tid == 0 && a.target) a.target[r] = id;
    if (tid < a.n_top) {
      a.top_ids[r * a.n_top + tid] = id;
      a.top_logprobs[r * a.n_top + tid] =
          bad ? nan : id < 0 ? -INFINITY : log_prob(logit_of_order((uint32_t)(key >> 32)));
    }
  }
  // given tokens: this row takes those of its node, and row 0 those without a node or a token
  for (int i = tid; i < a.n_tok; i += kLpThreads) {
    const int64_t at = (int64_t)b * a.n_tok + i;
    const bool early = i == tid && first;
    const int node = early ? given_node : a.nodes ? a.nodes[at] : i;
    const int tok = early ? given_tok : a.tokens[at];
    const bool wrong = node >= a.D || tok >= a.vocab;
    if (node < 0 || tok < 0 || wrong) {
      if (v == 0) {
        a.logprobs[at] = 0.f;
        if (wrong) record_error(a.status, TV_ERR_ARG);
      }
    } else if (node == v) {
      a.logprobs[at] = log_prob(early ? given : load_f(row.p + tok));
    }
  }
}

template <typename T, bool kCluster>
static cudaError_t launch_kernel(const T* logits, const LogprobArgs& a, int64_t rows, int ranks,
                                 cudaStream_t stream) {
  auto kernel = logprobs_kernel<T, kCluster>;
  const int smem = (int)sizeof(LpShared);
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e == cudaSuccess && ranks > 8)
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(rows * ranks));
  cfg.blockDim = dim3(kLpThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = ranks;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = kCluster ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, kernel, logits, a, ranks);
}

template <typename T>
static cudaError_t launch_logprobs(const T* logits, const LogprobArgs& a, int64_t rows,
                                   cudaStream_t stream) {
  // CTAs per row: enough for two per SM, each with a tile's worth of vectors
  const int64_t vecs = (int64_t)a.vocab * sizeof(T) / 16;
  int ranks = 1;
  while (ranks < kLpMaxRanks && rows * ranks < 2 * 152 && vecs / (2 * ranks) >= kLpTile / 2) ranks *= 2;
  return ranks == 1 ? launch_kernel<T, false>(logits, a, rows, 1, stream)
                    : launch_kernel<T, true>(logits, a, rows, ranks, stream);
}

}  // namespace tv

int tv_launch_logprobs(const tv_shape* s, int vocab, int64_t ld, int logits_dtype,
                       const void* logits, int n_tok, const int32_t* tokens, const int32_t* nodes,
                       float scale, int n_top, float* lse, float* entropy, float* logprobs,
                       int32_t* top_ids, float* top_logprobs, int32_t* target, int32_t* status,
                       cudaStream_t stream) {
  const tv::LogprobArgs a = {s->D,    vocab,    n_tok,   n_top,        ld,     scale, tokens, nodes, lse,
                             entropy, logprobs, top_ids, top_logprobs, target, status};
  const int64_t rows = (int64_t)s->B * s->D;
  const cudaError_t e = logits_dtype == TV_BF16
                            ? tv::launch_logprobs((const __nv_bfloat16*)logits, a, rows, stream)
                            : tv::launch_logprobs((const float*)logits, a, rows, stream);
  if (e != cudaSuccess) {
    cudaGetLastError();
    return tv_set_error(TV_ERR_CUDA, "tv_token_logprobs: launch failed: %s", cudaGetErrorString(e));
  }
  return tv_check_launch("tv_token_logprobs");
}

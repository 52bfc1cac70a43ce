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
// logit is >= t, so a logit below t is no alternative.  In the pass a thread only notes its two
// largest tiles and the largest logit of its other tiles; at the end t is taken from the threads'
// largest logits and the few tiles that reach t are looked at again, a vector per thread (all
// vectors of a thread where a third tile reaches t).  The logits found, little more than K, are
// ranked by counting: a key's place is the number of larger keys (a key is the logit's order, then
// the lower id, so keys differ).  Where many logits equal t and the list overflows, one more scan in
// the order of the ids takes what lies above t and the first K of those equal to it; should what
// lies above t alone overflow, one scan per alternative.
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

constexpr int kLpUnroll = 4;                        // 16-byte vectors per thread and tile
constexpr int kLpStages = 3;                        // tiles in flight
constexpr int kLpMaxTop = 32;
constexpr int kLpCand = 512;                        // candidate list
constexpr int kLpMaxRanks = 16;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

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

// Exponents are taken in base 2: with c = scale log2 e, a logit x contributes 2^{x c - m c}.  In the
// pass that is one fused multiply-add with the rounded product b = fl(m c), and the sums are
// relative to 2^b; the residual m c - b, at most 2^-24 |m c|, is taken out of ln S at the end.  Where
// |m c| is so large that the residual is no longer small ("far": a largest logit beyond thousands)
// the exponent is (x - m) c instead and the sums are relative to m itself.  Exponents below
// kMinExp count as it: 2^-256 is 0 here, and -inf stays out of the products.
constexpr float kMinExp = -256.f;
constexpr float kFar = 1e4f;

// Partial sums of a set of logits: their maximum m (-inf: none above -inf yet), S, and T = sum of
// exponent * 2^exponent.  A NaN or +inf logit makes S NaN.
struct Partial {
  float m, s, t;
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
__device__ __forceinline__ bool is_far(float m, float c) { return !(fabsf(m * c) < kFar); }

// m c - fl(m c)
__device__ __forceinline__ float residual_of(float m, float c) {
  return fmaf(m, c, -__fmul_rn(m, c));
}

// p relative to a maximum m >= p.m
__device__ __forceinline__ void rebase(Partial& p, float m, float c) {
  if (m > p.m) {
    // the sums are relative to the rounded products (not contracted) or, far, to m c itself; where
    // one of the two is far, the difference of p.m c and m c also takes the other's residual
    // (selected, not branched to: the masked batch of 120 rows 10.05 us, 10.26 us with branches)
    const bool far = is_far(m, c), was_far = is_far(p.m, c);
    const float r = residual_of(far ? p.m : m, c), mixed = far == was_far ? 0.f : far ? -r : r;
    const float d = far || was_far ? (p.m - m) * c + mixed
                                   : __fmul_rn(p.m, c) - __fmul_rn(m, c);
    const float e = fmaxf(d, kMinExp), f = exp2_approx(e);
    p.t = (p.t + e * p.s) * f;
    p.s *= f;
    p.m = m;
  }
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
  // vectors [first_whole, end_whole) lie inside the row
  __device__ __forceinline__ int first_whole() const { return skew == 0 ? 0 : 1; }
  __device__ __forceinline__ int end_whole() const { return (skew + vocab) / kVec; }
  __device__ __forceinline__ int id(int i, int j) const { return i * kVec - skew + j; }
  __device__ __forceinline__ uint4 whole(int i) const {
    return *reinterpret_cast<const uint4*>(p + (i * kVec - skew));
  }
  // any vector; -inf where it reaches past the row
  __device__ __forceinline__ uint4 load(int i) const {
    if (i >= first_whole() && i < end_whole()) return whole(i);
    const int e0 = i * kVec - skew;
    uint32_t u[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      if constexpr (sizeof(T) == 2) {
        const int e = e0 + 2 * q;
        const uint32_t lo = e >= 0 && e < vocab ? bits(e) : 0xff80u;
        const uint32_t up = e + 1 >= 0 && e + 1 < vocab ? bits(e + 1) : 0xff80u;
        u[q] = lo | up << 16;
      } else {
        const int e = e0 + q;
        u[q] = e >= 0 && e < vocab ? bits(e) : 0xff800000u;
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
  // largest value of n vectors (NaN ignored)
  template <int n>
  __device__ static __forceinline__ float largest(const uint4 (&w)[n]) {
    if constexpr (sizeof(T) == 2) {
      auto h = [](uint32_t u) { return *reinterpret_cast<const __nv_bfloat162*>(&u); };
      __nv_bfloat162 m[n];
#pragma unroll
      for (int k = 0; k < n; ++k)
        m[k] = __hmax2(__hmax2(h(w[k].x), h(w[k].y)), __hmax2(h(w[k].z), h(w[k].w)));
#pragma unroll
      for (int k = 1; k < n; ++k) m[0] = __hmax2(m[0], m[k]);
      return fmaxf(__low2float(m[0]), __high2float(m[0]));
    } else {
      float m[n];
#pragma unroll
      for (int k = 0; k < n; ++k)
        m[k] = fmaxf(sm100::max3f(__uint_as_float(w[k].x), __uint_as_float(w[k].y),
                                  __uint_as_float(w[k].z)), __uint_as_float(w[k].w));
#pragma unroll
      for (int k = 1; k < n; ++k) m[0] = fmaxf(m[0], m[k]);
      return m[0];
    }
  }
};

__device__ __forceinline__ uint64_t max_u64(uint64_t a, uint64_t b) { return a > b ? a : b; }

// Shared memory of one CTA.  The lists of the end share the space of the tiles, which are done by
// then: what a CTA takes decides how many rows run at once on an SM.
template <int kThreads, bool kCluster>
struct LpShared {
  static constexpr int kWarps = kThreads / 32;
  struct Lists {
    uint64_t cand[kLpCand];
    int hit[2 * kThreads];         // tile * kThreads + thread: a thread's tile to look at again
    uint16_t column[kThreads];     // threads with more than two of them
    uint64_t ties[kLpMaxTop];      // keys of the first logits equal to the bound
  };
  union {
    uint4 ring[kLpStages][kLpUnroll][kThreads];   // tiles in flight; a thread reads only its own
    Lists list;
  };
  Partial warp_part[kWarps];
  uint64_t top[kLpMaxTop];         // largest keys, descending (0: none)
  alignas(16) uint32_t orders[kThreads];   // threads' largest logits (kth_bound)
  uint32_t kth;
  int count, hits, columns;
  uint64_t scan[kWarps];
  // rank 0's, written by the CTAs of the cluster: their shares of the row and their top lists
  Partial part[kCluster ? kLpMaxRanks : 1];
  uint64_t peer[kCluster ? kLpMaxRanks * kLpMaxTop : 1];
  uint64_t peer_bound;
};
static_assert(kLpMaxRanks * kLpMaxTop <= kLpCand, "every CTA's keys fit into cand");

// The K-th largest of the threads' orders o: every thread counts its place among all.
template <int kThreads, bool kCluster>
__device__ __noinline__ uint32_t kth_of_all(LpShared<kThreads, kCluster>& sm, uint32_t o, int K) {
  sm.orders[threadIdx.x] = o;
  __syncthreads();
  const uint4* all = reinterpret_cast<const uint4*>(sm.orders);
  int place = 0;
#pragma unroll 4
  for (int j = 0; j < kThreads / 4; ++j) {
    const uint4 x = all[j];
    const int d = (int)threadIdx.x - 4 * j;   // equal orders: threads in front count
    place += (x.x > o || (x.x == o && d > 0)) + (x.y > o || (x.y == o && d > 1)) +
             (x.z > o || (x.z == o && d > 2)) + (x.w > o || (x.w == o && d > 3));
  }
  if (place == K - 1) sm.kth = o;
  __syncthreads();
  return sm.kth;
}

// Lower bound (as an order) of the K-th largest logit that the CTA has seen, m being a thread's
// largest; the order of the lowest finite value where there are fewer.  It is the K-th largest among
// the 32 / warps largest threads of every warp, which for K up to 32 / warps is the K-th largest
// thread.  For more alternatives 128 threads count all of their places instead (512 rows of 32000
// bf16 logits, 32 alternatives: 16.8 us without, 14.4 us with), 256 threads do not (256 rows of
// 128000 fp32 logits, 20 alternatives: 25.1 us without, 27.6 us with).
template <int kThreads, bool kCluster>
__device__ __forceinline__ uint32_t kth_bound(LpShared<kThreads, kCluster>& sm, float m, int K) {
  constexpr int kWarps = kThreads / 32;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  constexpr int per = 32 / kWarps;
  uint32_t o = order_of(m), t;
  if (kThreads <= 128 && K > per) {
    t = kth_of_all(sm, o, K);
  } else {
#pragma unroll 1
    for (int i = 0; i < per; ++i) {
      uint32_t w = 0u;
      if (i < K) {
        w = __reduce_max_sync(0xffffffffu, o);
        const uint32_t at = __ballot_sync(0xffffffffu, o == w);
        if (lane == __ffs(at) - 1) o = 0u;
      }
      if (lane == 0) sm.orders[i * kWarps + warp] = w;
    }
    __syncthreads();
    const uint32_t v = sm.orders[lane];
    if (K == 1) {
      t = __reduce_max_sync(0xffffffffu, v);
    } else {
      int place = 0;
#pragma unroll
      for (int j = 0; j < 32; ++j) {
        const uint32_t x = __shfl_sync(0xffffffffu, v, j);
        place += x > v || (x == v && j < lane) ? 1 : 0;
      }
      t = __reduce_max_sync(0xffffffffu, place == K - 1 ? v : 0u);
    }
  }
  return max(t, kOrderLowest);
}

// Appends the logits >= bound of vector i to the candidate list.
template <typename T, int kThreads, bool kCluster>
__device__ __forceinline__ void list_vector(LpShared<kThreads, kCluster>& sm, const Row<T>& row, int i,
                                            float bound) {
  const uint4 q[1] = {row.load(i)};
  if (Row<T>::largest(q) < bound) return;
  float x[Row<T>::kVec];
  Row<T>::unpack(q[0], x);
#pragma unroll
  for (int j = 0; j < Row<T>::kVec; ++j)
    if (x[j] >= bound) {
      const int at = atomicAdd(&sm.count, 1);
      if (at < kLpCand) sm.list.cand[at] = key_of(x[j], row.id(i, j));
    }
}

// The CTA's K largest keys by one scan of its vectors [lo, hi) per key, into sm.top.
template <typename T, int kThreads, bool kCluster>
__device__ __noinline__ void scan_top(LpShared<kThreads, kCluster>& sm, const Row<T>& row, int lo,
                                      int hi, int K) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  uint64_t last = ~0ull;
  for (int k = 0; k < K; ++k) {
    uint64_t best = 0ull;
    for (int i = lo + threadIdx.x; i < hi; i += kThreads) {
      float x[Row<T>::kVec];
      Row<T>::unpack(row.load(i), x);
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
    for (int w = 0; w < kThreads / 32; ++w) best = max_u64(best, sm.scan[w]);
    if (threadIdx.x == 0) sm.top[k] = best;
    last = best;
  }
}

// Rebuilds the candidate list after an overflow, with the K-th largest of all threads' largest logits
// (m: this thread's) as the bound: the logits above it, and the K lowest ids of those equal to it.
// Returns its length (more than kLpCand: it overflowed again).
template <typename T, int kThreads, bool kCluster>
__device__ __noinline__ int list_with_ties(LpShared<kThreads, kCluster>& sm, const Row<T>& row, int lo,
                                           int hi, float m, int K) {
  constexpr int kVec = Row<T>::kVec;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  __syncthreads();
  if (tid == 0) sm.count = 0;
  const float bound = logit_of_order(max(kth_of_all(sm, order_of(m), K), kOrderLowest));
  int ties = 0;   // found so far, the same in every thread
  for (int i0 = lo; i0 < hi; i0 += kThreads) {
    const int i = i0 + tid;
    uint32_t equal = 0u;   // bit j: element j of the thread's vector
    if (i < hi) {
      float x[kVec];
      Row<T>::unpack(row.load(i), x);
#pragma unroll
      for (int j = 0; j < kVec; ++j) {
        if (x[j] == bound) equal |= 1u << j;
        if (x[j] > bound) {
          const int at = atomicAdd(&sm.count, 1);
          if (at < kLpCand) sm.list.cand[at] = key_of(x[j], row.id(i, j));
        }
      }
    }
    if (ties >= K || !__syncthreads_or(equal != 0u)) continue;
    // their places in the order of the ids: vectors ascend with the threads
    const int n = __popc(equal);
    int before = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, before, o);
      if (lane >= o) before += y;
    }
    if (lane == 31) sm.scan[warp] = before;
    __syncthreads();
    int at = ties + before - n;
    for (int w = 0; w < kThreads / 32; ++w) {
      const int c = (int)sm.scan[w];
      if (w < warp) at += c;
      ties += c;
    }
#pragma unroll
    for (int j = 0; j < kVec; ++j)
      if (equal >> j & 1u) {
        if (at < K) sm.list.ties[at] = key_of(bound, row.id(i, j));
        ++at;
      }
    __syncthreads();   // the counts are read
  }
  __syncthreads();
  const int above = sm.count, n = min(ties, K);
  if (above + n <= kLpCand && tid < n) sm.list.cand[above + tid] = sm.list.ties[tid];
  __syncthreads();
  return above + n;
}

// Places of the n keys of `list` among each other: out[place] = key for the places below K.
template <int kThreads>
__device__ __noinline__ void rank_keys(const uint64_t* list, int n, int K, uint64_t* out) {
  for (int i = threadIdx.x; i < n; i += kThreads) {
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

__device__ __forceinline__ uint4 ld_shared_16(uint32_t src) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(src));
  return v;
}

// Joins the partials held by the lanes of a warp (every lane gets the result).
template <int kLanes>
__device__ __forceinline__ Partial warp_join(Partial p, float c) {
  const uint32_t top = __reduce_max_sync(0xffffffffu, order_of(p.m));
  rebase(p, logit_of_order(top), c);
#pragma unroll
  for (int o = kLanes / 2; o > 0; o >>= 1) {
    p.s += __shfl_xor_sync(0xffffffffu, p.s, o);
    p.t += __shfl_xor_sync(0xffffffffu, p.t, o);
  }
  return p;
}

template <typename T, int kThreads, bool kCluster>
__global__ void __launch_bounds__(kThreads) logprobs_kernel(const T* logits,
                                                            const LogprobArgs a, int ranks) {
  constexpr int kWarps = kThreads / 32;
  constexpr int kTile = kThreads * kLpUnroll;   // vectors per tile
  extern __shared__ __align__(16) unsigned char smem_raw[];
  LpShared<kThreads, kCluster>& sm = *reinterpret_cast<LpShared<kThreads, kCluster>*>(smem_raw);
  pdl_wait();   // nothing is read before the kernel in front has completed
  const int rank = kCluster ? (int)cg::this_cluster().block_rank() : 0;
  const int r32 = kCluster ? blockIdx.x / ranks : blockIdx.x;   // rows: at most 2^21
  const int b = r32 / a.D, v = r32 - b * a.D;
  const int64_t r = r32;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const Row<T> row(logits + r * a.ld, a.vocab);
  constexpr int kVec = Row<T>::kVec;
  // (made to look different from thread to thread, so that it lives in an ordinary register: the
  // packed instructions of the pass would fetch it from the uniform ones every time)
  const float c = fmaf(__int2float_rn(tid), 0.f, a.scale * kLog2e);
  const int K = a.n_top > 1 ? a.n_top : 1;
  // The CTA's vectors [lo, hi): its whole ones make `rows` rows of one vector per thread, which are
  // streamed in tiles of kLpUnroll rows; what is left (less than a row, and the ends of the vocabulary)
  // counts as two rows and a tile in front of them.
  const int per = kCluster ? (row.n_vec + ranks - 1) / ranks : row.n_vec;
  const int lo = min(row.n_vec, rank * per), hi = min(row.n_vec, lo + per);
  const int whole_lo = max(lo, min(hi, row.first_whole()));
  const int rows = max(0, min(hi, row.end_whole()) - whole_lo) / kThreads;
  const int head = whole_lo - lo, rest = whole_lo + rows * kThreads;   // left over: [lo, whole_lo), [rest, hi)
  // vector of row r (0, 1: left over) of a thread, -1: none
  auto vector_of = [&](int r, int thread) {
    if (r >= 2) return r - 2 < rows ? whole_lo + (r - 2) * kThreads + thread : -1;
    const int j = r * kThreads + thread;
    return j < head ? lo + j : rest + j - head < hi ? rest + j - head : -1;
  };
  const int tiles = (rows + kLpUnroll - 1) / kLpUnroll;

  // a tile's copies into its stage
  const uint32_t ring = sm100::smem_u32(&sm.ring[0][0][tid]);
  constexpr uint32_t kStageBytes = sizeof(sm.ring[0]);
  const T* next_src = row.p + ((whole_lo + tid) * kVec - row.skew);
  int next_rows = rows;
  uint32_t next_slot = ring;
  auto fetch = [&] {
#pragma unroll
    for (int u = 0; u < kLpUnroll; ++u)
      if (u < next_rows) cp_async_16(next_slot + u * kThreads * 16, next_src + u * kThreads * kVec);
    asm volatile("cp.async.commit_group;" ::: "memory");
    next_rows -= kLpUnroll;
    next_src += kTile * kVec;
    next_slot = next_slot == ring + (kLpStages - 1) * kStageBytes ? ring : next_slot + kStageBytes;
  };
#pragma unroll 1
  for (int t = 0; t < kLpStages - 1; ++t) fetch();
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
  if (tid == 0) sm.count = sm.hits = sm.columns = 0;
  if (tid < K) sm.top[tid] = 0ull;

  const uint64_t c2 = pack_f32x2(c, c);
  Partial p = {-INFINITY, 0.f, 0.f};
  // largest logits of the three largest tiles (the first: p.m), and which the first two are
  float second = -INFINITY, third = -INFINITY;
  int tile1 = 0, tile2 = 0;
  auto note_tile = [&](float m, int t) {
    third = fmaxf(third, fminf(second, m));
    if (m > second) {
      tile2 = m > p.m ? tile1 : t;
      second = fminf(p.m, m);
    }
    if (m > p.m) {
      tile1 = t;
      rebase(p, m, c);
    }
  };
  // adds a vector's logits to the sums, exponents bounded: any logits, any maximum
  auto add_vector = [&](const uint4& w, float& s, float& t) {
    const bool far = is_far(p.m, c);
    const float base = p.m == -INFINITY ? 0.f : p.m, shift = -__fmul_rn(p.m, c);
    float x[kVec];
    Row<T>::unpack(w, x);
#pragma unroll
    for (int j = 0; j < kVec; ++j) {
      const float y = max_nan(far ? (x[j] - base) * c : fmaf(x[j], c, shift), kMinExp);
      const float e = exp2_approx(y);
      s += e;
      t += y * e;
    }
  };
  {
    const int i0 = vector_of(0, tid), i1 = vector_of(1, tid);
    if (i0 >= 0) {
      const uint4 w[2] = {row.load(i0), row.load(i1 >= 0 ? i1 : i0)};
      note_tile(Row<T>::largest(w), 0);
      add_vector(w[0], p.s, p.t);
      if (i1 >= 0) add_vector(w[1], p.s, p.t);
    }
  }
  uint32_t slot = ring;
  int left = rows;
#pragma unroll 1
  for (int t = 1; t <= tiles; ++t, left -= kLpUnroll) {
    fetch();
    asm volatile("cp.async.wait_group %0;" ::"n"(kLpStages - 1) : "memory");
    uint4 w[kLpUnroll];
#pragma unroll
    for (int u = 0; u < kLpUnroll; ++u)   // (a row that is not there: the first one again, not added)
      w[u] = ld_shared_16(slot + (u < left ? u : 0) * kThreads * 16);
    note_tile(Row<T>::largest(w), t);
    const float shift = -__fmul_rn(p.m, c);
    const uint64_t shift2 = pack_f32x2(shift, shift);
    uint64_t s2 = pack_f32x2(0.f, 0.f), t2 = s2;
#pragma unroll
    for (int u = 0; u < kLpUnroll; ++u) {
      if (u >= left) break;
      float x[kVec];
      Row<T>::unpack(w[u], x);
#pragma unroll
      for (int j = 0; j < kVec; j += 2) {
        const uint64_t y = fma_f32x2(pack_f32x2(x[j], x[j + 1]), c2, shift2);
        float y0, y1;
        unpack_f32x2(y, y0, y1);
        const uint64_t e = pack_f32x2(exp2_approx(y0), exp2_approx(y1));
        s2 = add_f32x2(s2, e);
        t2 = fma_f32x2(y, e, t2);
      }
    }
    float ds, dt, s1, t1;
    unpack_f32x2(s2, ds, s1);
    unpack_f32x2(t2, dt, t1);
    ds += s1;
    dt += t1;
    if (!(dt == dt) || is_far(p.m, c)) {
      // a masked logit (-inf times 0) or far exponents: the same sums with bounded exponents
      ds = dt = 0.f;
#pragma unroll 1
      for (int u = 0; u < min(left, kLpUnroll); ++u)
        add_vector(ld_shared_16(slot + u * kThreads * 16), ds, dt);
    }
    p.s += ds;
    p.t += dt;
    slot = slot == ring + (kLpStages - 1) * kStageBytes ? ring : slot + kStageBytes;
  }
  // the CTA's sums
  const float largest = p.m;
  p = warp_join<32>(p, c);
  if (lane == 0) sm.warp_part[warp] = p;
  const float bound = logit_of_order(kth_bound(sm, largest, K));   // (its barrier: warp_part)
  p = warp_join<kWarps>(sm.warp_part[lane % kWarps], c);
  if (third >= bound) {
    sm.list.column[atomicAdd(&sm.columns, 1)] = (uint16_t)tid;
  } else if (largest >= bound) {
    const int two = second >= bound ? 1 : 0, at = atomicAdd(&sm.hits, 1 + two);
    sm.list.hit[at] = tile1 * kThreads + tid;
    if (two) sm.list.hit[at + 1] = tile2 * kThreads + tid;
  }
  __syncthreads();
  const int looks = sm.hits * kLpUnroll, columns = sm.columns;
#pragma unroll 1
  for (int k = tid; k < looks + columns * kThreads; k += kThreads) {
    // a row of a tile, or (whole CTA) the rows of a thread
    if (k < looks) {
      const int hit = sm.list.hit[k / kLpUnroll], u = k % kLpUnroll, tile = hit / kThreads;
      const int r = tile == 0 ? u : 2 + (tile - 1) * kLpUnroll + u;
      const int i = tile == 0 && u >= 2 ? -1 : vector_of(r, hit % kThreads);
      if (i >= 0) list_vector(sm, row, i, bound);
    } else {
      if (*(volatile int*)&sm.count > kLpCand) break;   // too many equal logits
      const int q = k - looks, thread = sm.list.column[q / kThreads];
      for (int r = q % kThreads; r < rows + 2; r += kThreads) {
        const int i = vector_of(r, thread);
        if (i >= 0) list_vector(sm, row, i, bound);
      }
    }
  }
  __syncthreads();
  int n = sm.count;
  if (n > kLpCand) n = list_with_ties(sm, row, lo, hi, largest, K);
  if (n > kLpCand)
    scan_top(sm, row, lo, hi, K);
  else
    rank_keys<kThreads>(sm.list.cand, n, K, sm.top);
  __syncthreads();
  if constexpr (kCluster) {
    // every CTA leaves its sums and keys in rank 0's shared memory, which joins them
    auto cluster = cg::this_cluster();
    asm volatile("barrier.cluster.wait.aligned;" ::: "memory");   // rank 0 has started
    LpShared<kThreads, kCluster>* to = cluster.map_shared_rank(&sm, 0);
    if (tid == 0) to->part[rank] = p;
    if (tid < K) to->peer[rank * K + tid] = sm.top[tid];
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
    if (rank != 0) return;
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
    const Partial q = {-INFINITY, 0.f, 0.f};
    p = warp_join<kLpMaxRanks>(lane % kLpMaxRanks < ranks ? sm.part[lane % kLpMaxRanks] : q, c);
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
    for (int i = tid; i < ranks * K; i += kThreads) {
      const uint64_t key = sm.peer[i];
      if (key != 0ull && key >= least) sm.list.cand[atomicAdd(&sm.count, 1)] = key;
    }
    __syncthreads();
    rank_keys<kThreads>(sm.list.cand, sm.count, K, sm.top);
    __syncthreads();
  }

  const bool bad = !(p.s == p.s) || p.m == INFINITY;   // a NaN or +inf among the logits
  const bool none = !bad && p.m == -INFINITY;
  const float nan = __int_as_float(0x7fffffff);
  // ln S relative to m: the rounding of m c taken out (-inf for an empty row)
  const float residual = is_far(p.m, c) ? 0.f : residual_of(p.m, c);
  const float ln_s = logf(p.s), log_s = ln_s - residual * kLn2;
  auto log_prob = [&](float x) {
    return bad ? nan : x == -INFINITY ? x : (x - p.m) * a.scale - log_s;
  };
  if (tid == 0) {
    if (bad) record_error(a.status, TV_ERR_VALUE);
    if (a.lse) a.lse[r] = bad ? nan : none ? -INFINITY : p.m * a.scale + log_s;
    if (a.entropy)
      a.entropy[r] = bad ? nan : none ? 0.f : fmaxf(ln_s - kLn2 * (p.t / p.s), 0.f);
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
  for (int i = tid; i < a.n_tok; i += kThreads) {
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

template <typename T, int kThreads, bool kCluster>
static cudaError_t launch_kernel(const T* logits, const LogprobArgs& a, int64_t rows, int ranks,
                                 cudaStream_t stream) {
  auto kernel = logprobs_kernel<T, kThreads, kCluster>;
  const int smem = (int)sizeof(LpShared<kThreads, kCluster>);
  cudaError_t e = cudaSuccess;
  if (smem > 48 * 1024)
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e == cudaSuccess && ranks > 8)
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(rows * ranks));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = ranks;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = kCluster ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, logits, a, ranks);
}

template <typename T>
static cudaError_t launch_logprobs(const T* logits, const LogprobArgs& a, int64_t rows,
                                   cudaStream_t stream) {
  const int64_t vecs = (int64_t)a.vocab * sizeof(T) / 16;
  // Long rows are shared by a cluster while little more than the SMs are taken: 6 rows of 200000 fp32
  // logits 20.8 us as one CTA each, 10.2 us over 16; 48 rows 23.5 and 16.5 us (over 4); but 120 rows
  // of 50001 bf16 logits 8.1 us, 9.6 us over 2.  Shorter shares than 2500 vectors do not pay for the
  // cluster's barriers: 8 rows of 32000 bf16 logits 6.8 us, 7.5 us over 2.
  int ranks = 1;
  while (ranks < kLpMaxRanks && rows * ranks * 2 <= 200 && vecs / (2 * ranks) >= 2500) ranks *= 2;
  if (ranks > 1) return launch_kernel<T, 256, true>(logits, a, rows, ranks, stream);
  // many rows fill the SMs with small CTAs, whose ends cost less (512 rows of 2048 bf16 logits: 6.1
  // us with 128 threads, 7.3 us with 256); fewer rows want more loads in flight per row (256 rows of
  // 128000 fp32 logits: 31.5 and 25.3 us); very many short rows take two warps each (1372 rows of
  // 2875 fp32 logits: 8.7 us with 64 threads, 11.4 us with 128; 4096 of 16000 bf16: 34.6 and 38.0;
  // but 512 rows of 8000 bf16: 7.7 and 6.9)
  if (rows >= 8 * 152 && vecs <= 2048) return launch_kernel<T, 64, false>(logits, a, rows, 1, stream);
  return rows >= 512 ? launch_kernel<T, 128, false>(logits, a, rows, 1, stream)
                     : launch_kernel<T, 256, false>(logits, a, rows, 1, stream);
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

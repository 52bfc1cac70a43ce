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
// The alternatives come out of the same pass.  K distinct threads whose largest logits are >= t
// show that the K-th largest logit of the row is >= t, so a logit below t is no alternative: after
// the first tile of the row (and again after 2, 4, 8, ... tiles) such a t is taken from the
// threads' running maxima, and only logits >= t, a few per tile, go to a candidate list in shared
// memory.  At the end the list is ranked by counting: a key's place is the number of larger keys
// (a key is the logit's order, then the lower id, so keys differ).  A list that overflows (rows of
// many equal logits, ascending rows) is replaced by one scan of the row per alternative.
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

constexpr int kLpThreads = 256;
constexpr int kLpWarps = kLpThreads / 32;
constexpr int kLpUnroll = 4;                        // 16-byte vectors per thread and tile
constexpr int kLpTile = kLpThreads * kLpUnroll;     // vectors per tile
constexpr int kLpMaxTop = 32;
constexpr int kLpCand = 1024;                       // candidate list
constexpr int kLpMaxRanks = 8;
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

// Shared memory of one CTA.  part and top are read by the other CTAs of the cluster.
struct LpShared {
  Partial warp_part[kLpWarps];
  Partial part;                    // the CTA's share of the row
  uint64_t top[kLpMaxTop];         // its largest keys, descending (0: none)
  uint32_t bound[2][kLpWarps][2];
  int count, kept;
  uint64_t scan[kLpWarps];
  uint64_t cand[kLpCand];
  uint64_t sel[kLpCand];
};

// Lower bound (as an order) of the K-th largest logit that the CTA has seen, from the threads'
// largest ones: either K threads of one warp are at or above it, or ceil(K / 8) of every warp.
__device__ __forceinline__ uint32_t kth_bound(LpShared& sm, int parity, float m, int K) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int r = (K + kLpWarps - 1) / kLpWarps;
  uint32_t o = order_of(m);
  uint32_t kth = 0u, rth = 0u;
  const int rounds = K <= 4 ? K : r;
  for (int i = 1; i <= rounds; ++i) {
    const uint32_t w = __reduce_max_sync(0xffffffffu, o);
    if (i == r) rth = w;
    if (i == K) kth = w;
    const uint32_t at = __ballot_sync(0xffffffffu, o == w);
    if (lane == __ffs(at) - 1) o = 0u;
  }
  if (lane == 0) {
    sm.bound[parity][warp][0] = kth;
    sm.bound[parity][warp][1] = rth;
  }
  __syncthreads();
  uint32_t one = 0u, every = 0xffffffffu;
#pragma unroll
  for (int w = 0; w < kLpWarps; ++w) {
    one = max(one, sm.bound[parity][w][0]);
    every = min(every, sm.bound[parity][w][1]);
  }
  uint32_t t = max(one, every);
  if (t < kOrderLowest && K > 4) {
    // some warp has too few logits (a short or masked stretch): the K-th of one warp after all
    o = order_of(m);
    for (int i = 1; i < K; ++i) {
      const uint32_t w = __reduce_max_sync(0xffffffffu, o);
      if (w < kOrderLowest) break;
      const uint32_t at = __ballot_sync(0xffffffffu, o == w);
      if (lane == __ffs(at) - 1) o = 0u;
    }
    o = __reduce_max_sync(0xffffffffu, o);
    __syncthreads();
    if (lane == 0) sm.bound[parity][warp][0] = o;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kLpWarps; ++w) t = max(t, sm.bound[parity][w][0]);
  }
  return max(t, kOrderLowest);
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
__device__ __forceinline__ void rank_keys(const uint64_t* list, int n, int K, uint64_t* out) {
  for (int i = threadIdx.x; i < n; i += kLpThreads) {
    const uint64_t key = list[i];
    int place = 0;
#pragma unroll 8
    for (int j = 0; j < n; ++j) place += list[j] > key ? 1 : 0;
    if (place < K) out[place] = key;
  }
}

template <typename T, bool kCluster>
__global__ void __launch_bounds__(kLpThreads) logprobs_kernel(const T* __restrict__ logits,
                                                              const LogprobArgs a, int ranks) {
  __shared__ LpShared sm;
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

  if (tid == 0) sm.count = sm.kept = 0;
  if (tid < K) sm.top[tid] = 0ull;
  uint4 next[kLpUnroll];
  auto fetch = [&](int i0) {
    if (i0 > 0 && i0 + kLpTile <= hi && i0 + kLpTile < row.n_vec) {   // no edge in the tile
#pragma unroll
      for (int u = 0; u < kLpUnroll; ++u) next[u] = row.whole(i0 + u * kLpThreads + tid);
    } else {
#pragma unroll
      for (int u = 0; u < kLpUnroll; ++u) next[u] = row.edge(i0 + u * kLpThreads + tid, hi);
    }
  };
  Partial p = {-INFINITY, 0.f, 0.f};
  float bound = 0.f;
  int parity = 0, refresh = 1;
  fetch(lo);
  for (int t = 0, i0 = lo; i0 < hi; ++t, i0 += kLpTile) {
    uint4 w[kLpUnroll];
    float vmax[kLpUnroll];
#pragma unroll
    for (int u = 0; u < kLpUnroll; ++u) w[u] = next[u];
    if (i0 + kLpTile < hi) fetch(i0 + kLpTile);
    float m = p.m;
#pragma unroll
    for (int u = 0; u < kLpUnroll; ++u) {
      vmax[u] = Row<T>::largest(w[u]);
      m = fmaxf(m, vmax[u]);
    }
    rebase(p, m, ks);
    const float base = p.m == -INFINITY ? 0.f : p.m;
    const uint64_t neg = pack_f32x2(-base, -base), c2 = pack_f32x2(ks.c, ks.c);
    uint64_t s2 = pack_f32x2(0.f, 0.f), t2 = s2;
#pragma unroll
    for (int u = 0; u < kLpUnroll; ++u) {
      float x[kVec];
      Row<T>::unpack(w[u], x);
#pragma unroll
      for (int j = 0; j < kVec; j += 2) {
        float d0, d1, y0, y1;
        unpack_f32x2(add_f32x2(pack_f32x2(x[j], x[j + 1]), neg), d0, d1);
        const uint64_t d = pack_f32x2(max_nan(d0, ks.dmin), max_nan(d1, ks.dmin));
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
    p.t += t0 + t1;
    // candidates; the first tile sets the bound before it looks at its own logits
    if (t == 0) bound = logit_of_order(kth_bound(sm, 0, p.m, K));
#pragma unroll
    for (int u = 0; u < kLpUnroll; ++u) {
      if (vmax[u] >= bound) {
        float x[kVec];
        Row<T>::unpack(w[u], x);
#pragma unroll
        for (int j = 0; j < kVec; ++j)
          if (x[j] >= bound) {
            const int at = atomicAdd(&sm.count, 1);
            if (at < kLpCand) sm.cand[at] = key_of(x[j], row.id(i0 + u * kLpThreads + tid, j));
          }
      }
    }
    if (t == refresh) {
      parity ^= 1;
      bound = logit_of_order(kth_bound(sm, parity, p.m, K));
      refresh = 2 * refresh + 1;   // after 2, 4, 8, ... tiles
    }
  }
  // the CTA's sums
  const float largest = p.m;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const Partial q = {__shfl_xor_sync(0xffffffffu, p.m, o), __shfl_xor_sync(0xffffffffu, p.s, o),
                       __shfl_xor_sync(0xffffffffu, p.t, o)};
    p = join(p, q, ks);
  }
  if (lane == 0) sm.warp_part[warp] = p;
  // the final bound leaves little of the list (its barrier also publishes the list and the sums)
  const uint32_t final_bound = kth_bound(sm, parity ^ 1, largest, K);
  p = sm.warp_part[0];
#pragma unroll
  for (int w = 1; w < kLpWarps; ++w) p = join(p, sm.warp_part[w], ks);
  if (tid == 0) sm.part = p;
  const int n = sm.count;
  if (n > kLpCand) {
    scan_top(sm, row, lo, hi, K);
  } else {
    for (int i = tid; i < n; i += kLpThreads) {
      const uint64_t key = sm.cand[i];
      if ((uint32_t)(key >> 32) >= final_bound) sm.sel[atomicAdd(&sm.kept, 1)] = key;
    }
    __syncthreads();
    rank_keys(sm.sel, sm.kept, K, sm.top);
  }
  __syncthreads();
  if constexpr (kCluster) {
    // rank 0 joins the CTAs' sums and keys
    auto cluster = cg::this_cluster();
    cluster.sync();
    if (rank == 0) {
      for (int i = tid; i < ranks * K; i += kLpThreads) {
        const int q = i / K;
        sm.sel[i] = cluster.map_shared_rank(&sm, q)->top[i - q * K];
      }
      for (int q = 1; q < ranks; ++q) p = join(p, cluster.map_shared_rank(&sm, q)->part, ks);
    }
    cluster.sync();   // every CTA's shared memory has been read
    if (rank != 0) return;
    if (tid < K) sm.top[tid] = 0ull;
    __syncthreads();
    // (0 stands for no key: its place is behind the others, and equal places hold equal zeros)
    rank_keys(sm.sel, ranks * K, K, sm.top);
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
    const int node = a.nodes ? a.nodes[at] : i, tok = a.tokens[at];
    const bool wrong = node >= a.D || tok >= a.vocab;
    if (node < 0 || tok < 0 || wrong) {
      if (v == 0) {
        a.logprobs[at] = 0.f;
        if (wrong) record_error(a.status, TV_ERR_ARG);
      }
    } else if (node == v) {
      a.logprobs[at] = log_prob(load_f(row.p + tok));
    }
  }
}

template <typename T>
static cudaError_t launch_logprobs(const T* logits, const LogprobArgs& a, int64_t rows,
                                   cudaStream_t stream) {
  // CTAs per row: enough for two per SM, each with a tile's worth of vectors
  const int64_t vecs = (int64_t)a.vocab * sizeof(T) / 16;
  int ranks = 1;
  while (ranks < kLpMaxRanks && rows * ranks < 2 * 152 && vecs / (2 * ranks) >= kLpThreads) ranks *= 2;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(rows * ranks));
  cfg.blockDim = dim3(kLpThreads);
  cfg.stream = stream;
  if (ranks == 1) return cudaLaunchKernelEx(&cfg, logprobs_kernel<T, false>, logits, a, 1);
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = ranks;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, logprobs_kernel<T, true>, logits, a, ranks);
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

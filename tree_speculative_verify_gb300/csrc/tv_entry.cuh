// The compressor routines shared by prefill, the scratch pad and the appending of new tokens: the
// same arithmetic in the same order, so that equal rows give bit-identical entries.  The entry's
// formula and its orders are in tv_compress.cu.
#pragma once

#include <cooperative_groups.h>
#include <math.h>

#include "tv_common.cuh"

namespace tv {

constexpr int kThreads = 256;                   // every compressor CTA: eight warps
constexpr int kWarps = kThreads / 32;
constexpr int kC128Ranks = 8;                   // CTAs per 128-token block (one cluster)
constexpr int kC128Tokens = 128 / kC128Ranks;   // tokens per CTA: two per warp
static_assert(kC128Tokens == 2 * kWarps, "two C128 tokens per warp");

// Raw 16-byte vector and its conversion to fp32 (loads are issued first, converted later, so
// many loads are in flight at once).
template <typename T>
__device__ __forceinline__ uint4 ld16(const T* p) { return *reinterpret_cast<const uint4*>(p); }
__device__ __forceinline__ void cvt16(uint4 u, __nv_bfloat16*, float* out) {
  const __nv_bfloat162* h = reinterpret_cast<const __nv_bfloat162*>(&u);
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const float2 f = __bfloat1622float2(h[k]);
    out[2 * k] = f.x;
    out[2 * k + 1] = f.y;
  }
}
__device__ __forceinline__ void cvt16(uint4 u, float*, float* out) {
  out[0] = __uint_as_float(u.x);
  out[1] = __uint_as_float(u.y);
  out[2] = __uint_as_float(u.z);
  out[3] = __uint_as_float(u.w);
}

template <typename T>
struct VecWidth;
template <>
struct VecWidth<__nv_bfloat16> {
  static constexpr int n = 8;
};
template <>
struct VecWidth<float> {
  static constexpr int n = 4;
};

// 16-byte asynchronous copy global -> shared.  The copies a thread issued are committed as a group
// (cp_async_commit); cp_async_wait(n) waits until at most the n most recent groups are pending;
// a barrier then makes every thread's copies visible to the CTA.
__device__ __forceinline__ void cp_async16(void* smem, const void* gmem) {
  const unsigned s = (unsigned)__cvta_generic_to_shared(smem);
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(s), "l"(gmem) : "memory");
}
__device__ __forceinline__ void cp_async_commit() {
  asm volatile("cp.async.commit_group;" ::: "memory");
}
__device__ __forceinline__ void cp_async_wait(int pending) {
  if (pending > 0)
    asm volatile("cp.async.wait_group 1;" ::: "memory");
  else
    asm volatile("cp.async.wait_group 0;" ::: "memory");
}

constexpr int kMaxPairs = kMaxHeadDim / 2 / kC128Ranks;   // dimension pairs a rank finishes

// Shared memory of a C4 CTA (prefill and scratch pad).
template <typename T>
struct C4Smem {
  T rows4[4][2][kMaxHeadDim];   // the block's rows: token t: [0] = K row, [1] = V row
  float gate4[kMaxHeadDim];
  float z4[4];                  // gate logits
};

// Shared memory of a C128 cluster CTA (prefill and scratch pad).
template <typename T>
struct C128Smem {
  T rows[kC128Tokens][2][kMaxHeadDim];     // this rank's 16 block rows: [0] = K row, [1] = V row
  float gate128[kMaxHeadDim];
  float4 recv[2][kC128Ranks][kMaxPairs];   // by entry parity: sums (K 2p, K 2p+1, V 2p, V 2p+1)
                                           // of the dimension pairs this rank finishes, per
                                           // sending rank
  float2 ms[2][kC128Ranks];                // by entry parity: every rank's (max logit, sum of
                                           // weights)
  float z[kC128Tokens];                    // gate logits
  float w[kC128Tokens];                    // weights exp(z_t - m) (m: this rank's maximum)
};

// Copies rows (K and V) of the tokens t < n_tok with take[t] (all if take is null) into the row
// slots dst[t]: each thread issues 16-byte copies, all in flight at once.
template <typename T>
__device__ __forceinline__ void fetch_rows(T (*dst)[2][kMaxHeadDim], const T* const* srcK,
                                           const T* const* srcV, int n_tok, const bool* take,
                                           int d) {
  constexpr int VW = VecWidth<T>::n;
  const int per_row = d / VW;
  for (int t = 0; t < n_tok; ++t) {
    if (take != nullptr && !take[t]) continue;
    for (int c = threadIdx.x; c < 2 * per_row; c += blockDim.x) {
      const int which = c >= per_row;
      const int q = c - which * per_row;
      cp_async16(&dst[t][which][q * VW], (which ? srcV[t] : srcK[t]) + q * VW);
    }
  }
}

// A warp's view of one row: lane l holds the 16-byte groups l, l + 32, ... (KV of them at the
// largest head dimension; groups past d are zero).
template <typename T>
struct Lane16 {
  static constexpr int VW = VecWidth<T>::n;
  static constexpr int KV = kMaxHeadDim / (32 * VW);
};

// Gate logit z = K . g of one row, by one warp, from the lane's groups x[0..KV) of the row and
// the gate in shared memory: per lane in group then element order, then a butterfly sum over the
// lanes (every lane returns the same value).  The same arithmetic whether the row sits in shared
// memory or in registers.
template <typename T>
__device__ __forceinline__ float lane_logit(const uint4 (&x)[Lane16<T>::KV], const float* gate,
                                            int d, int lane) {
  constexpr int VW = Lane16<T>::VW;
  float acc = 0.f;
#pragma unroll
  for (int k = 0; k < Lane16<T>::KV; ++k) {
    const int i = lane * VW + 32 * VW * k;
    if (i >= d) break;
    float f[VW];
    cvt16(x[k], (T*)nullptr, f);
#pragma unroll
    for (int e = 0; e < VW; ++e) acc = fmaf(f[e], gate[i + e], acc);
  }
  return warp_sum(acc);
}

template <typename T>
__device__ __forceinline__ float row_logit(const T* row, const float* gate, int d, int lane) {
  constexpr int VW = Lane16<T>::VW;
  uint4 x[Lane16<T>::KV];
#pragma unroll
  for (int k = 0; k < Lane16<T>::KV; ++k) {
    const int i = lane * VW + 32 * VW * k;
    x[k] = i < d ? *reinterpret_cast<const uint4*>(row + i) : make_uint4(0u, 0u, 0u, 0u);
  }
  return lane_logit<T>(x, gate, d, lane);
}

// Two consecutive elements as fp32.
__device__ __forceinline__ float2 ld_pair(const float* p) { return *reinterpret_cast<const float2*>(p); }
__device__ __forceinline__ float2 ld_pair(const __nv_bfloat16* p) {
  return __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(p));
}

// Weighted sums over n_tok token rows in shared memory for the dimension pair (2p, 2p+1): tokens
// in order, one fused multiply-add each.  Returns (K 2p, K 2p+1, V 2p, V 2p+1).
template <typename T, int N>
__device__ __forceinline__ float4 pair_sums(const T (*rows)[2][kMaxHeadDim], const float* w,
                                            int p) {
  float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
  for (int t = 0; t < N; ++t) {
    const float2 k = ld_pair(&rows[t][0][2 * p]);
    const float2 v = ld_pair(&rows[t][1][2 * p]);
    a.x = fmaf(w[t], k.x, a.x);
    a.y = fmaf(w[t], k.y, a.y);
    a.z = fmaf(w[t], v.x, a.z);
    a.w = fmaf(w[t], v.y, a.w);
  }
  return a;
}

// ---- C4: one entry per CTA -------------------------------------------------------------------
// One entry from the 4 rows in sm.rows4 (position order; the caller has fetched them): warp t
// forms logit z_t; with M = max z_t and w_t = exp(z_t - M), dimension i of the entry is
// (sum_t w_t K_t[i], tokens in order) / (sum_t w_t).  Prefill and the scratch pad both run this
// routine, so equal rows give bit-identical entries.  out2K / out2V (nullable): a second place
// the entry is written to.  pending_after: 1 if the caller committed one more copy group after
// this entry's rows (the C128 rows), which need not have landed yet.
template <typename T>
__device__ void entry4(int d, const float* gate, T* outK, T* outV, T* out2K, T* out2V,
                       int pending_after, C4Smem<T>& sm) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  cp_async_wait(pending_after);   // groups committed after this entry's rows may stay pending
  __syncthreads();
  if (warp < 4) {
    const float z = row_logit<T>(sm.rows4[warp][0], gate, d, lane);
    if (lane == 0) sm.z4[warp] = z;
  }
  __syncthreads();
  const float M = fmaxf(fmaxf(sm.z4[0], sm.z4[1]), fmaxf(sm.z4[2], sm.z4[3]));
  float w[4], S = 0.f;
#pragma unroll
  for (int t = 0; t < 4; ++t) {
    w[t] = expf(sm.z4[t] - M);
    S += w[t];
  }
  for (int p = threadIdx.x; 2 * p < d; p += blockDim.x) {
    float4 a = pair_sums<T, 4>(sm.rows4, w, p);
    a.x /= S;
    a.y /= S;
    a.z /= S;
    a.w /= S;
    store_f(outK + 2 * p, a.x);
    store_f(outK + 2 * p + 1, a.y);
    store_f(outV + 2 * p, a.z);
    store_f(outV + 2 * p + 1, a.w);
    if (out2K != nullptr) {
      store_f(out2K + 2 * p, a.x);
      store_f(out2K + 2 * p + 1, a.y);
      store_f(out2V + 2 * p, a.z);
      store_f(out2V + 2 * p + 1, a.w);
    }
  }
  __syncthreads();   // rows4 and z4 are free for the next entry
}

// ---- C128: one entry per cluster --------------------------------------------------------------
// One 128-token entry by a cluster of eight CTAs: rank r holds the block's tokens 16r .. 16r+15
// in sm.rows (the caller has fetched them); warp w forms the logits of tokens 2w and 2w+1.  Each
// rank takes its own maximum m_r, forms w_t = exp(z_t - m_r) and, per dimension pair, sums w_t K_t
// and w_t V_t over its tokens in order; it sends the pair sums to the rank that finishes the pair
// and (m_r, sum_t w_t) to every rank -- one cluster barrier.  The finishing rank rescales the
// eight ranks' sums to M = max m_r (factor exp(m_r - M)), adds them in rank order and divides by
// the rescaled sum of weights.  All orders are fixed: the entry depends only on the block's rows,
// so prefill and the scratch pad agree bit for bit.  parity: the entry's index & 1 among the
// cluster's consecutive entries (the receive buffers alternate, so a rank that runs ahead into
// the next entry never writes a buffer that a slower rank still reads).  after_rows() runs on
// every thread once the rank's sums are sent, before the cluster barrier: the caller may refetch
// rows there (after a barrier of its own, since other threads may still read them).
template <typename T, typename AfterRows>
__device__ void entry128(int d, const float* gate, T* outK, T* outV, int parity, C128Smem<T>& sm,
                         AfterRows&& after_rows) {
  namespace cg = cooperative_groups;
  cg::cluster_group cl = cg::this_cluster();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int rank = (int)cl.block_rank();
  const int t0 = 2 * warp;
  const int ppr = (d / 2 + kC128Ranks - 1) / kC128Ranks;   // dimension pairs per rank
  cp_async_wait(0);
  __syncthreads();
  const float z0 = row_logit<T>(sm.rows[t0][0], gate, d, lane);
  const float z1 = row_logit<T>(sm.rows[t0 + 1][0], gate, d, lane);
  if (lane == 0) {
    sm.z[t0] = z0;
    sm.z[t0 + 1] = z1;
  }
  __syncthreads();
  float m = sm.z[0];
  for (int t = 1; t < kC128Tokens; ++t) m = fmaxf(m, sm.z[t]);
  if (threadIdx.x < kC128Tokens) sm.w[threadIdx.x] = expf(sm.z[threadIdx.x] - m);
  __syncthreads();
  for (int p = threadIdx.x; 2 * p < d; p += blockDim.x) {
    const float4 a = pair_sums<T, kC128Tokens>(sm.rows, sm.w, p);
    const int owner = p / ppr;
    *cl.map_shared_rank(&sm.recv[parity][rank][p - owner * ppr], owner) = a;
  }
  if (threadIdx.x < kC128Ranks) {   // (m, sum of weights) to every rank
    float s = 0.f;
    for (int t = 0; t < kC128Tokens; ++t) s += sm.w[t];
    *cl.map_shared_rank(&sm.ms[parity][rank], (int)threadIdx.x) = make_float2(m, s);
  }
  after_rows();
  cl.sync();   // every rank's sums have arrived
  pdl_wait();   // (scratch pad) the kernel before this one has completed before any store
  const int p = rank * ppr + (int)threadIdx.x;
  if ((int)threadIdx.x < ppr && 2 * p < d) {
    float M = sm.ms[parity][0].x;
    for (int q = 1; q < kC128Ranks; ++q) M = fmaxf(M, sm.ms[parity][q].x);
    float S = 0.f;
    float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int q = 0; q < kC128Ranks; ++q) {
      const float f = expf(sm.ms[parity][q].x - M);
      const float4 x = sm.recv[parity][q][threadIdx.x];
      S = fmaf(f, sm.ms[parity][q].y, S);
      a.x = fmaf(f, x.x, a.x);
      a.y = fmaf(f, x.y, a.y);
      a.z = fmaf(f, x.z, a.z);
      a.w = fmaf(f, x.w, a.w);
    }
    store_f(outK + 2 * p, a.x / S);
    store_f(outK + 2 * p + 1, a.y / S);
    store_f(outV + 2 * p, a.z / S);
    store_f(outV + 2 * p + 1, a.w / S);
  }
  __syncthreads();   // the rows may be refetched for the next entry
}

}  // namespace tv

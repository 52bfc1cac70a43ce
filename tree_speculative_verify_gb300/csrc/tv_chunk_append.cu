// New tokens into the persistent cache: rows rotated by position, entries of completed blocks,
// lengths ("Adapting Tree-Structured Speculative Decoding to DeepSeek-V4 for Efficient Inference"
// §2.2: online compression of the sequence as it grows; §4.2: the cache's three layers).
#include "tv_chunk.cuh"
#include "tv_entry.cuh"

namespace tv {

struct AppendArgs {
  Chunk c;
  int H, d, rope, pairs;
  int64_t ld;
  const float* inv_freq;
  int32_t* status;
};

// What becomes of request b: 0, or the error that leaves it as it was.
__device__ __forceinline__ int append_state(const Chunk& c, int b) {
  const int lo = c.starts[b], hi = c.starts[b + 1];
  if (lo < 0 || hi < lo || hi > c.n_new) return TV_ERR_ARG;
  const int n = hi - lo, L = c.L[b];
  if (n == 0) return TV_OK;
  if (L < 0) return TV_ERR_ARG;
  if (!chunk_fits(c, (int64_t)L + n)) return TV_ERR_CAPACITY;
  if (c.pg.page_tokens != 0)
    for (int g = L / c.pg.page_tokens; g <= (L + n - 1) / c.pg.page_tokens; ++g) {
      const int32_t page = c.pg.table[(int64_t)b * c.pg.max_pages + g];
      if (page < 0 || page >= c.pg.n_pool_pages) return TV_ERR_ARG;
    }
  return TV_OK;
}

// cos and sin of position * f: the angle in turns and its fraction in fp64 (an fp32 angle of 2^16
// radians is off by 2^-9), the functions of the fraction in fp32.
__device__ __forceinline__ void turn_of(int position, float f, float* cosine, float* sine) {
  const double turns = (double)position * ((double)f * 0.15915494309189533577);
  sincospif(2.f * (float)(turns - rint(turns)), sine, cosine);
}

// Element e of a row of d, its last r elements rotated.
template <typename T>
__device__ __forceinline__ T rotated(const T* row, int e, const AppendArgs& a, int position) {
  const int r = a.rope, k = e - (a.d - r);
  if (k < 0) return row[e];
  const int half = r / 2, i = a.pairs == TV_ROPE_PAIRS ? k / 2 : k % half;
  const bool second = a.pairs == TV_ROPE_PAIRS ? k & 1 : k >= half;
  const int x = a.d - r + (a.pairs == TV_ROPE_PAIRS ? 2 * i : i);
  const int y = x + (a.pairs == TV_ROPE_PAIRS ? 1 : half);
  float c, s;
  turn_of(position, a.inv_freq[i], &c, &s);
  const float u = load_f(row + x), v = load_f(row + y);
  T out;
  store_f(&out, second ? u * s + v * c : u * c - v * s);
  return out;
}

// A CTA per new token: its raw rows and its queries.
template <typename T>
__global__ void append_rows_kernel(AppendArgs a, const T* K, const T* V, const T* Q, T* Qr, T* rawK,
                                   T* rawV) {
  const int t = blockIdx.x, b = request_of(a.c.starts, a.c.B, t);
  if (b < 0 || append_state(a.c, b) != TV_OK) return;
  const int p = a.c.L[b] + t - a.c.starts[b];
  const int64_t row = layer_row(a.c.pg, b, p, a.c.raw_cap, 1, a.status) * a.d;
  for (int e = threadIdx.x; e < a.d; e += blockDim.x) {
    rawK[row + e] = rotated(K + t * a.ld, e, a, p);
    rawV[row + e] = V[t * a.ld + e];
  }
  if (Q == nullptr) return;
  extern __shared__ __align__(16) unsigned char smem_raw[];
  T* head = reinterpret_cast<T*>(smem_raw);   // (Qr may be Q)
  for (int h = 0; h < a.H; ++h) {
    const int64_t at = ((int64_t)t * a.H + h) * a.d;
    __syncthreads();
    for (int e = threadIdx.x; e < a.d; e += blockDim.x) head[e] = Q[at + e];
    __syncthreads();
    for (int e = threadIdx.x; e < a.d; e += blockDim.x) Qr[at + e] = rotated(head, e, a, p);
  }
}

// A CTA (C4) or a cluster (C128) per new token that completes a block.
template <typename T>
__global__ void __launch_bounds__(kThreads)
    append4_kernel(AppendArgs a, const T* rawK, const T* rawV, const float* g, T* CK, T* CV) {
  extern __shared__ __align__(16) unsigned char smem_raw[];
  C4Smem<T>& sm = *reinterpret_cast<C4Smem<T>*>(smem_raw);
  __shared__ const T* rowK[4];
  __shared__ const T* rowV[4];
  const int t = blockIdx.x, b = request_of(a.c.starts, a.c.B, t);
  if (b < 0 || append_state(a.c, b) != TV_OK) return;
  const int p = a.c.L[b] + t - a.c.starts[b];
  if ((p + 1) % 4 != 0) return;
  for (int i = threadIdx.x; i < a.d; i += blockDim.x) sm.gate4[i] = g[i];
  if (threadIdx.x < 4) {
    const int64_t row = layer_row(a.c.pg, b, p - 3 + threadIdx.x, a.c.raw_cap, 1, a.status) * a.d;
    rowK[threadIdx.x] = rawK + row;
    rowV[threadIdx.x] = rawV + row;
  }
  __syncthreads();
  fetch_rows<T>(sm.rows4, rowK, rowV, 4, nullptr, a.d);
  cp_async_commit();
  const int64_t out = layer_row(a.c.pg, b, p / 4, a.c.c4_cap, 4, a.status) * a.d;
  entry4<T>(a.d, sm.gate4, CK + out, CV + out, nullptr, nullptr, 0, sm);
}

template <typename T>
__global__ void __cluster_dims__(kC128Ranks, 1, 1) __launch_bounds__(kThreads)
    append128_kernel(AppendArgs a, const T* rawK, const T* rawV, const float* g, T* CK, T* CV) {
  extern __shared__ __align__(16) unsigned char smem_raw[];
  C128Smem<T>& sm = *reinterpret_cast<C128Smem<T>*>(smem_raw);
  __shared__ const T* rowK[kC128Tokens];
  __shared__ const T* rowV[kC128Tokens];
  const int rank = (int)cooperative_groups::this_cluster().block_rank();
  const int t = blockIdx.x / kC128Ranks, b = request_of(a.c.starts, a.c.B, t);
  if (b < 0 || append_state(a.c, b) != TV_OK) return;
  const int p = a.c.L[b] + t - a.c.starts[b];
  if ((p + 1) % 128 != 0) return;
  for (int i = threadIdx.x; i < a.d; i += blockDim.x) sm.gate128[i] = g[i];
  if (threadIdx.x < kC128Tokens) {
    const int64_t row = layer_row(a.c.pg, b, p - 127 + kC128Tokens * rank + threadIdx.x, a.c.raw_cap,
                                  1, a.status) * a.d;
    rowK[threadIdx.x] = rawK + row;
    rowV[threadIdx.x] = rawV + row;
  }
  __syncthreads();
  fetch_rows<T>(sm.rows, rowK, rowV, kC128Tokens, nullptr, a.d);
  cp_async_commit();
  const int64_t out = layer_row(a.c.pg, b, p / 128, a.c.c128_cap, 128, a.status) * a.d;
  entry128<T>(a.d, sm.gate128, CK + out, CV + out, 0, sm, [] {});
}

// The lengths advance once everything that reads them is done; errors are recorded here.
__global__ void append_lengths_kernel(AppendArgs a) {
  const int b = blockIdx.x * blockDim.x + threadIdx.x;
  if (b >= a.c.B) return;
  const int state = append_state(a.c, b);
  if (state != TV_OK)
    record_error(a.status, state);
  else
    a.c.L[b] += a.c.starts[b + 1] - a.c.starts[b];
}

template <typename T>
static int launch_append(const tv_shape* s, const AppendArgs& a, const void* K, const void* V,
                         const void* Q, const float* g4, const float* g128, void* Qr, void* rawK,
                         void* rawV, void* c4K, void* c4V, void* c128K, void* c128V,
                         cudaStream_t stream) {
  const char* fn = "tv_chunk_append";
  if (a.c.n_new > 0) {
    append_rows_kernel<T><<<a.c.n_new, 128, sizeof(T) * kMaxHeadDim, stream>>>(
        a, (const T*)K, (const T*)V, (const T*)Q, (T*)Qr, (T*)rawK, (T*)rawV);
    if (int rc = tv_check_launch(fn)) return rc;
    if (s->comp_mask & TV_COMP_C4) {
      append4_kernel<T><<<a.c.n_new, kThreads, sizeof(C4Smem<T>), stream>>>(
          a, (const T*)rawK, (const T*)rawV, g4, (T*)c4K, (T*)c4V);
      if (int rc = tv_check_launch(fn)) return rc;
    }
    if (s->comp_mask & TV_COMP_C128) {
      const int smem = (int)sizeof(C128Smem<T>);
      if (cudaFuncSetAttribute(append128_kernel<T>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                               smem) != cudaSuccess)
        return tv_check_launch(fn);
      append128_kernel<T><<<(unsigned)a.c.n_new * kC128Ranks, kThreads, smem, stream>>>(
          a, (const T*)rawK, (const T*)rawV, g128, (T*)c128K, (T*)c128V);
      if (int rc = tv_check_launch(fn)) return rc;
    }
  }
  append_lengths_kernel<<<(a.c.B + 255) / 256, 256, 0, stream>>>(a);
  return tv_check_launch(fn);
}

}  // namespace tv

int tv_launch_append(const tv_shape* s, int n_new, const int32_t* starts, const void* K,
                     const void* V, int64_t ld_kv, const void* Q, int rope_dim, int rope_pairs,
                     const float* inv_freq, const float* g4, const float* g128, void* Qr,
                     void* rawK, void* rawV, void* c4K, void* c4V, void* c128K, void* c128V,
                     int32_t* L, int32_t* status, cudaStream_t stream) {
  const tv::AppendArgs a = {tv::chunk_of(s, n_new, starts, L), s->H, s->d, rope_dim, rope_pairs,
                            ld_kv, inv_freq, status};
  return s->dtype == TV_BF16
             ? tv::launch_append<__nv_bfloat16>(s, a, K, V, Q, g4, g128, Qr, rawK, rawV, c4K, c4V,
                                                c128K, c128V, stream)
             : tv::launch_append<float>(s, a, K, V, Q, g4, g128, Qr, rawK, rawV, c4K, c4V, c128K,
                                        c128V, stream);
}

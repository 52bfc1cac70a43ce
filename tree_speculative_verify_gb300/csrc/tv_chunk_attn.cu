// Attention of a chunk of new tokens over the compressed cache that holds them, CUDA cores
// ("Adapting Tree-Structured Speculative Decoding to DeepSeek-V4 for Efficient Inference" §2.2,
// §3.1: what a position of an ordinary causal sequence sees).
//
// Per row (token at position p, head): s_j = scale q.k_j over the visible entries -- C4 j < p/4,
// C128 j < p/128, raw rows raw_lo(p) .. p -- in one pass with the running maximum m and sum l of
// exp(s - m); O = sum exp(s_j - m) v_j / l, lse = m + ln l.
#include <math.h>

#include "tv_chunk.cuh"

namespace tv {

struct ChunkAttnArgs {
  Chunk c;
  int H, d, W, tail_mode;
  float scale_log2;
  float* lse;
  int32_t* status;
};

// 0, or the error that leaves request b's rows alone.
__device__ __forceinline__ int attn_state(const Chunk& c, int b) {
  const int lo = c.starts[b], hi = c.starts[b + 1];
  if (lo < 0 || hi < lo || hi > c.n_new) return TV_ERR_ARG;
  if (hi == lo) return TV_OK;
  const int L = c.L[b];
  if (L < hi - lo) return TV_ERR_ARG;
  return chunk_fits(c, L) ? TV_OK : TV_ERR_CAPACITY;
}

__global__ void chunk_errors_kernel(Chunk c, int32_t* status) {
  const int b = blockIdx.x * blockDim.x + threadIdx.x;
  if (b >= c.B) return;
  const int state = attn_state(c, b);
  if (state != TV_OK) record_error(status, state);
}

// A warp per row.
template <typename T>
__global__ void chunk_rows_kernel(ChunkAttnArgs a, const T* Q, const T* c4K, const T* c4V,
                                  const T* c128K, const T* c128V, const T* rawK, const T* rawV,
                                  T* O) {
  const int lane = threadIdx.x & 31, d = a.d;
  const int64_t row = (int64_t)blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5);
  if (row >= (int64_t)a.c.n_new * a.H) return;
  const int t = (int)(row / a.H), b = request_of(a.c.starts, a.c.B, t);
  if (b < 0 || attn_state(a.c, b) != TV_OK) return;
  const int p = a.c.L[b] - (a.c.starts[b + 1] - t);
  const int n4 = a.c.comp_mask & TV_COMP_C4 ? p / 4 : 0;
  const int n128 = a.c.comp_mask & TV_COMP_C128 ? p / 128 : 0;
  const int lo = raw_lo_of(p, a.tail_mode, a.W, m_min_of(a.c.comp_mask));
  float q[kMaxHeadDim / 32], o[kMaxHeadDim / 32];
#pragma unroll
  for (int k = 0; k < kMaxHeadDim / 32; ++k) {
    const int e = lane + 32 * k;
    q[k] = e < d ? load_f(Q + row * d + e) * a.scale_log2 : 0.f;
    o[k] = 0.f;
  }
  float m = -INFINITY, l = 0.f;
  for (int j = 0; j < n4 + n128 + p + 1 - lo; ++j) {
    const T *k, *v;
    if (j < n4) {
      const int64_t r = layer_row(a.c.pg, b, j, a.c.c4_cap, 4, a.status) * d;
      k = c4K + r;
      v = c4V + r;
    } else if (j < n4 + n128) {
      const int64_t r = layer_row(a.c.pg, b, j - n4, a.c.c128_cap, 128, a.status) * d;
      k = c128K + r;
      v = c128V + r;
    } else {
      const int64_t r = layer_row(a.c.pg, b, lo + j - n4 - n128, a.c.raw_cap, 1, a.status) * d;
      k = rawK + r;
      v = rawV + r;
    }
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < kMaxHeadDim / 32; ++i)
      if (lane + 32 * i < d) s = fmaf(q[i], load_f(k + lane + 32 * i), s);
    s = warp_sum(s);
    const float top = fmaxf(m, s), alpha = exp2f(m - top), e = exp2f(s - top);
    l = l * alpha + e;
#pragma unroll
    for (int i = 0; i < kMaxHeadDim / 32; ++i)
      if (lane + 32 * i < d) o[i] = o[i] * alpha + e * load_f(v + lane + 32 * i);
    m = top;
  }
#pragma unroll
  for (int i = 0; i < kMaxHeadDim / 32; ++i)
    if (lane + 32 * i < d) store_f(O + row * d + lane + 32 * i, o[i] / l);
  if (lane == 0) a.lse[row] = (m + log2f(l)) * 0.6931471805599453f;
}

template <typename T>
static int launch_chunk_attn(const ChunkAttnArgs& a, const void* Q, const void* c4K,
                             const void* c4V, const void* c128K, const void* c128V,
                             const void* rawK, const void* rawV, void* O, cudaStream_t stream) {
  const char* fn = "tv_chunk_attn";
  chunk_errors_kernel<<<(a.c.B + 255) / 256, 256, 0, stream>>>(a.c, a.status);
  if (int rc = tv_check_launch(fn)) return rc;
  if (a.c.n_new == 0) return TV_OK;
  const int64_t rows = (int64_t)a.c.n_new * a.H;
  chunk_rows_kernel<T><<<(unsigned)((rows + 7) / 8), 256, 0, stream>>>(
      a, (const T*)Q, (const T*)c4K, (const T*)c4V, (const T*)c128K, (const T*)c128V,
      (const T*)rawK, (const T*)rawV, (T*)O);
  return tv_check_launch(fn);
}

}  // namespace tv

int tv_launch_chunk_attn(const tv_shape* s, int n_new, const int32_t* starts, const void* Q,
                         const void* c4K, const void* c4V, const void* c128K, const void* c128V,
                         const void* rawK, const void* rawV, const int32_t* L, float scale,
                         void* O, float* lse, int32_t* status, cudaStream_t stream) {
  const tv::ChunkAttnArgs a = {tv::chunk_of(s, n_new, starts, L), s->H, s->d, s->W, s->tail_mode,
                               scale * 1.4426950408889634f, lse, status};
  return s->dtype == TV_BF16
             ? tv::launch_chunk_attn<__nv_bfloat16>(a, Q, c4K, c4V, c128K, c128V, rawK, rawV, O, stream)
             : tv::launch_chunk_attn<float>(a, Q, c4K, c4V, c128K, c128V, rawK, rawV, O, stream);
}

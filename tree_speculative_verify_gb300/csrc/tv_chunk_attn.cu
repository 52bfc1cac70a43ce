// Attention of a chunk of new tokens over the compressed cache that holds them, CUDA cores
// ("Adapting Tree-Structured Speculative Decoding to DeepSeek-V4 for Efficient Inference" §2.2,
// §3.1: what a position of an ordinary causal sequence sees).
//
// Per row (token at position p, head): s_j = scale q.k_j over the visible entries -- C4 j < p/4,
// C128 j < p/128, raw rows raw_lo(p) .. p -- in one pass with the running maximum m and sum l of
// exp(s - m); O = sum exp(s_j - m) v_j / l, lse = m + ln l.  Everything in fp32.
//
// A CTA takes R rows of one request (token-major, so R / H neighbouring tokens) and a share of the
// entries that its last token sees, N at a time: K and V rows in shared memory as fp32, a register
// tile of R/16 x N/16 logits per thread, the probabilities through shared memory, a register tile of
// R/16 rows x 1/16 of the columns of O.  The copies of V run under the logits, those of the next K
// under O.  Requests of few rows (decoding) take R = 16, and while the CTAs do not fill the SMs the
// entries are split over several, whose partial sums a second kernel joins.
//
// Bound by the fused multiply-adds and the shared-memory reads that feed them: fp32, 7 requests of 486
// tokens behind 7000, 11 heads of d = 64, 128 and 256: 586, 1189 and 2487 us (32 to 34 TFLOP/s of 78);
// small tiles read shared memory for half as many operations each: 100 requests of one token behind
// 7000, 16 heads, d = 64 and 256: 81 and 269 us (1.3 and 1.5 TB/s).
#include <math.h>

#include "tv_chunk.cuh"
#include "tv_entry.cuh"

namespace tv {

struct ChunkAttnArgs {
  Chunk c;
  int H, d, W, tail_mode;
  int n_chunks;       // most shares of an item's entries
  float scale_log2;
  float* lse;
  float* part;        // [n_new * H][n_chunks][d + 4]: O, m (base 2), l
  int32_t* status;
};

constexpr int kShare = 128;   // least entries of a share

// R rows of one request and what they see.  Slots as in the tensor-core kernel: request b's tiles of R
// rows start at slot floor(starts[b] * H / R) + b.
struct RowTile {
  int b, row0, rows;   // first row of all n_new * H, rows (0: nothing to do)
  int first, pos0;     // first row within the request, position of the request's first new token
  int n4, n128, t0, entries, shares;
};

__device__ __forceinline__ RowTile row_tile(const ChunkAttnArgs& a, int R, int slot) {
  RowTile t;
  t.rows = 0;
  t.shares = 1;
  int lo = 0, hi = a.c.B;
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if ((int64_t)a.c.starts[mid] * a.H / R + mid <= slot)
      lo = mid + 1;
    else
      hi = mid;
  }
  const int b = lo - 1;
  if (b < 0 || attn_state(a.c, b) != TV_OK) return t;
  const int s0 = a.c.starts[b], n = a.c.starts[b + 1] - s0;
  const int64_t first = ((int64_t)slot - ((int64_t)s0 * a.H / R + b)) * R, rows = (int64_t)n * a.H;
  if (first >= rows) return t;
  t.b = b;
  t.first = (int)first;
  t.row0 = (int)((int64_t)s0 * a.H + first);
  t.rows = (int)(rows - first < R ? rows - first : R);
  t.pos0 = a.c.L[b] - n;
  const int p_lo = t.pos0 + t.first / a.H, p_hi = t.pos0 + (t.first + t.rows - 1) / a.H;
  t.n4 = a.c.comp_mask & TV_COMP_C4 ? p_hi / 4 : 0;
  t.n128 = a.c.comp_mask & TV_COMP_C128 ? p_hi / 128 : 0;
  t.t0 = raw_lo_of(p_lo, a.tail_mode, a.W, m_min_of(a.c.comp_mask));
  t.entries = t.n4 + t.n128 + p_hi + 1 - t.t0;
  t.shares = min(a.n_chunks, (t.entries + kShare - 1) / kShare);
  return t;
}

// 16 bytes into shared memory behind the thread's back (zeros if not there), in groups.
__device__ __forceinline__ void copy16(float* to, const void* from, bool there) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(
                   (uint32_t)__cvta_generic_to_shared(to)),
               "l"(from), "r"(there ? 16 : 0)
               : "memory");
}
__device__ __forceinline__ void copies_close() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int kOpen>
__device__ __forceinline__ void copies_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(kOpen) : "memory");
}

template <typename T, int R, int N, int DM>
struct SimtTile {
  static constexpr int kPitch = DM + 4;   // (rows 4 banks apart)
  float q[R][kPitch];
  float k[N][kPitch];
  float v[N][kPitch];
  float p[R][N + 4];
  int64_t at[2][N];   // rows of this tile's and the next one's entries, -1: none
};

// CTAs per SM that registers are left for: as many as shared memory holds, at most 2 (small tiles 3).
template <typename T, int R, int N, int DM>
constexpr int simt_ctas() {
  const int fit = (int)(227 * 1024 / sizeof(SimtTile<T, R, N, DM>)), most = R == 16 ? 3 : 2;
  return fit < most ? fit : most;
}

template <typename T, int R, int N, int DM>
__global__ void __launch_bounds__(256, (simt_ctas<T, R, N, DM>()))
    chunk_simt_kernel(ChunkAttnArgs a, const T* Q, const T* c4K, const T* c4V, const T* c128K,
                      const T* c128V, const T* rawK, const T* rawV, T* O) {
  using Tile = SimtTile<T, R, N, DM>;
  constexpr int RI = R / 16, EI = N / 16, CI = DM / 64, VW = VecWidth<T>::n;
  extern __shared__ __align__(16) unsigned char smem_raw[];
  Tile& sm = *reinterpret_cast<Tile*>(smem_raw);
  const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4, d = a.d;
  pdl_wait();
  pdl_launch_dependents();
  if (blockIdx.x == 0 && blockIdx.y == 0)
    for (int b = tid; b < a.c.B; b += 256) {
      const int state = attn_state(a.c, b);
      if (state != TV_OK) record_error(a.status, state);
    }
  const RowTile t = row_tile(a, R, blockIdx.x);
  if (t.rows == 0 || (int)blockIdx.y >= t.shares) return;
  const int e_lo = (int)((int64_t)t.entries * blockIdx.y / t.shares);
  const int e_hi = (int)((int64_t)t.entries * (blockIdx.y + 1) / t.shares);

  // Where entry e lives: its row, and which layer by e itself.
  auto locate = [&](int e) -> int64_t {
    if (e >= e_hi) return -1;
    if (e < t.n4) return layer_row(a.c.pg, t.b, e, a.c.c4_cap, 4, a.status);
    if (e < t.n4 + t.n128) return layer_row(a.c.pg, t.b, e - t.n4, a.c.c128_cap, 128, a.status);
    return layer_row(a.c.pg, t.b, t.t0 + e - t.n4 - t.n128, a.c.raw_cap, 1, a.status);
  };
  if (tid < N) sm.at[0][tid] = locate(e_lo + tid);
  // queries, scaled; columns past d are zeros (as those of K and V are)
  constexpr int kVecs = DM / VW;
  for (int i = tid; i < R * kVecs; i += 256) {
    const int r = i / kVecs, c = (i % kVecs) * VW;
    float f[VW];
    uint4 x = make_uint4(0u, 0u, 0u, 0u);
    if (r < t.rows && c < d) x = ld16(Q + (int64_t)(t.row0 + r) * d + c);
    cvt16(x, (T*)nullptr, f);
#pragma unroll
    for (int k = 0; k < VW; k += 4)
      *reinterpret_cast<float4*>(&sm.q[r][c + k]) =
          make_float4(f[k] * a.scale_log2, f[k + 1] * a.scale_log2, f[k + 2] * a.scale_log2,
                      f[k + 3] * a.scale_log2);
  }
  // what this thread's rows see
  int lim4[RI], lim128[RI], lo[RI], hi[RI];
#pragma unroll
  for (int i = 0; i < RI; ++i) {
    const int r = min(ty + 16 * i, t.rows - 1), p = t.pos0 + (t.first + r) / a.H;
    lim4[i] = p / 4;
    lim128[i] = t.n4 + p / 128;
    const int base = t.n4 + t.n128 - t.t0;
    lo[i] = base + raw_lo_of(p, a.tail_mode, a.W, m_min_of(a.c.comp_mask));
    hi[i] = base + p;
  }
  float m[RI], l[RI];
  float4 o[RI][CI];
#pragma unroll
  for (int i = 0; i < RI; ++i) {
    m[i] = -INFINITY;
    l[i] = 0.f;
#pragma unroll
    for (int c = 0; c < CI; ++c) o[i][c] = make_float4(0.f, 0.f, 0.f, 0.f);
  }
  __syncthreads();
  // The K or V rows of the entries e0 .. e0 + N - 1 on their way into shared memory.
  auto fetch = [&](float (*to)[Tile::kPitch], const T* s4, const T* s128, const T* sraw, int e0,
                   const int64_t* at) {
    if constexpr (sizeof(T) == 4) {
#pragma unroll
      for (int u = 0; u < N * kVecs / 256; ++u) {
        const int i = u * 256 + tid, r = i / kVecs, c = (i % kVecs) * VW, e = e0 + r;
        const T* from = e < t.n4 ? s4 : e < t.n4 + t.n128 ? s128 : sraw;
        const bool there = at[r] >= 0 && c < d;
        copy16(&to[r][c], from + (there ? at[r] * d + c : 0), there);
      }
    } else {
      uint4 x[N * kVecs / 256];
#pragma unroll
      for (int u = 0; u < N * kVecs / 256; ++u) {
        const int i = u * 256 + tid, r = i / kVecs, c = (i % kVecs) * VW, e = e0 + r;
        const T* from = e < t.n4 ? s4 : e < t.n4 + t.n128 ? s128 : sraw;
        x[u] = make_uint4(0u, 0u, 0u, 0u);
        if (at[r] >= 0 && c < d) x[u] = ld16(from + at[r] * d + c);
      }
#pragma unroll
      for (int u = 0; u < N * kVecs / 256; ++u) {
        const int i = u * 256 + tid, r = i / kVecs, c = (i % kVecs) * VW;
        float f[VW];
        cvt16(x[u], (T*)nullptr, f);
#pragma unroll
        for (int k = 0; k < VW; k += 4)
          *reinterpret_cast<float4*>(&to[r][c + k]) = make_float4(f[k], f[k + 1], f[k + 2], f[k + 3]);
      }
    }
    copies_close();
  };
  fetch(sm.k, c4K, c128K, rawK, e_lo, sm.at[0]);
  int parity = 0;
  for (int e0 = e_lo; e0 < e_hi; e0 += N, parity ^= 1) {
    // V's rows arrive while the logits are formed, the next K rows while O is
    fetch(sm.v, c4V, c128V, rawV, e0, sm.at[parity]);
    if (tid < N) sm.at[parity ^ 1][tid] = locate(e0 + N + tid);
    copies_wait<1>();
    __syncthreads();
    // logits: rows ty + 16 i, entries tx + 16 j
    float s[RI][EI];
#pragma unroll
    for (int i = 0; i < RI; ++i)
#pragma unroll
      for (int j = 0; j < EI; ++j) s[i][j] = 0.f;
#pragma unroll 4
    for (int c = 0; c < DM; c += 4) {
      float4 x[RI], y[EI];
#pragma unroll
      for (int i = 0; i < RI; ++i) x[i] = *reinterpret_cast<const float4*>(&sm.q[ty + 16 * i][c]);
#pragma unroll
      for (int j = 0; j < EI; ++j) y[j] = *reinterpret_cast<const float4*>(&sm.k[tx + 16 * j][c]);
#pragma unroll
      for (int i = 0; i < RI; ++i)
#pragma unroll
        for (int j = 0; j < EI; ++j) {
          s[i][j] = fmaf(x[i].x, y[j].x, s[i][j]);
          s[i][j] = fmaf(x[i].y, y[j].y, s[i][j]);
          s[i][j] = fmaf(x[i].z, y[j].z, s[i][j]);
          s[i][j] = fmaf(x[i].w, y[j].w, s[i][j]);
        }
    }
#pragma unroll
    for (int i = 0; i < RI; ++i) {
      float top = m[i];
#pragma unroll
      for (int j = 0; j < EI; ++j) {
        const int e = e0 + tx + 16 * j;
        const bool seen = e < e_hi && (e < t.n4              ? e < lim4[i]
                                       : e < t.n4 + t.n128 ? e < lim128[i]
                                                             : e >= lo[i] && e <= hi[i]);
        s[i][j] = seen ? s[i][j] : -INFINITY;
        top = fmaxf(top, s[i][j]);
      }
#pragma unroll
      for (int w = 8; w > 0; w >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, w));
      const float base = top == -INFINITY ? 0.f : top;   // (nothing seen yet)
      const float alpha = exp2f(m[i] - base);
      m[i] = top;
      float sum = 0.f;
#pragma unroll
      for (int j = 0; j < EI; ++j) {
        const float e = exp2f(s[i][j] - base);
        sum += e;
        sm.p[ty + 16 * i][tx + 16 * j] = e;
      }
      l[i] = l[i] * alpha + sum;   // (this thread's entries only)
#pragma unroll
      for (int c = 0; c < CI; ++c) {
        o[i][c].x *= alpha;
        o[i][c].y *= alpha;
        o[i][c].z *= alpha;
        o[i][c].w *= alpha;
      }
    }
    copies_wait<0>();
    __syncthreads();
    if (e0 + N < e_hi) fetch(sm.k, c4K, c128K, rawK, e0 + N, sm.at[parity ^ 1]);
    // O: columns 4 tx + 64 c
#pragma unroll 2
    for (int e = 0; e < N; e += 4) {
      float4 x[RI];
#pragma unroll
      for (int i = 0; i < RI; ++i) x[i] = *reinterpret_cast<const float4*>(&sm.p[ty + 16 * i][e]);
#pragma unroll
      for (int k = 0; k < 4; ++k)
#pragma unroll
        for (int c = 0; c < CI; ++c) {
          const float4 y = *reinterpret_cast<const float4*>(&sm.v[e + k][4 * tx + 64 * c]);
#pragma unroll
          for (int i = 0; i < RI; ++i) {
            const float w = k == 0 ? x[i].x : k == 1 ? x[i].y : k == 2 ? x[i].z : x[i].w;
            o[i][c].x = fmaf(w, y.x, o[i][c].x);
            o[i][c].y = fmaf(w, y.y, o[i][c].y);
            o[i][c].z = fmaf(w, y.z, o[i][c].z);
            o[i][c].w = fmaf(w, y.w, o[i][c].w);
          }
        }
    }
    __syncthreads();
  }
#pragma unroll
  for (int i = 0; i < RI; ++i) {
    float sum = l[i];
#pragma unroll
    for (int w = 8; w > 0; w >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, w);
    const int r = ty + 16 * i;
    if (r >= t.rows) continue;
    const int64_t row = t.row0 + r;
    if (t.shares == 1) {
      const float inv = 1.f / sum;
#pragma unroll
      for (int c = 0; c < CI; ++c)
        if (4 * tx + 64 * c < d)
          store_f4(O + row * d + 4 * tx + 64 * c,
                   make_float4(o[i][c].x * inv, o[i][c].y * inv, o[i][c].z * inv, o[i][c].w * inv));
      if (tx == 0) a.lse[row] = (m[i] + log2f(sum)) * 0.6931471805599453f;
    } else {
      float* part = a.part + (row * a.n_chunks + blockIdx.y) * (d + 4);
#pragma unroll
      for (int c = 0; c < CI; ++c)
        if (4 * tx + 64 * c < d) *reinterpret_cast<float4*>(part + 4 * tx + 64 * c) = o[i][c];
      if (tx == 0) {
        part[d] = m[i];
        part[d + 1] = sum;
      }
    }
  }
}

// Joins the shares of a slot's rows: grid (slots, R / 8), a warp per row.
template <typename T>
__global__ void __launch_bounds__(256) chunk_simt_merge_kernel(ChunkAttnArgs a, int R, T* O) {
  const int lane = threadIdx.x & 31, d = a.d, r = 8 * blockIdx.y + (threadIdx.x >> 5);
  pdl_wait();
  pdl_launch_dependents();
  const RowTile t = row_tile(a, R, blockIdx.x);
  if (t.shares == 1 || r >= t.rows) return;
  const int64_t row = t.row0 + r;
  const int pitch = d + 4;
  const float* pr = a.part + row * a.n_chunks * pitch;
  // lane i weighs shares i and i + 32 (there are 64 at most)
  float m[2], l[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int c = min(lane + 32 * h, t.shares - 1);
    const float2 ml = *reinterpret_cast<const float2*>(pr + c * pitch + d);
    m[h] = lane + 32 * h < t.shares ? ml.x : -INFINITY;
    l[h] = ml.y;
  }
  const float M = warp_max(fmaxf(m[0], m[1]));
  float f[2] = {exp2f(m[0] - M), exp2f(m[1] - M)};
  const float sum = warp_sum(f[0] * l[0] + f[1] * l[1]), inv = 1.f / sum;
  __shared__ float weights[8][64];   // (lanes past d leave the column loop)
  float* weight = weights[threadIdx.x >> 5];
  weight[lane] = f[0];
  weight[lane + 32] = f[1];
  __syncwarp();
  for (int i = 4 * lane; i < d; i += 128) {
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 8
    for (int c = 0; c < t.shares; ++c) {
      const float w = weight[c];
      const float4 v = *reinterpret_cast<const float4*>(pr + c * pitch + i);
      acc = make_float4(fmaf(w, v.x, acc.x), fmaf(w, v.y, acc.y), fmaf(w, v.z, acc.z),
                        fmaf(w, v.w, acc.w));
    }
    store_f4(O + row * d + i, make_float4(acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv));
  }
  if (lane == 0) a.lse[row] = (M + log2f(sum)) * 0.6931471805599453f;
}

// Rows per CTA: 16 for batches whose requests have few rows on average, else as many as O's register
// tile allows.
static int simt_rows(const tv_shape* s, int n_new) {
  if ((int64_t)n_new * s->H <= 24 * (int64_t)s->B) return 16;
  return s->d > 256 ? 32 : 64;
}
static int64_t simt_slots(const tv_shape* s, int n_new) {
  return (int64_t)n_new * s->H / simt_rows(s, n_new) + s->B;
}
// Shares of an item's entries: enough CTAs with work that they even out over the SMs, up to the shares
// of a full cache.  Small tiles take many rounds of CTAs (at most one slot in two holds an item when every
// request has a token): 100 requests of one token, d = 64, 142 us with 2 CTAs with work per SM, 103 with
// 6, 85 with 10, 82 with 16.  Large ones fill the SMs about once, counted with the slots, of which a few
// hold nothing: 480 fp32 rows of d = 64 in each of 6 requests 56 us with 6 shares, 70 with 7, which start
// a second round; d = 512 (32 rows), 7 requests of 1600 rows, 2410 us with 2 CTAs per SM, 2101 with 3.
constexpr int kMostShares = 64;
constexpr int share_ctas(int R) { return 152 * (R == 16 ? 10 : R == 32 ? 3 : 2); }
static int simt_chunks(const tv_shape* s, int n_new) {
  const int R = simt_rows(s, n_new), ctas = share_ctas(R);
  int64_t items = (int64_t)n_new * s->H / R;
  if (R > 16)
    items += s->B;
  else if (items < s->B)
    items = s->B;
  int64_t entries = (s->tail_mode == TV_TAIL_WINDOW ? s->W : 128) + 64;
  if (s->comp_mask & TV_COMP_C4) entries += s->c4_cap;
  if (s->comp_mask & TV_COMP_C128) entries += s->c128_cap;
  int64_t n = (ctas + items - 1) / items;
  if (n > (entries + kShare - 1) / kShare) n = (entries + kShare - 1) / kShare;
  return (int)(n < 1 ? 1 : n > kMostShares ? kMostShares : n);
}

template <typename T, int R, int N, int DM>
static cudaError_t launch_simt(const ChunkAttnArgs& a, int64_t slots, const void* Q,
                               const void* c4K, const void* c4V, const void* c128K,
                               const void* c128V, const void* rawK, const void* rawV, void* O,
                               cudaStream_t stream) {
  const int smem = (int)sizeof(SimtTile<T, R, N, DM>);
  const cudaError_t e = allow_smem<chunk_simt_kernel<T, R, N, DM>>(smem);
  if (e != cudaSuccess) return e;
  return launch_pdl(chunk_simt_kernel<T, R, N, DM>, dim3((unsigned)slots, a.n_chunks), dim3(256), smem,
                    stream, a, (const T*)Q, (const T*)c4K, (const T*)c4V, (const T*)c128K,
                    (const T*)c128V, (const T*)rawK, (const T*)rawV, (T*)O);
}

template <typename T>
static int launch_chunk_attn(const ChunkAttnArgs& a, int R, int64_t slots, const void* Q,
                             const void* c4K, const void* c4V, const void* c128K,
                             const void* c128V, const void* rawK, const void* rawV, void* O,
                             cudaStream_t stream) {
#define TV_SIMT(R_, N_, DM_) \
  launch_simt<T, R_, N_, DM_>(a, slots, Q, c4K, c4V, c128K, c128V, rawK, rawV, O, stream)
  cudaError_t e;
  if (R == 16)
    e = a.d <= 64    ? TV_SIMT(16, 64, 64)
        : a.d <= 128 ? TV_SIMT(16, 64, 128)
        : a.d <= 256 ? TV_SIMT(16, 32, 256)
                     : TV_SIMT(16, 32, 512);
  else
    e = a.d <= 64    ? TV_SIMT(64, 64, 64)
        : a.d <= 128 ? TV_SIMT(64, 64, 128)
        : a.d <= 256 ? TV_SIMT(64, 32, 256)
                     : TV_SIMT(32, 32, 512);
#undef TV_SIMT
  if (e == cudaSuccess && a.n_chunks > 1)
    e = launch_pdl(chunk_simt_merge_kernel<T>, dim3((unsigned)slots, R / 8), dim3(256), 0, stream, a, R,
                   (T*)O);
  if (e != cudaSuccess) {
    cudaGetLastError();
    return tv_set_error(TV_ERR_CUDA, "tv_chunk_attn: launch failed: %s", cudaGetErrorString(e));
  }
  return TV_OK;
}

}  // namespace tv

// Shares s <= ctas / items + 1 with items <= ctas where s > 1, and rows <= R (items + 1), so rows times
// shares are at most R (ctas + items + s) <= R (2 ctas + 64), for every R that n_new or fewer tokens
// may give.
size_t tv_chunk_simt_workspace(const tv_shape* s, int n_new) {
  const int R = s->d > 256 ? 32 : 64;
  const auto bound = [](int R) { return (int64_t)R * (2 * tv::share_ctas(R) + tv::kMostShares); };
  const int64_t rows = (int64_t)n_new * s->H * tv::kMostShares;
  const int64_t most = bound(16) > bound(R) ? bound(16) : bound(R);
  return (size_t)(rows < most ? rows : most) * (s->d + 4) * sizeof(float);
}

int tv_launch_chunk_attn(const tv_shape* s, int n_new, const int32_t* starts, const void* Q,
                         const void* c4K, const void* c4V, const void* c128K, const void* c128V,
                         const void* rawK, const void* rawV, const int32_t* L, float scale,
                         void* O, float* lse, void* workspace, int32_t* status,
                         cudaStream_t stream) {
  const tv::ChunkAttnArgs a = {tv::chunk_of(s, n_new, starts, L), s->H, s->d, s->W, s->tail_mode,
                               tv::simt_chunks(s, n_new), scale * 1.4426950408889634f, lse,
                               (float*)workspace, status};
  const int R = tv::simt_rows(s, n_new);
  const int64_t slots = tv::simt_slots(s, n_new);
  return s->dtype == TV_BF16
             ? tv::launch_chunk_attn<__nv_bfloat16>(a, R, slots, Q, c4K, c4V, c128K, c128V, rawK,
                                                    rawV, O, stream)
             : tv::launch_chunk_attn<float>(a, R, slots, Q, c4K, c4V, c128K, c128V, rawK, rawV, O,
                                            stream);
}

// New tokens into the persistent cache: rows rotated by position, entries of completed blocks,
// lengths ("Adapting Tree-Structured Speculative Decoding to DeepSeek-V4 for Efficient Inference"
// §2.2: online compression of the sequence as it grows; §4.2: the cache's three layers).
//
// Keys and values: one cluster of eight CTAs per 128-position block with new tokens; CTA r owns its
// positions 16r .. 16r + 15.  It brings its new rows (and, for blocks that complete, the committed ones
// in front) into shared memory, rotates the new keys there, stores them, and forms the entries of the
// four C4 blocks it holds; a completed C128 block is joined over the cluster by the routine that
// prefill runs.  So every row is read once and entries depend on the stored rows alone.  Queries
// are rotated on the way from memory to memory.  Both are bound by HBM: 4 d es bytes per token and
// 2 H d es for its queries.  Measured, bf16, d = 512, 64 heads: 16384 tokens 363 us (328 at the rate of a
// copy), 41 of them keys, values and entries, whose exponentials, sums and cluster barriers take four
// times the bytes' 10 us; one token of 64 requests 13 us, of one request 6 us on the GPU, less than the
// 20 us that a call from Python takes.
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

template <typename T>
struct Layers {
  const float* g4;
  const float* g128;
  T *rawK, *rawV, *c4K, *c4V, *c128K, *c128V;
};

// Request b from its starts and length: 0, or the error that leaves it as it was.  The threads
// first, first + step, ... look at a page each; the caller joins what they found.
__device__ __forceinline__ int append_state(const Chunk& c, int b, int lo, int hi, int L, int first,
                                            int step) {
  if (lo < 0 || hi < lo || hi > c.n_new) return TV_ERR_ARG;
  const int n = hi - lo;
  if (n == 0) return TV_OK;
  if (L < 0) return TV_ERR_ARG;
  if (!chunk_fits(c, (int64_t)L + n)) return TV_ERR_CAPACITY;
  if (c.pg.page_tokens != 0)
    for (int g = L / c.pg.page_tokens + first; g <= (L + n - 1) / c.pg.page_tokens; g += step) {
      const int32_t page = c.pg.table[(int64_t)b * c.pg.max_pages + g];
      if (page < 0 || page >= c.pg.n_pool_pages) return TV_ERR_ARG;
    }
  return TV_OK;
}

// cos and sin of position * f: the angle in turns and its fraction in fp64 (an fp32 angle of 2^16
// radians is off by 2^-9), the functions of the fraction in fp32.
__device__ __forceinline__ float2 turn_of(int position, float f) {
  const double turns = (double)position * ((double)f * 0.15915494309189533577);
  float2 cs;
  sincospif(2.f * (float)(turns - rint(turns)), &cs.y, &cs.x);
  return cs;
}

__device__ __forceinline__ void rotate(float2 cs, float& x, float& y) {
  const float u = x * cs.x - y * cs.y, v = x * cs.y + y * cs.x;
  x = u;
  y = v;
}

// The elements of rotated pair i among the last r of d.
__device__ __forceinline__ int2 pair_of(const AppendArgs& a, int i) {
  const int first = a.d - a.rope;
  return a.pairs == TV_ROPE_PAIRS ? make_int2(first + 2 * i, first + 2 * i + 1)
                                  : make_int2(first + i, first + i + a.rope / 2);
}

template <typename T>
__device__ __forceinline__ uint4 pack16(const float* f);
template <>
__device__ __forceinline__ uint4 pack16<float>(const float* f) {
  return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]),
                    __float_as_uint(f[3]));
}
template <>
__device__ __forceinline__ uint4 pack16<__nv_bfloat16>(const float* f) {
  uint32_t w[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(f[2 * k], f[2 * k + 1]);
    w[k] = *reinterpret_cast<const uint32_t*>(&h);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// ---- queries ---------------------------------------------------------------------------------------
// Rows (token, head) row0 .. row1 - 1 of Q into Qr by one CTA; pos[i]: position of token t0 + i, -1:
// its rows are left alone; table: room for the tokens' cosines and sines.  Work items of two 16-byte
// vectors: a vector of the first halves of the rotated elements with its partner, or two vectors that
// need no partner (interleaved pairs lie in one vector); all of a thread's loads are in flight before
// its stores.  Qr may be Q (each item is read before it is written); then only rotated vectors move.
template <typename T, int U>
__device__ void turn_rows(const AppendArgs& a, const T* Q, T* Qr, int row0, int row1, int t0,
                          const int* pos, float2* table) {
  constexpr int VW = VecWidth<T>::n;
  const int half = a.rope / 2, first = a.d - a.rope, tid = threadIdx.x;
  const int tokens = (row1 - 1) / a.H - t0 + 1;
  const bool move = Q != Qr;
  const bool pairs = a.pairs == TV_ROPE_PAIRS;
  // halves whose vectors do not fall on 16 bytes: element by element
  const bool odd = !pairs && half % VW != 0;
  const int joined = pairs || odd ? 0 : half / VW;          // items of a vector and its partner
  const int skip = move ? 0 : pairs ? first / VW : odd ? a.d / VW : first / VW;   // vectors left out
  const int alone = a.d / VW - skip - 2 * joined;           // vectors without a partner
  const int per_row = (alone + 1) / 2 + joined;
  const int items = (row1 - row0) * per_row;
  const int near = (alone + 1) / 2;
  bool ready = false;
#pragma unroll 1
  for (int base = 0; base == 0 || base < items; base += U * blockDim.x) {
    uint4 x[U][2];
    int64_t at[U];    // first vector, -1: none
    int gap[U];       // distance of the second, 0: none
    int tok[U], e0[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int i = base + u * (int)blockDim.x + tid;
      at[u] = -1;
      gap[u] = 0;
      if (i >= items) continue;
      const int r = i / per_row, j = i - r * per_row;
      const int row = row0 + r;
      tok[u] = row / a.H - t0;
      if (pos[tok[u]] < 0) continue;
      const int v = j < near ? skip + j : first / VW + (j - near);
      gap[u] = j < near ? (j + near < alone ? near : 0) : joined;
      e0[u] = v * VW;
      at[u] = (int64_t)row * a.d + e0[u];
      x[u][0] = *reinterpret_cast<const uint4*>(Q + at[u]);
      if (gap[u]) x[u][1] = *reinterpret_cast<const uint4*>(Q + at[u] + gap[u] * VW);
    }
    if (!ready) {   // the angles, while the first rows are on their way
      for (int k = tid; k < tokens * half; k += blockDim.x) {
        const int p = pos[k / half];
        if (p >= 0) table[k] = turn_of(p, a.inv_freq[k % half]);
      }
      __syncthreads();
      ready = true;
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (at[u] < 0) continue;
      const float2* cs = table + tok[u] * half;
      float f[2][VW];
      const bool whole = joined > 0 && e0[u] >= first;
      if (whole) {
        cvt16(x[u][0], (T*)nullptr, f[0]);
        cvt16(x[u][1], (T*)nullptr, f[1]);
#pragma unroll
        for (int k = 0; k < VW; ++k) rotate(cs[e0[u] - first + k], f[0][k], f[1][k]);
        x[u][0] = pack16<T>(f[0]);
        x[u][1] = pack16<T>(f[1]);
      } else if (pairs) {
#pragma unroll
        for (int s = 0; s < 2; ++s) {
          const int e = e0[u] + s * gap[u] * VW;
          if (e + VW <= first || (s && !gap[u])) continue;
          cvt16(x[u][s], (T*)nullptr, f[0]);
#pragma unroll
          for (int k = 0; k < VW; k += 2)
            if (e + k >= first) rotate(cs[(e + k - first) / 2], f[0][k], f[0][k + 1]);
          x[u][s] = pack16<T>(f[0]);
        }
      }
      *reinterpret_cast<uint4*>(Qr + at[u]) = x[u][0];
      if (gap[u]) *reinterpret_cast<uint4*>(Qr + at[u] + gap[u] * VW) = x[u][1];
    }
  }
  if (odd) {
    __syncthreads();   // (the copies of these elements above are overwritten)
    for (int i = tid; i < (row1 - row0) * half; i += blockDim.x) {
      const int row = row0 + i / half, k = i % half, t = row / a.H - t0;
      if (pos[t] < 0) continue;
      const int2 e = pair_of(a, k);
      const int64_t at = (int64_t)row * a.d;
      float u = load_f(Q + at + e.x), v = load_f(Q + at + e.y);
      rotate(table[t * half + k], u, v);
      store_f(Qr + at + e.x, u);
      store_f(Qr + at + e.y, v);
    }
  }
}

// The same where the rows go elsewhere and a rotated vector's partner lies in the same warp: interleaved
// pairs (the vector itself), or halves of a power of two of vectors at a multiple of their length.  Eight
// neighbouring vectors apart per thread, copied or rotated as they come; less code and half the registers.
template <typename T>
__host__ __device__ __forceinline__ bool streams(const AppendArgs& a) {
  constexpr int VW = VecWidth<T>::n;
  if (a.rope == 0 || a.pairs == TV_ROPE_PAIRS) return true;
  const int half = a.rope / 2 / VW;   // vectors
  return a.rope % (2 * VW) == 0 && half <= 16 && (half & (half - 1)) == 0 && (a.d / VW) % (2 * half) == 0;
}

// positions() fills pos; it runs while the first rows are on their way.
template <typename T, typename F>
__device__ void stream_rows(const AppendArgs& a, const T* Q, T* Qr, int row0, int row1, int t0,
                            const int* pos, float2* table, F&& positions) {
  constexpr int VW = VecWidth<T>::n, U = 4;
  const int per_row = a.d / VW, half = a.rope / 2, first = a.d - a.rope, tid = threadIdx.x;
  const int n = (row1 - row0) * per_row, tokens = (row1 - 1) / a.H - t0 + 1;
  const int apart = a.pairs == TV_ROPE_PAIRS ? 0 : half / VW;   // lanes to the partner
  const T* const from = Q + (int64_t)row0 * a.d;
  T* const to = Qr + (int64_t)row0 * a.d;
#pragma unroll 1
  for (int base = 0; base < n; base += U * blockDim.x) {
    uint4 x[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int i = base + u * (int)blockDim.x + tid;
      if (i < n) x[u] = *reinterpret_cast<const uint4*>(from + (int64_t)i * VW);
    }
    if (base == 0) {
      positions();
      for (int k = tid; k < tokens * half; k += blockDim.x) {
        const int p = pos[k / half];
        if (p >= 0) table[k] = turn_of(p, a.inv_freq[k % half]);
      }
      __syncthreads();
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int i = base + u * (int)blockDim.x + tid;
      const int r = i / per_row, e = (i - r * per_row) * VW;
      const int t = i < n ? (row0 + r) / a.H - t0 : 0;
      const bool live = i < n && pos[t] >= 0;
      if (__any_sync(0xffffffffu, live && e + VW > first)) {
        const float2* cs = table + t * half;
        float f[VW];
        if (apart == 0) {
          if (live && e + VW > first) {
            cvt16(x[u], (T*)nullptr, f);
#pragma unroll
            for (int k = 0; k < VW; k += 2)
              if (e + k >= first) rotate(cs[(e + k - first) / 2], f[k], f[k + 1]);
            x[u] = pack16<T>(f);
          }
        } else {
          uint4 y;
          y.x = __shfl_xor_sync(0xffffffffu, x[u].x, apart);
          y.y = __shfl_xor_sync(0xffffffffu, x[u].y, apart);
          y.z = __shfl_xor_sync(0xffffffffu, x[u].z, apart);
          y.w = __shfl_xor_sync(0xffffffffu, x[u].w, apart);
          if (live && e >= first) {
            float g[VW];
            cvt16(x[u], (T*)nullptr, f);
            cvt16(y, (T*)nullptr, g);
            const bool second = e - first >= half;
            const float2* c = cs + (e - first) - (second ? half : 0);
#pragma unroll
            for (int k = 0; k < VW; ++k) {
              if (second) {
                rotate(c[k], g[k], f[k]);
              } else {
                rotate(c[k], f[k], g[k]);
              }
            }
            x[u] = pack16<T>(f);
          }
        }
      }
      if (live) *reinterpret_cast<uint4*>(to + (int64_t)i * VW) = x[u];
    }
  }
}

// Rows per CTA.  Streams of more than four waves take four times as many, and an ordinary launch:
// starting beside the keys' and values' CTAs, they stay slow after those have gone (16384 tokens of 64 heads
// behind 41 us of keys and values: 411 us, 365 one after the other, of which this kernel is 324, 6.6
// TB/s).  Shorter ones gain by it (10 requests of 32 heads, 38 MB of queries, 33 -> 25 us; in place 16384
// tokens take 113 us one after the other).
constexpr int kTurnRows = 32, kLongRows = 128, kTurnTokens = kTurnRows + 1;

constexpr int kCachedStarts = 1024;   // requests whose starts are searched in shared memory

// The starts, copied into shared memory where there is room for them.
__device__ __forceinline__ const int32_t* cached_starts(const Chunk& c, int32_t* copy) {
  if (c.B > kCachedStarts) return c.starts;
  for (int i = threadIdx.x; i <= c.B; i += blockDim.x) copy[i] = c.starts[i];
  __syncthreads();
  return copy;
}

// (at most kTurnTokens tokens: kRows == kLongRows with 8 heads or more)
template <typename T, bool kStream, int kRows>
__global__ void __launch_bounds__(256) append_queries_kernel(AppendArgs a, const T* Q, T* Qr) {
  extern __shared__ __align__(16) unsigned char smem_raw[];
  __shared__ int32_t starts_copy[kCachedStarts + 1];
  __shared__ int pos[kTurnTokens];
  const int rows = a.c.n_new * a.H, row0 = blockIdx.x * kRows;   // < 2^31
  const int row1 = rows - row0 > kRows ? row0 + kRows : rows;
  const int t0 = row0 / a.H, tokens = (row1 - 1) / a.H - t0 + 1;
  // nothing is read that the kernel in front (keys and values) writes: it waits for what is read here,
  // and writes the caches only
  auto positions = [&] {
    const int32_t* starts = cached_starts(a.c, starts_copy);
    if ((int)threadIdx.x < tokens) {
      const int t = t0 + threadIdx.x, b = request_of(starts, a.c.B, t);
      pos[threadIdx.x] = b < 0 || starts[b] < 0 || starts[b + 1] > a.c.n_new
                             ? -1
                             : (int)max(0, a.c.L[b]) + t - starts[b];
    }
    __syncthreads();
  };
  float2* table = reinterpret_cast<float2*>(smem_raw);
  if constexpr (kStream) {
    stream_rows(a, Q, Qr, row0, row1, t0, pos, table, positions);
  } else {
    positions();
    turn_rows<T, 4>(a, Q, Qr, row0, row1, t0, pos, table);
  }
  // one CTA's wait is enough for the kernel to complete after the one in front of it
  if (blockIdx.x == gridDim.x - 1) pdl_wait();
  pdl_launch_dependents();
}

// ---- keys and values -------------------------------------------------------------------------------
template <typename T>
struct AppendSmem {
  C128Smem<T> c;
  float gate4[kMaxHeadDim];
  float z4[kC128Tokens];
};

// Block `blk` of request b, whose new tokens take positions L0 .. L1 - 1 and come from rows t0 on: this
// CTA's 16 positions.  `joined`: entries the cluster has joined so far (its receive buffers take turns);
// the first one waits for the cluster's CTAs to have started.
template <typename T>
__device__ void append_block(const AppendArgs& a, const Layers<T>& y, const T* K, const T* V, int b,
                             int blk, int t0, int L0, int L1, int rank, int& joined,
                             AppendSmem<T>& sm) {
  constexpr int VW = VecWidth<T>::n;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, d = a.d;
  const bool has4 = a.c.comp_mask & TV_COMP_C4;
  const bool whole = (a.c.comp_mask & TV_COMP_C128) && 128 * (int64_t)blk + 128 <= L1;
  const int base = 128 * blk + kC128Tokens * rank;   // < 2^30
  const int lo = max(L0, base), hi = min(L1, base + kC128Tokens);
  if (!whole && lo >= hi) return;
  // rows wanted in shared memory: all of a block that completes, else the new ones with what is in
  // front of them in their C4 block
  const int from = whole ? base : has4 ? max(base, lo & ~3) : lo;
  const int64_t first = layer_row(a.c.pg, b, base, a.c.raw_cap, 1, a.status);   // (the block's page)
  const int per_row = d / VW;
  for (int c = tid; c < (hi - from) * 2 * per_row; c += blockDim.x) {
    const int t = c / (2 * per_row), q = c - t * 2 * per_row, v = q >= per_row;
    const int p = from + t, e = (q - v * per_row) * VW;
    const T* src = p < L0 ? (v ? y.rawV : y.rawK) + (first + p - base) * d
                          : (v ? V : K) + (int64_t)(t0 + p - L0) * a.ld;
    cp_async16(&sm.c.rows[p - base][v][e], src + e);
  }
  cp_async_commit();
  // the angles of the thread's first pairs while the rows are on their way
  const int half = a.rope / 2, turns = (hi - lo) * half;
  constexpr int kEarly = 2;
  float2 early[kEarly];
#pragma unroll
  for (int k = 0; k < kEarly; ++k) {
    const int i = tid + k * kThreads;
    if (i < turns) early[k] = turn_of(lo + i / half, a.inv_freq[i % half]);
  }
  cp_async_wait(0);
  __syncthreads();
  auto turn = [&](int i, float2 cs) {
    const int2 e = pair_of(a, i % half);
    T* row = sm.c.rows[lo + i / half - base][0];
    float u = load_f(row + e.x), v = load_f(row + e.y);
    rotate(cs, u, v);
    store_f(row + e.x, u);
    store_f(row + e.y, v);
  };
#pragma unroll
  for (int k = 0; k < kEarly; ++k)
    if (tid + k * kThreads < turns) turn(tid + k * kThreads, early[k]);
  for (int i = tid + kEarly * kThreads; i < turns; i += kThreads)
    turn(i, turn_of(lo + i / half, a.inv_freq[i % half]));
  if (turns > 0) __syncthreads();
  for (int c = tid; c < (hi - lo) * 2 * per_row; c += blockDim.x) {
    const int t = c / (2 * per_row), q = c - t * 2 * per_row, v = q >= per_row;
    const int e = (q - v * per_row) * VW;
    *reinterpret_cast<uint4*>((v ? y.rawV : y.rawK) + (first + lo + t - base) * d + e) =
        *reinterpret_cast<const uint4*>(&sm.c.rows[lo + t - base][v][e]);
  }
  // C4 blocks whose last position is new: the orders of entry4
  const int g0 = (lo - base) >> 2, g1 = (hi - base) >> 2;
  if (has4 && g0 < g1) {
    for (int t = 4 * g0 + warp; t < 4 * g1; t += kWarps) {
      const float z = row_logit<T>(sm.c.rows[t][0], sm.gate4, d, lane);
      if (lane == 0) sm.z4[t] = z;
    }
    __syncthreads();
    const int64_t out = layer_row(a.c.pg, b, base / 4, a.c.c4_cap, 4, a.status) * d;
    const int np = d / 2;
    for (int i = tid; i < (g1 - g0) * np; i += kThreads) {
      const int g = g0 + i / np, p = i % np;
      const float* z = sm.z4 + 4 * g;
      const float M = fmaxf(fmaxf(z[0], z[1]), fmaxf(z[2], z[3]));
      float w[4], S = 0.f;
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        w[t] = expf(z[t] - M);
        S += w[t];
      }
      const float4 s = pair_sums<T, 4>(sm.c.rows + 4 * g, w, p);
      const int64_t at = out + (int64_t)g * d + 2 * p;
      store_f(y.c4K + at, s.x / S);
      store_f(y.c4K + at + 1, s.y / S);
      store_f(y.c4V + at, s.z / S);
      store_f(y.c4V + at + 1, s.w / S);
    }
  }
  if (whole) {
    if (joined == 0) asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
    const int64_t out = layer_row(a.c.pg, b, blk, a.c.c128_cap, 128, a.status) * d;
    entry128<T>(d, sm.c.gate128, y.c128K + out, y.c128V + out, joined & 1, sm.c, [] {});
    ++joined;
  } else {
    __syncthreads();
  }
}

template <typename T>
__device__ __forceinline__ void load_gates(const AppendArgs& a, const Layers<T>& y, AppendSmem<T>& sm) {
  for (int i = threadIdx.x; i < a.d; i += blockDim.x) {
    if (a.c.comp_mask & TV_COMP_C4) sm.gate4[i] = y.g4[i];
    if (a.c.comp_mask & TV_COMP_C128) sm.c.gate128[i] = y.g128[i];
  }
}

// Many tokens: a cluster per slot of a 128-block.  Request b's blocks take the slots from
// floor(starts[b] / 128) + 2b on: its n tokens touch at most floor(n / 128) + 2 blocks, so requests
// stay apart and a slot's request is found by a search of the starts.
__device__ __forceinline__ int slot_of(int start, int b) { return start / 128 + 2 * b; }

// Whether that search finds request b for each of its slots, which starts that descend elsewhere may
// prevent: the searches for all of them take the way to b if its steps at or below b lie at or below b's first
// slot and those above b behind its last one.  Lane i looks at the i-th step, request step_to(); -1: there
// is none.
__device__ __forceinline__ int step_to(int B, int b, int lane) {
  int lo = 0, hi = B, at = -1;
  for (int step = 0; lo < hi; ++step) {
    const int mid = (lo + hi) >> 1;
    if (step == lane) at = mid;
    if (mid <= b)
      lo = mid + 1;
    else
      hi = mid;
  }
  return at;
}
__device__ __forceinline__ bool step_holds(int at, int start_at, int b, int start, int n, int L) {
  const int first = slot_of(start, b), last = first + (L % 128 + n - 1) / 128;
  return at < 0 || (at <= b ? slot_of(start_at, at) <= first : slot_of(start_at, at) > last);
}

template <typename T>
__global__ void __cluster_dims__(kC128Ranks, 1, 1) __launch_bounds__(kThreads)
    append_blocks_kernel(AppendArgs a, Layers<T> y, const T* K, const T* V) {
  extern __shared__ __align__(16) unsigned char smem_raw[];
  AppendSmem<T>& sm = *reinterpret_cast<AppendSmem<T>*>(smem_raw);
  __shared__ int32_t starts_copy[kCachedStarts + 1];
  pdl_wait();
  pdl_launch_dependents();
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
  const int slot = blockIdx.x / kC128Ranks, rank = blockIdx.x % kC128Ranks;
  const int32_t* starts = cached_starts(a.c, starts_copy);
  int lo = 0, hi = a.c.B;
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (slot_of(starts[mid], mid) <= slot)
      lo = mid + 1;
    else
      hi = mid;
  }
  const int b = lo - 1;
  int joined = 0;
  if (b >= 0) {
    const int s0 = starts[b], s1 = starts[b + 1], L0 = a.c.L[b];
    const int state = append_state(a.c, b, s0, s1, L0, threadIdx.x, kThreads);
    const int at = step_to(a.c.B, b, threadIdx.x & 31);
    const bool good = !__syncthreads_or(state != TV_OK ||
                                        !step_holds(at, starts[max(at, 0)], b, s0, s1 - s0, L0));
    const int blk = L0 / 128 + slot - slot_of(s0, b);
    if (good && s1 > s0 && (int64_t)128 * blk < L0 + (s1 - s0)) {
      load_gates(a, y, sm);
      append_block(a, y, K, V, b, blk, s0, L0, L0 + (s1 - s0), rank, joined, sm);
    }
  }
  if (joined == 0) asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// Few tokens: a cluster per request does all of it, its queries and its length included.  (Four CTAs per
// SM: 64 requests' 512 CTAs are resident at once.)
template <typename T>
__global__ void __cluster_dims__(kC128Ranks, 1, 1) __launch_bounds__(kThreads, 4)
    append_requests_kernel(AppendArgs a, Layers<T> y, const T* K, const T* V, const T* Q, T* Qr) {
  extern __shared__ __align__(16) unsigned char smem_raw[];
  AppendSmem<T>& sm = *reinterpret_cast<AppendSmem<T>*>(smem_raw);
  __shared__ int pos[kTurnTokens];
  const int b = blockIdx.x / kC128Ranks, rank = blockIdx.x % kC128Ranks;
  pdl_wait();
  pdl_launch_dependents();
  const int s0 = a.c.starts[b], s1 = a.c.starts[b + 1], L0 = a.c.L[b];
  int joined = 0;
  const int found = append_state(a.c, b, s0, s1, L0, threadIdx.x, kThreads);
  // (a missing page is found by some threads only, all else by every one)
  const int code = __syncthreads_or(found == TV_ERR_ARG) ? TV_ERR_ARG : found;
  // every CTA of the cluster has read the length
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
  const int n = s1 - s0, L1 = L0 + n;
  if (code == TV_OK && n > 0) {
    // the rank of the first new position begins with keys and values, the others with the queries
    const int kv = L0 % 128 / kC128Tokens;
    load_gates(a, y, sm);
    for (int blk = L0 / 128; blk <= (L1 - 1) / 128; ++blk)
      append_block(a, y, K, V, b, blk, s0, L0, L1, rank, joined, sm);
    if (Q != nullptr && rank != kv) {
      float2* table = reinterpret_cast<float2*>(smem_raw);   // (over the rows)
      // (rows of this path: few, n_new <= 2B)
      const int end = s1 * a.H, step = kTurnRows / 2;
      for (int r0 = s0 * a.H + ((rank - kv - 1) & 7) * step; r0 < end; r0 += (kC128Ranks - 1) * step) {
        const int r1 = min(end, r0 + step), t0 = r0 / a.H;
        __syncthreads();
        if (threadIdx.x < kTurnTokens) pos[threadIdx.x] = L0 + t0 + (int)threadIdx.x - s0;
        __syncthreads();
        turn_rows<T, 2>(a, Q, Qr, r0, r1, t0, pos, table);
      }
    }
  }
  if (joined == 0) asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
  if (rank == 0 && threadIdx.x == 0) {
    if (code != TV_OK)
      record_error(a.status, code);
    else if (n > 0)
      a.c.L[b] = L1;
  }
}

// The lengths advance once everything that reads them is done, of the requests whose blocks were found; errors
// are recorded here.  A warp per request.
__global__ void append_lengths_kernel(AppendArgs a) {
  const int b = blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5), lane = threadIdx.x & 31;
  if (b >= a.c.B) {
    pdl_wait();
    return;
  }
  // (nothing is read that the call's kernels in front write; they have waited for those in front of them)
  const int at = step_to(a.c.B, b, lane), start_at = a.c.starts[max(at, 0)];
  const int s0 = a.c.starts[b], s1 = a.c.starts[b + 1], L0 = a.c.L[b];
  const int code = append_state(a.c, b, s0, s1, L0, lane, 32);
  const bool lost = s1 > s0 && !step_holds(at, start_at, b, s0, s1 - s0, L0);
  const unsigned arg = __ballot_sync(0xffffffffu, code == TV_ERR_ARG || lost);
  const int state = arg != 0 ? TV_ERR_ARG : code;
  pdl_wait();
  pdl_launch_dependents();
  if (lane != 0) return;
  if (state != TV_OK)
    record_error(a.status, state);
  else
    a.c.L[b] = L0 + (s1 - s0);
}

template <typename T>
static int launch_append(const AppendArgs& a, const Layers<T>& y, const void* K, const void* V,
                         const void* Q, void* Qr, cudaStream_t stream) {
  const char* fn = "tv_chunk_append";
  const int n = a.c.n_new, B = a.c.B;
  // room for the cosines and sines of the tokens that a CTA's rows may touch
  auto table_of = [&](int rows) {
    const int tokens = (rows - 1) / a.H + 2 < rows ? (rows - 1) / a.H + 2 : rows;
    return (size_t)tokens * (a.rope / 2) * sizeof(float2);
  };
  const size_t table = table_of(kTurnRows);
  const size_t kv = sizeof(AppendSmem<T>) > table ? sizeof(AppendSmem<T>) : table;
  constexpr int kMost = 128 * 1024;   // the most that any call takes: 32 tokens' tables are 64 KB
  static_assert(sizeof(AppendSmem<T>) <= kMost, "shared memory of the appending CTAs");
  if (allow_smem<append_blocks_kernel<T>>(kMost) != cudaSuccess ||
      allow_smem<append_requests_kernel<T>>(kMost) != cudaSuccess ||
      allow_smem<append_queries_kernel<T, true, kLongRows>>(kMost) != cudaSuccess ||
      allow_smem<append_queries_kernel<T, true, kTurnRows>>(kMost) != cudaSuccess ||
      allow_smem<append_queries_kernel<T, false, kLongRows>>(kMost) != cudaSuccess ||
      allow_smem<append_queries_kernel<T, false, kTurnRows>>(kMost) != cudaSuccess)
    return tv_check_launch(fn);
  cudaError_t e = cudaSuccess;
  // Up to two tokens per request on average: a cluster per request.  Both kernels' times, 64 heads: 64
  // requests of one token 8 us and 14 with the other kernels, of 2 10 and 16, 256 of one 19 and 35; but one request
  // of 512 tokens in a batch of 256, the others idle, 549 and 35: the host does not know how tokens are spread.
  if (n <= 2 * (int64_t)B) {
    e = launch_pdl(append_requests_kernel<T>, dim3((unsigned)B * kC128Ranks), dim3(kThreads), kv,
                   stream, a, y, (const T*)K, (const T*)V, (const T*)Q, (T*)Qr);
  } else {
    const unsigned slots = (unsigned)(n / 128 + 2 * B);
    e = launch_pdl(append_blocks_kernel<T>, dim3(slots * kC128Ranks), dim3(kThreads),
                   sizeof(AppendSmem<T>), stream, a, y, (const T*)K, (const T*)V);
    const int64_t rows = (int64_t)n * a.H;
    if (e == cudaSuccess && Q != nullptr) {
      const bool stream_q = Q != Qr && streams<T>(a);
      const bool long_q = a.H >= 8 && rows >= 16 * 152 * kLongRows;   // (four waves of CTAs)
      const int per = long_q ? kLongRows : kTurnRows;
      auto kernel = stream_q ? (long_q ? append_queries_kernel<T, true, kLongRows>
                                       : append_queries_kernel<T, true, kTurnRows>)
                             : (long_q ? append_queries_kernel<T, false, kLongRows>
                                       : append_queries_kernel<T, false, kTurnRows>);
      const dim3 grid((unsigned)((rows + per - 1) / per));
      if (long_q) {
        kernel<<<grid, 256, table_of(per), stream>>>(a, (const T*)Q, (T*)Qr);
        e = cudaPeekAtLastError();
      } else {
        e = launch_pdl(kernel, grid, dim3(256), table_of(per), stream, a, (const T*)Q, (T*)Qr);
      }
    }
    if (e == cudaSuccess)
      e = launch_pdl(append_lengths_kernel, dim3((B + 7) / 8), dim3(256), 0, stream, a);
  }
  if (e != cudaSuccess) {
    cudaGetLastError();
    return tv_set_error(TV_ERR_CUDA, "%s: launch failed: %s", fn, cudaGetErrorString(e));
  }
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
  if (s->dtype == TV_BF16) {
    using T = __nv_bfloat16;
    const tv::Layers<T> y = {g4, g128, (T*)rawK, (T*)rawV, (T*)c4K, (T*)c4V, (T*)c128K, (T*)c128V};
    return tv::launch_append<T>(a, y, K, V, Q, Qr, stream);
  }
  const tv::Layers<float> y = {g4,          g128,        (float*)rawK,  (float*)rawV,
                               (float*)c4K, (float*)c4V, (float*)c128K, (float*)c128V};
  return tv::launch_append<float>(a, y, K, V, Q, Qr, stream);
}

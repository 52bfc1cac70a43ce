// Ragged batches of new tokens, shared by tv_chunk_append and tv_chunk_attn: request b's tokens are
// rows starts[b] .. starts[b+1] - 1 of n_new.
#pragma once

#include "tv_common.cuh"

namespace tv {

struct Chunk {
  int B, n_new, comp_mask;
  int64_t raw_cap, c4_cap, c128_cap;
  Paging pg;
  const int32_t* starts;
  int32_t* L;
};

inline Chunk chunk_of(const tv_shape* s, int n_new, const int32_t* starts, const int32_t* L) {
  return {s->B, n_new, s->comp_mask, s->raw_cap, s->c4_cap, s->c128_cap, paging_of(s), starts,
          const_cast<int32_t*>(L)};
}

// The request whose rows hold row t, -1: none.  starts ascends; where it does not, the answer may be
// any request whose rows hold t, or none.
__device__ __forceinline__ int request_of(const int32_t* starts, int B, int t) {
  int lo = 0, hi = B + 1;   // the number of starts <= t lies in lo .. hi
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (starts[mid] <= t)
      lo = mid + 1;
    else
      hi = mid;
  }
  const int b = lo - 1;
  return b >= 0 && b < B && starts[b + 1] > t ? b : -1;
}

// Whether `len` tokens fit into the caches of a request.
__device__ __forceinline__ bool chunk_fits(const Chunk& c, int64_t len) {
  return len <= c.raw_cap && (!(c.comp_mask & TV_COMP_C4) || len / 4 <= c.c4_cap) &&
         (!(c.comp_mask & TV_COMP_C128) || len / 128 <= c.c128_cap);
}

// What the tokens at positions p_lo .. p_hi see, as far as the last and from where the first does: C4
// entries, C128 entries, raw rows t0 .. end - 1.  align: t0 is a multiple of it, so that tiles of as many
// raw rows lie on one page each.
struct Span {
  int n4, n128, t0, end;
};

__device__ __forceinline__ Span span_of(int comp_mask, int tail_mode, int W, int p_lo, int p_hi,
                                        int align) {
  Span s;
  s.n4 = (comp_mask & TV_COMP_C4) ? p_hi / 4 : 0;
  s.n128 = (comp_mask & TV_COMP_C128) ? p_hi / 128 : 0;
  s.t0 = raw_lo_of(p_lo, tail_mode, W, m_min_of(comp_mask)) & ~(align - 1);
  s.end = p_hi + 1;
  return s;
}

// 0, or the error that leaves request b's rows alone in tv_chunk_attn.
__device__ __forceinline__ int attn_state(const Chunk& c, int b) {
  const int lo = c.starts[b], hi = c.starts[b + 1];
  if (lo < 0 || hi < lo || hi > c.n_new) return TV_ERR_ARG;
  if (hi == lo) return TV_OK;
  const int L = c.L[b];
  if (L < hi - lo) return TV_ERR_ARG;
  return chunk_fits(c, L) ? TV_OK : TV_ERR_CAPACITY;
}

}  // namespace tv

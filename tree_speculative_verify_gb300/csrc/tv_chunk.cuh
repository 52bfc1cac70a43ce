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

}  // namespace tv

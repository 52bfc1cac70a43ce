// How the chunk attention's work list is shared: arithmetic alone, for the kernel and for host compilers.
//
// A batch's items stand in one list.  An item takes kOpen places for opening it and one per half tile; of
// all places CTA c takes `share` from c * share on.  Places are counted in 64 bits: 1048576 new tokens of 64
// heads make 1.03 * 2^31 of them.
#pragma once

#include <stdint.h>

#ifdef __CUDACC__
#define TV_SHARED __host__ __device__ __forceinline__
#else
#define TV_SHARED inline
#endif

namespace tv {
namespace few {

// Places for opening an item (64 requests of one token: 61.5, 60.7, 61.2 and 64.4 us with 2, 3, 4 and 5; 19
// behind up to 1550 tokens: 26.7 with 2, 24.7 with 3 and 4) and least places of a CTA while there are CTAs
// left: a whole tile (one request of 8192 tokens: 29.2, 23.7, 25.9, 25.4 and 33.7 us with 1, 2, 3, 4 and 8),
// two while there is an item whose parts would be too many to join (4 requests of 16000 tokens: 38 us with 2,
// 32 with 4).
constexpr int kOpen = 3, kMinPlaces = 2, kLongItem = 48;

// Places of an item of so many half tiles (none: no item).
TV_SHARED int places_of(int units) { return units > 0 ? units + kOpen : 0; }

// ceil(total / ctas), for total < 2^48 - ctas and up to 2^15 CTAs: two short divisions.  (A long one is a routine of
// its own, which has to be fetched first: one request of 8192 tokens took 0.6 us more than with places of 32
// bits, 0.25 so.)
TV_SHARED int64_t even_share(int64_t total, int ctas) {
  const uint64_t n = (uint64_t)total + ctas - 1;
  const uint32_t high = (uint32_t)(n >> 16), q = high / (uint32_t)ctas, r = high - q * ctas;
  return (int64_t)q << 16 | (r << 16 | (uint32_t)(n & 0xffff)) / (uint32_t)ctas;
}

// The CTA that has place `at`.
TV_SHARED int holder_of(int64_t at, int64_t share, int ctas) {
  int lo = 0, hi = ctas;   // its number lies in lo .. hi - 1
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (mid * share <= at)
      lo = mid;
    else
      hi = mid;
  }
  return lo;
}

// Places per CTA, from those of the whole list and of its largest item (0: no items).
TV_SHARED int64_t share_of(int64_t total, int most, int ctas) {
  const int64_t least = most > kLongItem ? 2 * kMinPlaces : kMinPlaces;
  const int64_t even = even_share(total, ctas), few = least < total ? least : total;
  return even > few ? even : few;
}

// The CTAs that hold half tiles of an item of `places` places behind `before` others.
struct Piece {
  int first, ctas;
};
TV_SHARED Piece piece_of(int64_t before, int places, int64_t share, int ctas) {
  Piece p = {0, 0};
  if (places > 0) {
    p.first = holder_of(before + kOpen, share, ctas);
    p.ctas = holder_of(before + places - 1, share, ctas) - p.first + 1;
  }
  return p;
}

// A CTA's way through the list: `left` places remain; of the item at hand it has half tiles ub .. ue - 1.
struct Cut {
  int64_t left;
  int ub, ue;
  // Its first item, from place `begin` of it on.
  TV_SHARED void first(int begin, int64_t places) {
    ub = begin > kOpen ? begin - kOpen : 0;
    left = places - (begin < kOpen ? kOpen - begin : 0);
  }
  // The item behind the one at hand.
  TV_SHARED void next() {
    ub = 0;
    left -= kOpen;
  }
  // False if the last place was an item's opening.
  TV_SHARED bool take(int units) {
    ue = (int)(units < ub + left ? units : ub + left);
    left -= ue - ub;
    return ue > ub;
  }
};

}  // namespace few
}  // namespace tv

// Attention of few new tokens per request over the compressed cache (decoding), tensor cores, bf16, head
// dimensions 128, 256, 384 and 512.
//
// "Adapting Tree-Structured Speculative Decoding to DeepSeek-V4 for Efficient Inference" §2.2, §3.1:
// what a position of an ordinary causal sequence sees.
//
// 64 query rows (64 heads of one token, say) use a quarter of the rows that the tree attention's
// cluster computes, and the work is bound by reading the cache: 2 d es bytes per entry for 4 d 64
// operations.  So the products are transposed, entries and value columns in the MMA's M, rows in its N:
//   S^T = K Q^T    M = 128 entries, N = 64 rows, K = d      A = K tile, B = Q (shared memory, K-major)
//   O^T += V^T P^T M = 128 value columns (d / 128 times), N = 64, K = 128 entries
//                                                           A = V tile, B = P^T (both MN-major)
// O^T of 64 rows and 512 columns takes 256 TMEM columns, two S^T buffers 128: one CTA holds all of it,
// without a cluster, and every SM streams a share of the batch's tiles.
//
// Work is counted in half tiles (64 entries of one item; an item is 64 rows of one request), of which two
// make a tile: the batch's items stand in one list, request by request, each with kOpen places for opening it
// and one per half tile, which the CTAs share (tv_share.cuh); a share may end one item, hold whole ones
// and begin another.  An item that one CTA has whole is written at once; the others leave (O, m, l) per CTA
// in the workspace -- at most two per CTA -- which a second kernel joins in CTA order.
//
// Softmax: thread (entry, half of the rows) holds the entry's 32 logits; row maxima are reduced over
// the lanes by halving exchanges and over the four warps of a half through shared memory; a lane keeps
// its row's running maximum (raised lazily, by more than 2^8, as P in bf16 and l in fp32 allow), and the
// sums of a thread's own probabilities are only reduced at the item's end.  P is rounded to bf16, because both
// operands of an MMA have one type and V is bf16: relative errors of at most 2^-8 per entry, of either
// sign, which average out over the entries (1024 to 8192 tokens: 0.0020 of O's norm from the 64-bit
// result, 0.0017 with P in fp32, most of it O's own rounding); l sums the probabilities in fp32 as they are.
//
// Warps: 0 copies (TMA, a ring of 16 KB slots: 128 entries x 64 dimensions of K, or x 64 columns of
// V), 1 issues the MMAs, 2..9 softmax and epilogue.  Every wait is bounded as in the tree attention.
//
// Measured, d = 512, 64 heads, pages of 1024 tokens, with the gather of C128 entries in front and the join
// behind: 64 requests of 1024 to 8192 tokens, one new token each, 58 us (207 MB from memory, 28 us at the
// rate of a copy; the stream itself runs at 5 to 6 TB/s, the gather takes 5 us, finding the work 3, the
// last item's end 3, the join 5); one request of 8192 tokens 22 us, the length of the chain.  Tried and
// slower: the gather inside this kernel, C128 boxes of 8 rows straight from the pages, an L2 prefetch of
// the whole share, whole items per CTA.
#include <cuda.h>
#include <math.h>

#include "tv_attn_tc.cuh"
#include "tv_chunk.cuh"
#include "tv_share.cuh"
#include "tv_sm100.cuh"

namespace tv {
namespace few {

using namespace sm100;

constexpr int kRows = 64;          // query rows of an item
constexpr int kSmxWarps = 8;
constexpr int kThreads = 64 + 32 * kSmxWarps;
constexpr int kSlotBytes = 16384;
constexpr int kSlots = 8;          // (V slots are taken in pairs: an even number)
constexpr int kPBytes = 16384;     // P^T of a tile: 128 entries x 64 rows
constexpr float kRescaleThreshold = 8.f;   // log2 units

struct Params {
  CUtensorMap mQ, mC4K, mC4V, mC128K, mC128V, mRawK, mRawV;   // boxes of 64 rows x 64 columns
  Chunk c;
  int H, W, tail_mode;
  int64_t c128_stride;     // C128 rows per request
  bool gathered;           // pools: a page holds too few C128 entries for a box of 64, so the kernel in
                           // front copies them into the workspace, where the maps point
  float scale_log2;
  __nv_bfloat16* O;
  float* lse;
  float* part;             // [CTA][2][kRows][d + 4]: 0: an item begun before, 1: one that goes on
  int n_slots;
  Piece* pieces;           // [n_slots] of the slots' items (written by CTA 0)
  int32_t* status;
  uint64_t timeout_ns;
  int withhold_tile;       // test aid: no K copies for this tile of a segment (-1: none)
};

// An item: rows first .. of request b, its k-th, and the half tiles it takes.
struct Item {
  int b, k, row0, rows, pos0, first;
  Span s;
  int u4, u128, units;   // C4, C4 and C128, all
};

__device__ __forceinline__ Item item_of(const Params& p, int b, int k) {
  Item it;
  const int s0 = p.c.starts[b], n = p.c.starts[b + 1] - s0;
  it.b = b;
  it.k = k;
  it.first = k * kRows;
  it.row0 = s0 * p.H + it.first;
  it.rows = min(kRows, n * p.H - it.first);
  it.pos0 = p.c.L[b] - n;
  it.s = span_of(p.c.comp_mask, p.tail_mode, p.W, it.pos0 + it.first / p.H,
                 it.pos0 + (it.first + it.rows - 1) / p.H, p.c.pg.page_tokens != 0 ? 64 : 1);
  it.u4 = (it.s.n4 + 63) / 64;
  it.u128 = it.u4 + (it.s.n128 + 63) / 64;
  it.units = it.u128 + (it.s.end - it.s.t0 + 63) / 64;
  return it;
}

// (the dynamic window of a CTA is 227 KB)
template <int D>
struct __align__(1024) Smem {
  uint8_t q[D / 64][kRows * 128];
  uint8_t p[2][kPBytes];
  uint8_t ring[kSlots][kSlotBytes];
  uint64_t full[kSlots], empty[kSlots];
  uint64_t q_full, q_free;       // Q of a segment has landed; its S MMAs are done
  uint64_t s_full[2], s_free[2];
  uint64_t p_full[2];            // P_t is staged and O rescaled (one arrival per softmax warp)
  uint64_t pv_done[2];           // O += V_t P_t is complete (P_t's buffer is free)
  uint64_t o_full, o_free;       // a segment's O is complete; it has left TMEM
  uint64_t drain;
  float xmax[2][4][kRows];       // [tile parity][lane quadrant][row]: maxima, at a segment's end sums
  int64_t scan[kThreads / 32];   // places of the warps' slots
  int most[kThreads / 32];       // and the largest item
  int begin;                     // the CTA's first place in its first item
  int64_t places;                // places in all
  Item first;                    // its first item
  uint32_t tmem;
  int abort;
};

__device__ __forceinline__ int items_of(const Params& p, int b) {
  if (attn_state(p.c, b) != TV_OK) return 0;
  return (int)(((int64_t)(p.c.starts[b + 1] - p.c.starts[b]) * p.H + kRows - 1) / kRows);
}

// Slots of items: request b's start at floor(starts[b] * H / 64) + b, which leaves every request room
// for its items whatever the others have, so that a slot's item is found by a search of the starts.
__device__ __forceinline__ int slot_of(const Params& p, int b) {
  return (int)((int64_t)p.c.starts[b] * p.H / kRows) + b;
}
__device__ __forceinline__ int request_at(const Params& p, int slot) {   // -1: none
  int lo = 0, hi = p.c.B;
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (slot_of(p, mid) <= slot)
      lo = mid + 1;
    else
      hi = mid;
  }
  return lo - 1;
}

// One CTA's walk over its half tiles, the same in every warp: segments (item, half tiles ub .. ue - 1).
struct Walk : Cut {
  Item it;
  int n_items;   // of the request
  bool begun;
  template <typename S>
  __device__ Walk(const Params& p, const S& sm) {
    left = sm.places;
    if (left <= 0) return;
    it = sm.first;
    first(sm.begin, sm.places);
    n_items = -1;   // (looked up when the first item is done)
    begun = false;
  }
  __device__ bool next(const Params& p) {
    if (left <= 0) return false;
    if (begun) {
      int b = it.b, k = it.k + 1;
      if (n_items < 0) n_items = items_of(p, b);
      while (k >= n_items) {
        if (++b >= p.c.B) return false;
        n_items = items_of(p, b);
        k = 0;
      }
      it = item_of(p, b, k);
      Cut::next();
    }
    begun = true;
    return take(it.units);
  }
  __device__ bool whole() const { return ub == 0 && ue == it.units; }
};

// A tile: two neighbouring half tiles, or a last one.  Entries of a first half that is not full are
// masked, as are those past the second's, up to a multiple of 16.
struct Half {
  int kind, row0, valid;   // 0: C4, 1: C128, 2: raw; first entry, entries
};
struct Tile {
  Half first, second;
  int units, n16;          // halves; entries that the products take
};
__device__ __forceinline__ Half half_at(const Item& it, int u) {
  Half h;
  int end;
  if (u < it.u4) {
    h.kind = 0;
    h.row0 = 64 * u;
    end = it.s.n4;
  } else if (u < it.u128) {
    h.kind = 1;
    h.row0 = 64 * (u - it.u4);
    end = it.s.n128;
  } else {
    h.kind = 2;
    h.row0 = it.s.t0 + 64 * (u - it.u128);
    end = it.s.end;
  }
  h.valid = min(64, end - h.row0);
  return h;
}
__device__ __forceinline__ Tile tile_at(const Item& it, int u, int ue) {
  Tile x;
  x.units = min(2, ue - u);
  x.first = half_at(it, u);
  x.second = half_at(it, min(u + 1, ue - 1));   // (one half: the first again)
  x.n16 = (64 * (x.units - 1) + x.second.valid + 15) & ~15;
  return x;
}

// The row at which a half starts in its layer's map (64 entries from a multiple of 64 on lie on one
// page).
__device__ __forceinline__ int row_of(const Params& p, int b, const Half& h) {
  if (h.kind == 1) return (int)((int64_t)b * p.c128_stride + h.row0);
  return (int)(h.kind == 0 ? layer_row(p.c.pg, b, h.row0, p.c.c4_cap, 4, p.status)
                           : layer_row(p.c.pg, b, h.row0, p.c.raw_cap, 1, p.status));
}

template <typename S>
__device__ __forceinline__ void fail(S& sm, int32_t* status) {
  if (atomicExch(&sm.abort, 1) == 0) record_error(status, TV_ERR_TIMEOUT);
}

// ---- copies (warp 0) -------------------------------------------------------------------------------
template <int D>
__device__ void producer(const Params& p, Smem<D>& sm) {
  constexpr int kSlices = D / 64;
  const int lane = threadIdx.x & 31;
  Walk w(p, sm);
  int slot = 0, seg = 0;
  uint32_t phase = 0, issued = 0, issued_phase = 0;   // bit per slot: copied into, when last
  bool ok = true;
  auto wait = [&](uint64_t* bar, uint32_t parity) {
    if (!__all_sync(0xffffffffu, mbar_wait(bar, parity, &sm.abort, p.timeout_ns))) {
      if (lane == 0) fail(sm, p.status);
      ok = false;
    }
    return ok;
  };
  // lanes 0 and 1 copy the halves of a slot: `row` is theirs, `map` its half's
  auto load = [&](const Tile& x, int row, const CUtensorMap* map, bool issue) {
    for (int s = 0; s < kSlices; ++s) {
      if (!wait(&sm.empty[slot], phase ^ 1)) return;
      if (issue) {
        issued |= 1u << slot;
        issued_phase = (issued_phase & ~(1u << slot)) | phase << slot;
        if (lane == 0) mbar_arrive_expect_tx(&sm.full[slot], x.units * 8192);
        __syncwarp();
        if (lane < x.units) tma_load_2d(sm.ring[slot] + lane * 8192, map, 64 * s, row, &sm.full[slot]);
      }
      if (++slot == kSlots) {
        slot = 0;
        phase ^= 1;
      }
    }
  };
  auto map_of = [&](const Tile& x, bool v) {
    const int kind = lane & 1 ? x.second.kind : x.first.kind;
    return kind == 0 ? (v ? &p.mC4V : &p.mC4K) : kind == 1 ? (v ? &p.mC128V : &p.mC128K)
                                                           : (v ? &p.mRawV : &p.mRawK);
  };
  bool waited = !p.gathered;
  int queries = 0;   // segments whose Q was copied
  for (; ok && w.next(p); ++seg) {
    if (seg > 0 && !wait(&sm.q_free, (seg - 1) & 1)) break;
    queries = seg + 1;
    if (lane == 0) mbar_arrive_expect_tx(&sm.q_full, kSlices * kRows * 128);
    __syncwarp();
    if (lane < kSlices) tma_load_2d(sm.q[lane], &p.mQ, 64 * lane, w.it.row0, &sm.q_full);
    // K_0, K_1, V_0, K_2, V_1, ..: the order in which the MMAs take them; the next tile's rows are
    // looked up before this one's copies
    Tile x = tile_at(w.it, w.ub, w.ue), before = x;
    int row = row_of(p, w.it.b, lane & 1 ? x.second : x.first), before_row = row;
    for (int u = w.ub, t = 0; ok; ++t) {
      const bool more = u < w.ue;
      Tile after = x;
      int after_row = row;
      if (more && u + x.units < w.ue) {
        after = tile_at(w.it, u + x.units, w.ue);
        after_row = row_of(p, w.it.b, lane & 1 ? after.second : after.first);
      }
      if (more) {
        if (!waited && (x.first.kind == 1 || x.second.kind == 1)) {
          pdl_wait();
          waited = true;
        }
        load(x, row, map_of(x, false), t != p.withhold_tile);
      }
      if (t > 0 && ok) load(before, before_row, map_of(before, true), true);
      if (!more) break;
      u += x.units;
      before = x;
      before_row = row;
      x = after;
      row = after_row;
    }
  }
  // no copy may be in flight when the CTA exits, which only an abort can leave behind
  volatile int never = 0;
  for (int i = 0; i < kSlots; ++i)
    if (issued >> i & 1) mbar_wait(&sm.full[i], issued_phase >> i & 1, &never, p.timeout_ns / 4);
  if (queries > 0) mbar_wait(&sm.q_full, (queries - 1) & 1, &never, p.timeout_ns / 4);
}

// ---- MMAs (warp 1, lane 0) ------------------------------------------------------------------------
template <int D>
__device__ void mma(const Params& p, Smem<D>& sm) {
  constexpr int kSlices = D / 64, kBlocks = D / 128;
  const uint32_t tmem = sm.tmem, o_tmem = tmem + 256;
  const uint32_t id_s = idesc_bf16_f32(128, kRows, 0, 0), id_o = idesc_bf16_f32(128, kRows, 1, 1);
  const uint64_t ring = smem_desc_sw128(smem_u32(sm.ring[0]), 16, 1024);
  const uint64_t ring_mn = smem_desc_sw128(smem_u32(sm.ring[0]), kSlotBytes, 1024);
  const uint64_t q_desc = smem_desc_sw128(smem_u32(sm.q[0]), 16, 1024);
  const uint64_t p_desc = smem_desc_sw128(smem_u32(sm.p[0]), 16, 1024);
  Walk w(p, sm);
  int slot = 0, seg = 0;
  int64_t i = 0;   // tiles so far
  uint32_t phase = 0;
  bool ok = true;
  auto wait = [&](uint64_t* bar, uint32_t parity) {
    if (ok && !mbar_wait(bar, parity, &sm.abort, p.timeout_ns)) {
      fail(sm, p.status);
      ok = false;
    }
    return ok;
  };
  auto advance = [&] {
    if (++slot == kSlots) {
      slot = 0;
      phase ^= 1;
    }
  };
  auto add = [](uint64_t desc, uint32_t bytes) { return desc + (uint64_t)(bytes >> 4); };
  // O += V P of the i-th tile of all, the segment's t-th
  auto product_o = [&](const Tile& x, int t, int64_t i) {
    const int n_k = x.n16 / 16;
    if (!wait(&sm.p_full[i & 1], (i >> 1) & 1)) return;
    tc_fence_after();
    const uint64_t pd = add(p_desc, (i & 1) * kPBytes);
    for (int j = 0; j < kBlocks; ++j) {
      if (!wait(&sm.full[slot], phase)) return;
      if (!wait(&sm.full[slot + 1], phase)) return;
      tc_fence_after();
      const uint64_t vd = add(ring_mn, slot * kSlotBytes);
      for (int k = 0; k < n_k; ++k)
        mma1_ss(o_tmem + kRows * j, add(vd, 2048 * k), add(pd, 2048 * k), id_o, (t | k) ? 1u : 0u);
      mma1_commit(&sm.empty[slot]);
      advance();
      mma1_commit(&sm.empty[slot]);
      advance();
    }
    mma1_commit(&sm.pv_done[i & 1]);
  };
  for (; ok && w.next(p); ++seg) {
    if (!wait(&sm.q_full, seg & 1)) break;
    tc_fence_after();
    Tile before;
    int t = 0;
    for (int u = w.ub; u < w.ue && ok; ++t, ++i) {
      const Tile x = tile_at(w.it, u, w.ue);
      u += x.units;
      if (i >= 2 && !wait(&sm.s_free[i & 1], ((i - 2) >> 1) & 1)) break;
      tc_fence_after();
      for (int s = 0; s < kSlices && ok; ++s) {
        if (!wait(&sm.full[slot], phase)) break;
        tc_fence_after();
        const uint64_t kd = add(ring, slot * kSlotBytes), qd = add(q_desc, s * kRows * 128);
#pragma unroll
        for (int k = 0; k < 4; ++k)
          mma1_ss(tmem + kRows * (i & 1), add(kd, 32 * k), add(qd, 32 * k), id_s, (s | k) ? 1u : 0u);
        mma1_commit(&sm.empty[slot]);
        advance();
      }
      if (!ok) break;
      mma1_commit(&sm.s_full[i & 1]);
      if (u == w.ue) mma1_commit(&sm.q_free);
      if (t == 0 && seg > 0 && !wait(&sm.o_free, (seg - 1) & 1)) break;
      if (t > 0) product_o(before, t - 1, i - 1);
      before = x;
    }
    if (ok) product_o(before, t - 1, i - 1);
    if (!ok) break;
    mma1_commit(&sm.o_full);
  }
  // every MMA has completed before TMEM is released
  mma1_commit(&sm.drain);
  volatile int never = 0;
  mbar_wait(&sm.drain, 0, &never, p.timeout_ns / 4);
}

// ---- softmax and epilogue (warps 2..9) -------------------------------------------------------------
// Reduces x[0 .. 31] over the warp's lanes: lane i returns the result for x[i].
template <typename F>
__device__ __forceinline__ float lanes_reduce(float (&x)[32], int lane, F&& f) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const bool upper = lane & o;
#pragma unroll
    for (int j = 0; j < o; ++j) {
      const float keep = upper ? x[j + o] : x[j], send = upper ? x[j] : x[j + o];
      x[j] = f(keep, __shfl_xor_sync(0xffffffffu, send, o));
    }
  }
  return x[0];
}

__device__ __forceinline__ void half_sync(int half) {
  asm volatile("bar.sync %0, 128;" ::"r"(1 + half) : "memory");
}

template <int D>
__device__ void softmax(const Params& p, Smem<D>& sm) {
  constexpr int kBlocks = D / 128;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int quad = warp & 3, half = (warp - 2) >> 2;
  const int entry = 32 * quad + lane;
  const uint32_t tmem = sm.tmem + ((uint32_t)(32 * quad) << 16);
  const float sl2 = p.scale_log2;
  uint8_t* const line = sm.p[0] + (entry >> 3) * 1024 + (entry & 7) * 128;
  Walk w(p, sm);
  int seg = 0;
  int64_t g = 0;   // tiles so far
  // A wait that runs out sets the abort flag, after which every wait returns at once: the warps go on
  // through their barriers together and write nothing.
  bool ok = true;
  auto wait = [&](uint64_t* bar, uint32_t parity) {
    if (!__all_sync(0xffffffffu, mbar_wait(bar, parity, &sm.abort, p.timeout_ns))) {
      fail(sm, p.status);
      ok = false;
    }
  };
  // The code is run once for nothing, a tile and an epilogue, while the first copies are on their way (on
  // whatever TMEM holds, without barriers or results): fetched under load, as the second pass would find
  // it, a tile takes 7 us instead of 1.
  bool dry = true;
  if (w.left <= 0) return;
  bool waited = !p.gathered;
  for (;;) {
    Walk next = w;
    if (!next.next(p)) break;
    if (!dry) w = next;
    const Item it = next.it;
    const int ub = next.ub, ue = dry ? ub + 1 : next.ue;
    const bool whole = next.whole();
    const int my_row = 32 * half + lane;
    // the rows' tokens: row r belongs to position pos0 + (first + r) / H; one token in the common case
    const int p_first = it.pos0 + it.first / p.H;
    const int p_last = it.pos0 + (it.first + it.rows - 1) / p.H;   // (padding rows: anything)
    float m_ref = -INFINITY;
    float sum[32];
#pragma unroll
    for (int j = 0; j < 32; ++j) sum[j] = 0.f;
    for (int u = ub; u < ue;) {
      const Tile x = tile_at(it, u, ue);
      const int buf = dry ? 1 : g & 1;
      if (!dry) wait(&sm.s_full[buf], (g >> 1) & 1);
      tc_fence_after();
      float s[32];
      {
        uint32_t(&raw)[32] = reinterpret_cast<uint32_t(&)[32]>(s);
        tmem_ld32(tmem + kRows * buf + 32 * half, raw);
        tmem_wait_ld();
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0 && !dry) mbar_arrive(&sm.s_free[buf]);
      // who sees this thread's entry: positions from .. until (the warp's entries are of one half)
      const Half hf = quad >> 1 ? x.second : x.first;
      const int in_half = entry & 63, e = hf.row0 + in_half;
      int from, until = 0x7fffffff;
      if (hf.kind == 0) {
        from = 4 * e + 4;
      } else if (hf.kind == 1) {
        from = 128 * e + 128;
      } else {
        from = e;
        until = p.tail_mode == TV_TAIL_WINDOW ? e + p.W
                                              : e / m_min_of(p.c.comp_mask) * m_min_of(p.c.comp_mask) +
                                                    m_min_of(p.c.comp_mask) - 1;
      }
      if (in_half >= hf.valid || (quad >> 1) >= x.units) from = 0x7fffffff;
      if (!(from <= p_first && p_last <= until)) {
        if (p_first == p_last || from > p_last || until < p_first) {
#pragma unroll
          for (int j = 0; j < 32; ++j) s[j] = -INFINITY;
        } else {
          int q = it.first + 32 * half, at = q / p.H, in = q - at * p.H;
          at += it.pos0;
#pragma unroll
          for (int j = 0; j < 32; ++j) {
            if (at < from || at > until) s[j] = -INFINITY;
            if (++in == p.H) {
              in = 0;
              ++at;
            }
          }
        }
      }
      float top[32];
#pragma unroll
      for (int j = 0; j < 32; ++j) top[j] = s[j];
      float mx = lanes_reduce(top, lane, [](float a, float b) { return fmaxf(a, b); });
      sm.xmax[buf][quad][my_row] = mx;
      half_sync(half);
      mx = fmaxf(fmaxf(sm.xmax[buf][0][my_row], sm.xmax[buf][1][my_row]),
                 fmaxf(sm.xmax[buf][2][my_row], sm.xmax[buf][3][my_row]));
      const float mt = mx * sl2;
      const bool grow = mt > m_ref + kRescaleThreshold;
      const float m_new = grow ? mt : m_ref;
      const float alpha = grow && m_ref != -INFINITY ? exp2f(m_ref - m_new) : 1.f;
      const bool scales = __any_sync(0xffffffffu, alpha != 1.f);
      const float shift = m_new == -INFINITY ? 0.f : -m_new;
      m_ref = m_new;
      if (scales) {
#pragma unroll
        for (int j = 0; j < 32; ++j) sum[j] *= __shfl_sync(0xffffffffu, alpha, j);
      }
      uint32_t pk[16];
#pragma unroll
      for (int j = 0; j < 32; j += 2) {
        const float p0 = ex2_approx(fmaf(s[j], sl2, __shfl_sync(0xffffffffu, shift, j)));
        const float p1 = ex2_approx(fmaf(s[j + 1], sl2, __shfl_sync(0xffffffffu, shift, j + 1)));
        sum[j] += p0;
        sum[j + 1] += p1;
        const __nv_bfloat162 h = __floats2bfloat162_rn(p0, p1);
        pk[j / 2] = *reinterpret_cast<const uint32_t*>(&h);
      }
      // the MMA of tile g - 2 has read this P buffer
      if (g >= 2) wait(&sm.pv_done[buf], ((g - 2) >> 1) & 1);
#pragma unroll
      for (int c = 0; c < 4; ++c)
        *reinterpret_cast<uint4*>(line + buf * kPBytes + (((4 * half + c) ^ (entry & 7)) << 4)) =
            make_uint4(pk[4 * c], pk[4 * c + 1], pk[4 * c + 2], pk[4 * c + 3]);
      if (scales) {
        // O of this half's rows, once it holds every earlier tile (not the segment's first: alpha is 1)
        wait(&sm.pv_done[buf ^ 1], ((g - 1) >> 1) & 1);
        tc_fence_after();
#pragma unroll 1
        for (int j = 0; j < kBlocks; ++j) {
          uint32_t r[32];
          const uint32_t col = tmem + 256 + kRows * j + 32 * half;
          tmem_ld32(col, r);
          tmem_wait_ld();
#pragma unroll
          for (int i = 0; i < 32; ++i)
            r[i] = __float_as_uint(__uint_as_float(r[i]) * __shfl_sync(0xffffffffu, alpha, i));
          tmem_st32(col, r);
        }
        tmem_wait_st();
      }
      tc_fence_before();
      fence_proxy_async_smem();   // the MMA reads P through the async proxy
      __syncwarp();
      if (lane == 0 && !dry) mbar_arrive(&sm.p_full[buf]);
      u += x.units;
      if (!dry) ++g;
    }
    // the rows' sums over the warp's entries, then over the four warps
    float l = lanes_reduce(sum, lane, [](float a, float b) { return a + b; });
    float(&part)[4][kRows] = sm.xmax[g & 1];
    part[quad][my_row] = l;
    half_sync(half);
    l = (part[0][my_row] + part[1][my_row]) + (part[2][my_row] + part[3][my_row]);
    half_sync(half);   // all have read it
    if (!dry) wait(&sm.o_full, seg & 1);
    tc_fence_after();
    if (!waited && !dry) {   // no write before the kernel in front has completed
      pdl_wait();
      waited = true;
    }
    const bool live = ok && !dry;
    const float inv = l > 0.f ? 1.f / l : 0.f;
    if (quad == 0 && my_row < it.rows && live) {
      if (whole) {
        p.lse[(int64_t)it.row0 + my_row] = (m_ref + log2f(l)) * 0.6931471805599453f;
      } else {
        float* at = p.part + (((int64_t)blockIdx.x * 2 + (ub == 0)) * kRows + my_row) * (D + 4) + D;
        at[0] = m_ref;
        at[1] = l;
      }
    }
#pragma unroll 1
    for (int j = 0; j < kBlocks; ++j) {
      uint32_t r[32];
      tmem_ld32(tmem + 256 + kRows * j + 32 * half, r);
      tmem_wait_ld();
      const int col = 128 * j + entry;   // this lane's value column
      if (whole) {
        // two columns of a row per store: neighbouring lanes exchange rows
#pragma unroll
        for (int i = 0; i < 32; i += 2) {
          const float a = __uint_as_float(r[i]) * __shfl_sync(0xffffffffu, inv, i);
          const float b = __uint_as_float(r[i + 1]) * __shfl_sync(0xffffffffu, inv, i + 1);
          const float other = __shfl_xor_sync(0xffffffffu, lane & 1 ? a : b, 1);
          const int row = 32 * half + i + (lane & 1);
          const __nv_bfloat162 h = lane & 1 ? __floats2bfloat162_rn(other, b)
                                            : __floats2bfloat162_rn(a, other);
          if (row < it.rows && live)
            *reinterpret_cast<__nv_bfloat162*>(p.O + ((int64_t)it.row0 + row) * D + (col & ~1)) = h;
        }
      } else if (live) {
        float* at = p.part + (((int64_t)blockIdx.x * 2 + (ub == 0)) * kRows + 32 * half) * (D + 4) + col;
#pragma unroll
        for (int i = 0; i < 32; ++i)
          if (32 * half + i < it.rows) at[i * (D + 4)] = __uint_as_float(r[i]);
      }
    }
    tc_fence_before();
    __syncwarp();
    if (!dry) {
      if (lane == 0) mbar_arrive(&sm.o_free);
      ++seg;
    }
    dry = false;
  }
}

// Every CTA finds its own work: each thread looks at some slots, with the starts and lengths in the ring's
// memory (not in use yet; read from there in one round trip).  CTA 0 leaves the slots' CTAs for the
// kernel that joins, and reports bad requests.
constexpr int kCached = 4096;   // requests that are looked at there

template <int D>
__device__ void find_work(const Params& given, Smem<D>& sm) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, B = given.c.B, G = gridDim.x;
  Params p = given;
  if (tid == 0) sm.places = 0;
  if (B < kCached) {
    int32_t* const starts = reinterpret_cast<int32_t*>(sm.ring[0]);
    int32_t* const len = starts + kCached;
    for (int b = tid; b <= B; b += kThreads) {
      starts[b] = given.c.starts[b];
      if (b < B) len[b] = given.c.L[b];
    }
    p.c.starts = starts;
    p.c.L = len;
    __syncthreads();
  }
  if (blockIdx.x == 0)
    for (int b = tid; b < B; b += kThreads) {
      const int state = attn_state(p.c, b);
      if (state != TV_OK) record_error(p.status, state);
    }
  const int per = (p.n_slots + kThreads - 1) / kThreads;
  const int lo = min(p.n_slots, tid * per), hi = min(p.n_slots, lo + per);
  const int b0 = lo < hi ? request_at(p, lo) : 0;
  int b, most = 0;
  int64_t mine = 0;
  Item it;
  auto look = [&](int slot) {   // the slot's item; its places, 0: none
    while (b + 1 < B && slot_of(p, b + 1) <= slot) ++b;
    const int k = b < 0 ? 0 : slot - slot_of(p, b);
    it.units = 0;
    if (b >= 0 && k < items_of(p, b)) it = item_of(p, b, k);
    return places_of(it.units);
  };
  b = b0;
#pragma unroll 1
  for (int slot = lo; slot < hi; ++slot) {
    const int n = look(slot);
    mine += n;
    most = max(most, n);
  }
  int64_t x = mine;   // places in front of the thread's slots
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  most = __reduce_max_sync(0xffffffffu, most);
  if (lane == 31) {
    sm.scan[warp] = x;
    sm.most[warp] = most;
  }
  __syncthreads();
  int64_t total = 0;
  x -= mine;
#pragma unroll
  for (int w = 0; w < kThreads / 32; ++w) {
    const int64_t y = sm.scan[w];
    x += w < warp ? y : 0;
    total += y;
    most = max(most, sm.most[w]);
  }
  const int64_t q = share_of(total, most, G), start = blockIdx.x * q;
  if ((start >= x && start < x + mine) || (blockIdx.x == 0 && lo < hi)) {
    b = b0;
#pragma unroll 1
    for (int slot = lo; slot < hi; ++slot) {
      const int n = per == 1 ? (int)mine : look(slot);
      if (start >= x && start < x + n) {
        sm.first = it;
        sm.begin = (int)(start - x);
        sm.places = min(q, total - start);
      }
      if (blockIdx.x == 0) p.pieces[slot] = piece_of(x, n, q, G);
      x += n;
    }
  }
  fence_proxy_async_smem();   // (the ring's copies come behind these accesses)
  __syncthreads();
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1) few_kernel(const __grid_constant__ Params p) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  Smem<D>& sm = *reinterpret_cast<Smem<D>*>(smem_raw);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if ((smem_u32(smem_raw) & 1023u) != 0) {   // the swizzled tiles need it; the window starts so
    pdl_wait();
    if (threadIdx.x == 0) record_error(p.status, TV_ERR_CUDA);
    return;
  }
  if (threadIdx.x == 0) {
    for (int i = 0; i < kSlots; ++i) {
      mbar_init(&sm.full[i], 1);
      mbar_init(&sm.empty[i], 1);
    }
    mbar_init(&sm.q_full, 1);
    mbar_init(&sm.q_free, 1);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sm.s_full[i], 1);
      mbar_init(&sm.s_free[i], kSmxWarps);
      mbar_init(&sm.p_full[i], kSmxWarps);
      mbar_init(&sm.pv_done[i], 1);
    }
    mbar_init(&sm.o_full, 1);
    mbar_init(&sm.o_free, kSmxWarps);
    mbar_init(&sm.drain, 1);
    sm.abort = 0;
    fence_mbar_init();
    prefetch_tmap(&p.mQ);
    prefetch_tmap(&p.mC4K);
    prefetch_tmap(&p.mC4V);
  }
  if (warp == 1) {
    tmem_alloc1(&sm.tmem, 512);
    tmem_relinquish1();
  }
  // behind the gather, which has waited for everything in front of it, only its rows are waited for
  // (before the first tile with C128 entries, and before any output)
  if (!p.gathered) pdl_wait();
  pdl_launch_dependents();
  find_work(p, sm);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 0) {
    producer(p, sm);
  } else if (warp == 1) {
    if (lane == 0) mma(p, sm);
    __syncwarp();
  } else {
    softmax(p, sm);
  }
  pdl_wait();   // this kernel completes only after the one it depends on
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1) tmem_dealloc1(sm.tmem, 512);
}

// Joins the parts of items that several CTAs have: grid (slots, 64 / rows per CTA).  Few slots: D / 128
// warps per row with one vector of columns per lane and the loads of eight parts in flight (an item may
// have dozens of parts); many: a warp per row, which takes one wave of CTAs instead of four (64 items of
// two to four parts: 8 us with a warp per row, 12 us with four).
constexpr int kWideSlots = 48;

template <int D, bool kWide>
__global__ void __launch_bounds__(256) few_merge_kernel(const __grid_constant__ Params p) {
  constexpr int kPerRow = kWide ? D / 4 : 32;       // threads of a row
  constexpr int kVecs = kWide ? 1 : D / 128;        // vectors of four columns per thread
  constexpr int kRow = D + 4;
  const int lane = threadIdx.x & 31, slot = blockIdx.x, b = request_at(p, slot);
  const int k = b < 0 ? 0 : slot - slot_of(p, b);
  const bool some = b >= 0 && k < items_of(p, b);
  Item it;
  if (some) it = item_of(p, b, k);
  pdl_wait();
  pdl_launch_dependents();
  if (!some) return;
  const Piece piece = p.pieces[slot];
  const int c0 = piece.first, c1 = c0 + piece.ctas - 1;   // the CTAs that have the item
  const int r = (256 / kPerRow) * blockIdx.y + threadIdx.x / kPerRow, at = 4 * (threadIdx.x % kPerRow);
  if (c0 == c1 || r >= it.rows) return;
  // CTA c's part: the one that goes on (1) of the first CTA, the one begun before (0) of the others
  auto part = [&](int c) { return p.part + (((int64_t)c * 2 + (c == c0)) * kRows + r) * kRow; };
  float4 acc[kVecs];
#pragma unroll
  for (int j = 0; j < kVecs; ++j) acc[j] = make_float4(0.f, 0.f, 0.f, 0.f);
  // 32 parts at a time: lane i weighs part i
  float M = -INFINITY, sum = 0.f;
  for (int first = c0; first <= c1; first += 32) {
    const int n = min(32, c1 - first + 1);
    const float2 ml = *reinterpret_cast<const float2*>(part(first + min(lane, n - 1)) + D);
    const float m = lane < n ? ml.x : -INFINITY;
    const float top = fmaxf(M, warp_max(m)), base = top == -INFINITY ? 0.f : top;
    const float old = exp2f(M - base), f = lane < n ? exp2f(m - base) : 0.f;
    M = top;
    sum = sum * old + warp_sum(f * ml.y);
#pragma unroll
    for (int j = 0; j < kVecs; ++j)
      acc[j] = make_float4(acc[j].x * old, acc[j].y * old, acc[j].z * old, acc[j].w * old);
#pragma unroll (kWide ? 8 : 3)
    for (int i = 0; i < n; ++i) {
      const float w = __shfl_sync(0xffffffffu, f, i);
      const float* from = part(first + i) + at;
#pragma unroll
      for (int j = 0; j < kVecs; ++j) {
        const float4 v = *reinterpret_cast<const float4*>(from + 128 * j);
        acc[j] = make_float4(fmaf(w, v.x, acc[j].x), fmaf(w, v.y, acc[j].y), fmaf(w, v.z, acc[j].z),
                             fmaf(w, v.w, acc[j].w));
      }
    }
  }
  const float inv = 1.f / sum;
  const int64_t row = (int64_t)it.row0 + r;
#pragma unroll
  for (int j = 0; j < kVecs; ++j)
    store_f4(p.O + row * D + at + 128 * j,
             make_float4(acc[j].x * inv, acc[j].y * inv, acc[j].z * inv, acc[j].w * inv));
  if (at == 0) p.lse[row] = (M + log2f(sum)) * 0.6931471805599453f;
}

}  // namespace few
}  // namespace tv

// ---- host side --------------------------------------------------------------------------------------
bool tv_few_ok(const tv_shape* s) {
  // rows of the tensor maps: 31 bits (page pools' raw rows and C4 entries always are)
  const int64_t lim = (int64_t)1 << 31, B = s->B;
  return s->dtype == TV_BF16 && s->d % 128 == 0 &&
         (!(s->comp_mask & TV_COMP_C128) || B * (s->c128_cap + 63) < lim) &&
         (s->page_tokens > 0 ||
          (B * s->raw_cap < lim && (!(s->comp_mask & TV_COMP_C4) || B * s->c4_cap < lim)));
}

namespace {

int sm_count() {
  int dev = 0, n = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) {
    cudaGetLastError();
    return 152;
  }
  return n;
}

int64_t slots_of(const tv_shape* s, int n_new) {
  return (int64_t)n_new * s->H / tv::few::kRows + s->B;
}
size_t table_bytes(const tv_shape* s, int n_new) { return (slots_of(s, n_new) + 31) / 32 * 256; }

template <int D>
cudaError_t launch_few(const tv::few::Params& p, int ctas, int slots, cudaStream_t stream) {
  using namespace tv::few;
  static_assert(sizeof(Smem<D>) <= 232448, "shared memory of one CTA exceeds the 227 KB limit");
  cudaError_t e = tv::allow_smem<few_kernel<D>>((int)sizeof(Smem<D>));
  if (e != cudaSuccess) return e;
  e = tv::launch_pdl(few_kernel<D>, dim3(ctas), dim3(kThreads), sizeof(Smem<D>), stream, p);
  if (e != cudaSuccess) return e;
  if constexpr (1024 % D == 0)   // (whole rows per CTA)
    if (slots <= kWideSlots)
      return tv::launch_pdl(few_merge_kernel<D, true>, dim3(slots, kRows * D / 1024), dim3(256), 0, stream,
                            p);
  return tv::launch_pdl(few_merge_kernel<D, false>, dim3(slots, kRows / 8), dim3(256), 0, stream, p);
}

}  // namespace

size_t tv_few_workspace(const tv_shape* s, int n_new) {
  return 2 * tv_chunk_gather_bytes(s) + table_bytes(s, n_new) +
         (size_t)sm_count() * 2 * tv::few::kRows * (s->d + 4) * sizeof(float);
}

int tv_launch_few(const tv_shape* s, int n_new, const int32_t* starts, const void* Q,
                  const void* c4K, const void* c4V, const void* c128K, const void* c128V,
                  const void* rawK, const void* rawV, const int32_t* L, float scale, void* O,
                  float* lse, void* workspace, int32_t* status, cudaStream_t stream) {
  using namespace tv::few;
  const char* fn = "tv_chunk_attn";
  Params p;
  const bool c4 = s->comp_mask & TV_COMP_C4, c128 = s->comp_mask & TV_COMP_C128;
  const bool paged = s->page_tokens > 0;
  char* ws = reinterpret_cast<char*>(workspace);
  const size_t gather = tv_chunk_gather_bytes(s);
  const uint64_t pool = (uint64_t)s->n_pool_pages * (paged ? s->page_tokens : 0), B = (uint64_t)s->B;
  auto rows_or_one = [](uint64_t r) { return r > 0 ? r : (uint64_t)1; };
  const uint64_t rawrows = rows_or_one(paged ? pool : B * (uint64_t)s->raw_cap);
  // an inactive compressor's maps are pointed at the raw rows (never read: it has no tiles)
  const uint64_t c4rows = !c4 ? rawrows : rows_or_one(paged ? pool / 4 : B * (uint64_t)s->c4_cap);
  p.gathered = gather > 0;
  p.c128_stride = p.gathered ? tv_chunk_c128_stride(s) : s->c128_cap;
  const uint64_t c128rows = !c128 ? rawrows : rows_or_one(B * (uint64_t)p.c128_stride);
  const void* k4 = c4 ? c4K : rawK;
  const void* v4 = c4 ? c4V : rawV;
  const void* k128 = !c128 ? rawK : p.gathered ? ws : c128K;
  const void* v128 = !c128 ? rawV : p.gathered ? ws + gather : c128V;
  const int d = s->d;
  if (!(tv_make_map(&p.mQ, Q, 2, d, (uint64_t)n_new * s->H, 1, kRows) &&
        tv_make_map(&p.mC4K, k4, 2, d, c4rows, 1, 64) && tv_make_map(&p.mC4V, v4, 2, d, c4rows, 1, 64) &&
        tv_make_map(&p.mC128K, k128, 2, d, c128rows, 1, 64) &&
        tv_make_map(&p.mC128V, v128, 2, d, c128rows, 1, 64) &&
        tv_make_map(&p.mRawK, rawK, 2, d, rawrows, 1, 64) &&
        tv_make_map(&p.mRawV, rawV, 2, d, rawrows, 1, 64)))
    return tv_set_error(TV_ERR_CUDA, "%s: tensor-map encoding failed", fn);
  p.c = tv::chunk_of(s, n_new, starts, L);
  p.H = s->H;
  p.W = s->W;
  p.tail_mode = s->tail_mode;
  p.scale_log2 = scale * 1.4426950408889634f;
  p.O = reinterpret_cast<__nv_bfloat16*>(O);
  p.lse = lse;
  p.n_slots = (int)slots_of(s, n_new);
  p.pieces = reinterpret_cast<Piece*>(ws + 2 * gather);
  p.part = reinterpret_cast<float*>(ws + 2 * gather + table_bytes(s, n_new));
  p.status = status;
  tv_attn_test_aid(&p.timeout_ns, &p.withhold_tile);
  if (p.gathered)
    if (int rc = tv_chunk_gather(s, starts, L, c128K, c128V, ws, status, stream)) return rc;
  const int ctas = sm_count(), slots = (int)slots_of(s, n_new);
  const cudaError_t e = d == 512   ? launch_few<512>(p, ctas, slots, stream)
                        : d == 384 ? launch_few<384>(p, ctas, slots, stream)
                        : d == 256 ? launch_few<256>(p, ctas, slots, stream)
                                   : launch_few<128>(p, ctas, slots, stream);
  if (e != cudaSuccess) {
    cudaGetLastError();
    return tv_set_error(TV_ERR_CUDA, "%s: launch failed: %s", fn, cudaGetErrorString(e));
  }
  return tv_check_launch(fn);
}

// Beam search's selection over beams and vocabulary.
//
// tv_token_logprobs' kernel reads the logits once and leaves every beam's `width` best tokens with
// their log probabilities in the workspace; no other token of a beam can be among its group's
// `width` best.  A CTA per group then scores the beams' lists, which are sorted, and a warp merges
// them: lane w holds the head of beam w's list, and `width` times the best head goes on.
//
// A candidate's score is scores[w] + scale (x - m) - ln S, with m the beam's largest logit and ln S
// the log of its sum relative to m, which is what the log probability of m itself is (up to sign).
// Both x and m are exact and the score is taken in fp64, so all that two beams' scores are off by is what ln S
// is: fp32 sums of approximate exponentials (2^-21) and its rounding (2^-24 of a number of a few units).
// Within a beam the order is the logits'.
//
// The logits' stream bounds it: 64 groups of 8 beams over 32000 bf16 logits 15 us (4.8 at the rate of a
// copy; 13 and 6 for the two kernels alone), 16 of 16 over 128001 fp32 36 us (19); 4 beams of one request
// 11 us, the two launches.  All the beams' lists merged by one warp without the CTA's scoring in front:
// 25 us instead of 15.
#include <math.h>

#include "tv_common.cuh"

int tv_launch_logprobs(const tv_shape* s, int vocab, int64_t ld, int logits_dtype,
                       const void* logits, int n_tok, const int32_t* tokens, const int32_t* nodes,
                       float scale, int n_top, float* lse, float* entropy, float* logprobs,
                       int32_t* top_ids, float* top_logprobs, int32_t* target, int32_t* status,
                       cudaStream_t stream);

namespace tv {

constexpr int kMaxWidth = 32;

struct BeamArgs {
  int B, width, eos;
  int64_t ld;
  float scale;
  const float* scores;
  const int32_t* done;
  const int32_t* ids;      // [B][width] every beam's best tokens, -1: none
  const float* logprobs;   // [B][width]
  int32_t* source;
  int32_t* token;
  float* new_scores;
  int32_t* new_done;
  int32_t* rank;
  int32_t* status;
};

// Doubles as integers in the same order (-0 as 0).
__device__ __forceinline__ uint64_t key_of(double x) {
  const int64_t bits = __double_as_longlong(x + 0.0);
  return (uint64_t)bits ^ (bits < 0 ? ~0ull : 1ull << 63);
}
__device__ __forceinline__ double of_key(uint64_t key) {
  return __longlong_as_double((int64_t)(key ^ (key >> 63 ? 1ull << 63 : ~0ull)));
}
constexpr uint64_t kNoCandidate = ~0xfff0000000000000ull;   // of -inf

template <typename T>
__global__ void __launch_bounds__(256) beam_kernel(BeamArgs a, const T* logits) {
  __shared__ uint64_t key[kMaxWidth][kMaxWidth];   // [place in the list][beam]
  __shared__ int32_t id[kMaxWidth][kMaxWidth];
  const int W = a.width, first = blockIdx.x * W;
  pdl_wait();
  pdl_launch_dependents();
  // the beams' candidates, all at once (what a group reads of scores and done is read before it
  // writes them)
  for (int i = threadIdx.x; i < W * W; i += blockDim.x) {
    const int w = i / W, h = i - w * W;
    const int64_t b = first + w;
    const float sum = a.scores[b], lp = a.logprobs[b * W];
    const bool ended = a.done != nullptr && a.done[b] != 0;
    const int top = a.ids[b * W];
    int t = a.ids[b * W + h];
    double s = -INFINITY;
    if (!(sum < INFINITY)) {   // NaN, +inf
      if (h == 0) record_error(a.status, TV_ERR_VALUE);
    } else if (sum > -INFINITY && ended) {
      t = a.eos;
      if (h == 0) s = sum;
    } else if (sum > -INFINITY && t >= 0) {
      const T* row = logits + b * a.ld;
      s = (double)sum + ((double)a.scale * ((double)load_f(row + t) - (double)load_f(row + top)) +
                         (double)lp);
    } else if (sum > -INFINITY && h == 0 && !(lp == lp)) {   // (its ids are -1)
      record_error(a.status, TV_ERR_VALUE);
    }
    key[h][w] = key_of(s);
    id[h][w] = t;
  }
  __syncthreads();
  if (threadIdx.x >= 32) return;
  const int lane = threadIdx.x;
  const bool beam = lane < W;
  const bool over = beam && a.done != nullptr && a.done[first + lane] != 0;
  __syncwarp();
  // the `width` best: lane k keeps the k-th, lane w holds the head of list w
  int head = 0, from = -1, tok = -1;
  double best = -INFINITY;
  uint64_t mine = beam ? key[0][lane] : 0;
  for (int k = 0; k < W; ++k) {
    const uint32_t hi = __reduce_max_sync(0xffffffffu, (uint32_t)(mine >> 32));
    const uint32_t low = (uint32_t)(mine >> 32) == hi ? (uint32_t)mine : 0u;
    const uint32_t lo = __reduce_max_sync(0xffffffffu, low);
    const uint64_t top = (uint64_t)hi << 32 | lo;
    if (top <= kNoCandidate) break;   // candidates have run out
    const int w = __ffs(__ballot_sync(0xffffffffu, mine == top)) - 1;   // equal: the lower beam
    const int at = __shfl_sync(0xffffffffu, head, w);
    if (lane == k) {
      best = of_key(top);
      from = w;
      tok = id[at][w];
    }
    if (lane == w) {
      ++head;
      mine = head < W ? key[head][lane] : 0;
    }
  }
  // slots: a beam's best continuation (the first of it) stays, the others fill the free ones
  const unsigned lower = (1u << lane) - 1u, all = W == 32 ? ~0u : (1u << W) - 1u;
  const unsigned same = __match_any_sync(0xffffffffu, from);
  const bool stays = from >= 0 && (same & lower) == 0;
  const unsigned taken = __reduce_or_sync(0xffffffffu, stays ? 1u << from : 0u);
  const unsigned moves = __ballot_sync(0xffffffffu, beam && !stays);
  int slot = from;
  if (beam && !stays) slot = (int)__fns(all & ~taken, 0, __popc(moves & lower) + 1);
  const bool was = __shfl_sync(0xffffffffu, (int)over, from >= 0 ? from : 0);
  if (!beam) return;
  const int b = first + slot;
  a.source[b] = from >= 0 ? first + from : -1;
  a.token[b] = tok;
  a.new_scores[b] = (float)best;
  if (a.new_done) a.new_done[b] = from >= 0 && (was || tok == a.eos) ? 1 : 0;
  if (a.rank) a.rank[b] = from >= 0 ? lane : -1;
}

}  // namespace tv

size_t tv_beam_workspace(const tv_shape* s, int width) {
  return ((size_t)s->B * width * 8 + 255) / 256 * 256;
}

int tv_launch_beam(const tv_shape* s, int width, int vocab, int64_t ld, int logits_dtype,
                   const void* logits, const float* scores, const int32_t* done, int eos,
                   float scale, int32_t* source, int32_t* token, float* new_scores,
                   int32_t* new_done, int32_t* rank, void* workspace, int32_t* status,
                   cudaStream_t stream) {
  tv_shape rows = *s;
  rows.D = 1;
  int32_t* ids = (int32_t*)workspace;
  float* logprobs = (float*)(ids + (size_t)s->B * width);
  if (int rc = tv_launch_logprobs(&rows, vocab, ld, logits_dtype, logits, 0, nullptr, nullptr, scale,
                                  width, nullptr, nullptr, nullptr, ids, logprobs, nullptr, nullptr,
                                  stream))
    return rc;
  const tv::BeamArgs a = {s->B, width, eos, ld, scale, scores, done, ids, logprobs, source, token,
                          new_scores, new_done, rank, status};
  const dim3 grid(s->B / width), block(width * width >= 256 ? 256 : (width * width + 31) / 32 * 32);
  const cudaError_t e =
      logits_dtype == TV_BF16
          ? tv::launch_pdl(tv::beam_kernel<__nv_bfloat16>, grid, block, 0, stream, a,
                           (const __nv_bfloat16*)logits)
          : tv::launch_pdl(tv::beam_kernel<float>, grid, block, 0, stream, a, (const float*)logits);
  if (e != cudaSuccess) {
    cudaGetLastError();
    return tv_set_error(TV_ERR_CUDA, "tv_beam_select: launch failed: %s", cudaGetErrorString(e));
  }
  return tv_check_launch("tv_beam_select");
}

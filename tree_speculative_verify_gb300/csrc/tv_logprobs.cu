// From logits to the integers and log probabilities a tree round works with: per (request, node)
// row the log-sum-exp, the entropy, the target token, the best alternatives, and the log
// probabilities of given tokens (a draft tree's tokens under their parents).
//
// With m = max x, y_i = scale * (x_i - m), S = sum e^{y_i} and T = sum y_i e^{y_i}:
//   lse = scale * m + ln S,  entropy = ln S - T / S,  log p_i = y_i - ln S.
// One CTA per row.  A thread keeps its own running (m, S, T) in base 2 and rescales when its
// maximum grows, so the row is read once for the sums; the partial triples are joined over the
// CTA at the end.  The alternatives are found by one scan of the row per alternative (the largest
// key below the last one found), a key being the logit's order and, for equal logits, the lower
// id first.
#include <float.h>

#include "tv_common.cuh"

namespace tv {

constexpr int kLpThreads = 256;
constexpr int kLpWarps = kLpThreads / 32;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

struct LogprobArgs {
  int D, vocab, n_tok, n_top;
  int64_t ld;
  float scale;
  const int32_t* tokens;
  const int32_t* nodes;
  float* lse;
  float* entropy;
  float* logprobs;
  int32_t* top_ids;
  float* top_logprobs;
  int32_t* target;
  int32_t* status;
};

// Partial sums of a set of logits: their maximum (-inf: none above -inf yet), and S and T (base 2)
// relative to it.  A NaN or +inf logit makes S NaN.
struct Partial {
  float m, s, t;
};

__device__ __forceinline__ float exp2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// p relative to the larger maximum m; a set without a logit above -inf has s = t = 0 (or NaN)
__device__ __forceinline__ void rebase(Partial& p, float m, float c) {
  if (m > p.m) {
    const float shift = (p.m - m) * c;
    const float f = exp2_approx(shift);
    p.t = p.s == 0.f ? 0.f : (p.t + fmaxf(shift, -256.f) * p.s) * f;
    p.s *= f;
    p.m = m;
  }
}

__device__ __forceinline__ Partial join(Partial a, Partial b, float c) {
  const float m = fmaxf(a.m, b.m);
  rebase(a, m, c);
  rebase(b, m, c);
  return {m, a.s + b.s, a.t + b.t};
}

// Order of a logit as an unsigned number; equal logits (and -0, +0) give equal numbers.
__device__ __forceinline__ uint32_t order_of(float x) {
  const uint32_t u = __float_as_uint(x + 0.f);
  return u ^ ((u >> 31) ? 0xffffffffu : 0x80000000u);
}
__device__ __forceinline__ float logit_of_order(uint32_t o) {
  return __uint_as_float(o ^ ((o >> 31) ? 0x80000000u : 0xffffffffu));
}
// Selection key: larger logits first, then lower ids.  0: not a candidate (-inf or NaN).
__device__ __forceinline__ uint64_t key_of(float x, int id) {
  return x > -INFINITY ? ((uint64_t)order_of(x) << 32) | (uint32_t)~id : 0ull;
}

// A row as 16-byte vectors: vector i holds the elements i * kVec - skew + (0 .. kVec-1).  Rows
// may start at any element; only the first and the last vector can reach past the row.
template <typename T>
struct Row {
  static constexpr int kVec = 16 / sizeof(T);
  const T* p;
  int vocab, skew, n_vec;
  __device__ Row(const T* row, int v) : p(row), vocab(v) {
    skew = (int)(((uintptr_t)row & 15u) / sizeof(T));
    n_vec = (skew + v + kVec - 1) / kVec;
  }
  // -inf where the vector reaches past the row
  __device__ __forceinline__ void load(int i, float (&x)[kVec]) const {
    const int e0 = i * kVec - skew;
    if (e0 >= 0 && e0 + kVec <= vocab) {
      const uint4 w = *reinterpret_cast<const uint4*>(p + e0);
      unpack(w, x);
    } else {
#pragma unroll
      for (int j = 0; j < kVec; ++j)
        x[j] = e0 + j >= 0 && e0 + j < vocab ? load_f(p + e0 + j) : -INFINITY;
    }
  }
  __device__ static __forceinline__ void unpack(const uint4& w, float (&x)[kVec]) {
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if constexpr (sizeof(T) == 2) {
        x[2 * j] = __uint_as_float(u[j] << 16);
        x[2 * j + 1] = __uint_as_float(u[j] & 0xffff0000u);
      } else {
        x[j] = __uint_as_float(u[j]);
      }
    }
  }
};

__device__ __forceinline__ uint64_t max_u64(uint64_t a, uint64_t b) { return a > b ? a : b; }

template <typename T>
__global__ void __launch_bounds__(kLpThreads) logprobs_kernel(const T* __restrict__ logits,
                                                              const LogprobArgs a) {
  __shared__ Partial s_part[kLpWarps];
  __shared__ uint64_t s_key[kLpWarps];
  const int64_t r = blockIdx.x;
  const int b = (int)(r / a.D), v = (int)(r - (int64_t)b * a.D);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const Row<T> row(logits + r * a.ld, a.vocab);
  constexpr int kVec = Row<T>::kVec;
  const float c = a.scale * kLog2e;

  Partial p = {-INFINITY, 0.f, 0.f};
  for (int i = tid; i < row.n_vec; i += kLpThreads) {
    float x[kVec];
    row.load(i, x);
    float m = x[0];
#pragma unroll
    for (int j = 1; j < kVec; ++j) m = fmaxf(m, x[j]);
    rebase(p, m, c);
    const float base = fmaxf(p.m, -FLT_MAX);
#pragma unroll
    for (int j = 0; j < kVec; ++j) {
      const float y = (x[j] - base) * c;
      const float e = exp2_approx(y);
      p.s += e;
      p.t += fmaxf(y, -256.f) * e;
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const Partial q = {__shfl_xor_sync(0xffffffffu, p.m, o), __shfl_xor_sync(0xffffffffu, p.s, o),
                       __shfl_xor_sync(0xffffffffu, p.t, o)};
    p = join(p, q, c);
  }
  if (lane == 0) s_part[warp] = p;
  __syncthreads();
  p = s_part[0];
  for (int w = 1; w < kLpWarps; ++w) p = join(p, s_part[w], c);

  const bool bad = !(p.s == p.s) || p.m == INFINITY;   // a NaN or +inf among the logits
  const bool none = !bad && p.m == -INFINITY;
  const float nan = __int_as_float(0x7fffffff);
  const float log_s = logf(p.s);   // -inf for an empty row
  auto log_prob = [&](float x) {
    return bad ? nan : x == -INFINITY ? x : (x - p.m) * a.scale - log_s;
  };
  if (tid == 0) {
    if (bad) record_error(a.status, TV_ERR_VALUE);
    if (a.lse) a.lse[r] = bad ? nan : none ? -INFINITY : p.m * a.scale + log_s;
    if (a.entropy) a.entropy[r] = bad ? nan : none ? 0.f : fmaxf(log_s - kLn2 * (p.t / p.s), 0.f);
  }
  // given tokens: this row takes those of its node, and row 0 those without a node or a token
  for (int i = tid; i < a.n_tok; i += kLpThreads) {
    const int64_t at = (int64_t)b * a.n_tok + i;
    const int node = a.nodes ? a.nodes[at] : i, tok = a.tokens[at];
    const bool wrong = node >= a.D || tok >= a.vocab;
    if (node < 0 || tok < 0 || wrong) {
      if (v == 0) {
        a.logprobs[at] = 0.f;
        if (wrong) record_error(a.status, TV_ERR_ARG);
      }
    } else if (node == v) {
      a.logprobs[at] = log_prob(load_f(row.p + tok));
    }
  }
  // alternatives, one scan each
  const int n = a.n_top > 1 ? a.n_top : 1;
  uint64_t last = ~0ull;
  for (int k = 0; k < n; ++k) {
    uint64_t best = 0ull;
    if (!bad)
      for (int i = tid; i < row.n_vec; i += kLpThreads) {
        float x[kVec];
        row.load(i, x);
#pragma unroll
        for (int j = 0; j < kVec; ++j) {
          const uint64_t key = key_of(x[j], i * kVec - row.skew + j);
          if (key < last) best = max_u64(best, key);
        }
      }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) best = max_u64(best, __shfl_xor_sync(0xffffffffu, best, o));
    __syncthreads();
    if (lane == 0) s_key[warp] = best;
    __syncthreads();
    for (int w = 0; w < kLpWarps; ++w) best = max_u64(best, s_key[w]);
    last = best;
    if (tid == 0) {
      const int id = best ? (int)~(uint32_t)best : -1;
      if (k == 0 && a.target) a.target[r] = id;
      if (k < a.n_top) {
        a.top_ids[r * a.n_top + k] = id;
        a.top_logprobs[r * a.n_top + k] =
            bad ? nan : id < 0 ? -INFINITY : log_prob(logit_of_order((uint32_t)(best >> 32)));
      }
    }
    if (best == 0ull) last = 0ull;   // nothing below: the other places stay empty
  }
}

}  // namespace tv

int tv_launch_logprobs(const tv_shape* s, int vocab, int64_t ld, int logits_dtype,
                       const void* logits, int n_tok, const int32_t* tokens, const int32_t* nodes,
                       float scale, int n_top, float* lse, float* entropy, float* logprobs,
                       int32_t* top_ids, float* top_logprobs, int32_t* target, int32_t* status,
                       cudaStream_t stream) {
  tv::LogprobArgs a = {s->D,   vocab,    n_tok,   n_top,        ld,     scale, tokens, nodes, lse,
                       entropy, logprobs, top_ids, top_logprobs, target, status};
  const dim3 grid((unsigned)(s->B * s->D)), block(tv::kLpThreads);
  if (logits_dtype == TV_BF16)
    tv::logprobs_kernel<<<grid, block, 0, stream>>>((const __nv_bfloat16*)logits, a);
  else
    tv::logprobs_kernel<<<grid, block, 0, stream>>>((const float*)logits, a);
  return tv_check_launch("tv_token_logprobs");
}

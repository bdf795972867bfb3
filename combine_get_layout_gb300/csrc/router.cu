// The router gate on the GPU: scores, grouped top-K choice and gate weights
// (ep_route), the same with the balance and z losses (ep_route_balance), and
// the gradient of both by the logits (ep_route_backward).
//
// One warp owns one token at a time; lane `lane` holds VPL of its E logits
// in registers (element_of below), so a token's row is read once and every
// reduction over experts is a warp reduction.  The statistics of the losses
// are summed in registers over a CTA's run of tokens, then once per (CTA,
// sequence) in a fixed order: no floating-point atomics, so the same inputs
// give the same bits.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <math_constants.h>

#include <type_traits>

#include "../../include/ep.h"
#include "ep_device.cuh"
#include "ep_internal.h"

namespace ep {
namespace {

constexpr int kRouteThreads = 256;
constexpr int kRouteWarps = kRouteThreads / 32;
constexpr int kMaxGroups = 32;
constexpr unsigned kFull = 0xffffffffu;

struct RouteParams {
  const void* logits;        // [T, ld] fp32 or bf16
  int64_t ld;
  const float* bias;         // [E] or null (sigmoid)
  const uint8_t* mask;       // [T] or null
  int T, E, K, G, kept;
  int per;                   // experts a group
  int per_log2;              // its logarithm where it is 4, 8, ... 128, else -1
  uint32_t per_inverse;      // expert e is in group e * per_inverse >> 21 (e < 2048)
  bool renorm;
  float scale;
  int64_t* idx;              // [T, K]
  float* w;                  // [T, K]
  // balance
  const int32_t* seq_start;  // [B + 1] or null (B = 1)
  int B;
  int tokens_per_cta;
  float* part_prob;          // [CTAs + B, E]
  int32_t* part_count;       // [CTAs + B, E]
  int32_t* part_tokens;      // [CTAs + B]
  float* part_z;             // [CTAs + B]
  unsigned* done;            // cleared for the second kernel
};

// Index of register r of this lane: one logit a load (V = 1), or V
// neighbouring ones.
template <int V>
__device__ __forceinline__ int element_of(int r, int lane) {
  return (r / V * 32 + lane) * V + r % V;
}

// A token's logits in registers, -inf past the last expert.
template <int VPL, int V, bool BF16>
__device__ __forceinline__ void load_row(const void* base, int64_t offset, int E, int lane,
                                         float (&x)[VPL]) {
#pragma unroll
  for (int r = 0; r < VPL; r += V) {
    const int e = element_of<V>(r, lane);
    if constexpr (V == 1) {
      if constexpr (BF16) {
        x[r] = e < E ? __uint_as_float(uint32_t(static_cast<const uint16_t*>(base)[offset + e]) << 16)
                     : -CUDART_INF_F;
      } else {
        x[r] = e < E ? static_cast<const float*>(base)[offset + e] : -CUDART_INF_F;
      }
    } else {
      static_assert(V == 4, "vectors of four logits");
#pragma unroll
      for (int i = 0; i < 4; ++i) x[r + i] = -CUDART_INF_F;
      if (e < E) {
        if constexpr (BF16) {
          const uint2 v = *reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(base) +
                                                          offset + e);
          x[r] = bf16_lo(v.x);
          x[r + 1] = bf16_hi(v.x);
          x[r + 2] = bf16_lo(v.y);
          x[r + 3] = bf16_hi(v.y);
        } else {
          const float4 v =
              *reinterpret_cast<const float4*>(static_cast<const float*>(base) + offset + e);
          x[r] = v.x;
          x[r + 1] = v.y;
          x[r + 2] = v.z;
          x[r + 3] = v.w;
        }
      }
    }
  }
}

template <bool BF16>
__device__ __forceinline__ float load_one(const void* base, int64_t at) {
  if constexpr (BF16)
    return __uint_as_float(uint32_t(static_cast<const uint16_t*>(base)[at]) << 16);
  else
    return static_cast<const float*>(base)[at];
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int d = 16; d; d >>= 1) v += __shfl_xor_sync(kFull, v, d);
  return v;
}

// Largest of the lanes' values; a NaN counts only where all are NaN.
__device__ __forceinline__ float warp_max(float v) {
  float m;
  asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(m) : "f"(v));
  return m;
}

constexpr float kLog2e = 1.4426950408889634f;

// 2^x and 1 / x to 2^-22 of the value: what a score is rounded to anyway
// once 32-bit sums and products have passed over it.
__device__ __forceinline__ float fast_exp2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ float fast_reciprocal(float x) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

__device__ __forceinline__ float sigmoid(float x) {
  return fast_reciprocal(1.0f + fast_exp2(-kLog2e * x));
}

// exp(l - top); the difference first, so that no size of logit overflows.
__device__ __forceinline__ float soft_score(float l, float top) {
  return fast_exp2((l - top) * kLog2e);
}

// Softmax scores of a token before their division: s = exp(x - top), top the
// row's maximum; returns their total.  -inf scores 0, and so does all of a
// row of nothing else.
template <int VPL>
__device__ __forceinline__ float soft_scores(const float (&x)[VPL], float (&s)[VPL], float top) {
  const float base = top == -CUDART_INF_F ? 0.0f : top;
  float total = 0.0f;
#pragma unroll
  for (int r = 0; r < VPL; ++r) {
    s[r] = soft_score(x[r], base);
    total += s[r];
  }
  return warp_sum(total);
}

// Scores of a token as soft_scores or sigmoid has them, their total, and
// (softmax) the row's maximum.
template <int VPL, bool SIG>
__device__ __forceinline__ float scores(const float (&x)[VPL], float (&s)[VPL], float* top) {
  if constexpr (SIG) {
    float total = 0.0f;
#pragma unroll
    for (int r = 0; r < VPL; ++r) {
      s[r] = sigmoid(x[r]);      // exp2(+inf) = inf, its reciprocal 0
      total += s[r];
    }
    *top = 0.0f;
    return warp_sum(total);
  } else {
    float m = x[0];
#pragma unroll
    for (int r = 1; r < VPL; ++r) m = fmaxf(m, x[r]);
    *top = warp_max(m);
    return soft_scores<VPL>(x, s, *top);
  }
}

// The `kept` best of G groups (G <= 32) by the scores that lanes g < G hold,
// as a bit mask; equal scores go to the lower group, -inf is never kept.
__device__ __forceinline__ uint32_t best_groups(float score, int G, int kept, int lane) {
  uint32_t keep = 0;
  float left = lane < G ? score : -CUDART_INF_F;
  for (int i = 0; i < kept; ++i) {
    const float top = warp_max(left);
    const uint32_t at = __ballot_sync(kFull, left == top);
    // no NaN reaches this, so that a lane always answers
    const int g = __ffs(at) - 1;
    keep |= top > -CUDART_INF_F ? 1u << g : 0u;
    if (lane == g) left = -CUDART_INF_F;
  }
  return keep;
}

// Adds (best, second) of another set to a running pair.
__device__ __forceinline__ void top_two(float& best, float& second, float b, float s) {
  second = fmaxf(fminf(best, b), fmaxf(second, s));
  best = fmaxf(best, b);
}

// Sigmoid: a group's two best scores' sum, an expert out of service adding
// none.  Softmax: its best.
template <bool SIG>
__device__ __forceinline__ float group_score(float best, float second) {
  return SIG && second > -CUDART_INF_F ? best + second : best;
}

// Clears the choice scores of every group but the best.  Groups of 4, 8, ...
// 128 experts are whole aligned runs of lanes of one vector (V = 4), and
// reduce by shuffles; other sizes go through this warp's shared scratch of E
// floats.
template <int VPL, int V, bool SIG>
__device__ __forceinline__ void keep_groups(const RouteParams& p, float (&c)[VPL], float* row,
                                            int lane) {
#pragma unroll
  for (int r = 0; r < VPL; ++r) c[r] = fmaxf(c[r], -CUDART_INF_F);      // a NaN is not chosen
  if constexpr (V == 4) {
    if (p.per_log2 > 0) {
      // a group is 2^span lanes of a vector, a vector 2^(5 - span) groups
      const int span = p.per_log2 - 2, local = lane >> span, of_vector = 5 - span;
      const int at = (lane & ((1 << of_vector) - 1)) << span;      // where group `lane` begins
      float mine = -CUDART_INF_F;
#pragma unroll
      for (int v = 0; v < VPL / 4; ++v) {
        const float hi0 = fmaxf(c[4 * v], c[4 * v + 1]), lo0 = fminf(c[4 * v], c[4 * v + 1]);
        const float hi1 = fmaxf(c[4 * v + 2], c[4 * v + 3]), lo1 = fminf(c[4 * v + 2], c[4 * v + 3]);
        float best = hi0, second = lo0;
        top_two(best, second, hi1, lo1);
#pragma unroll
        for (int i = 0; i < 5; ++i) {
          if (i >= span) break;
          const float b = __shfl_xor_sync(kFull, best, 1 << i);
          if constexpr (SIG) {
            const float s = __shfl_xor_sync(kFull, second, 1 << i);
            top_two(best, second, b, s);
          } else {
            best = fmaxf(best, b);
          }
        }
        const float score = __shfl_sync(kFull, group_score<SIG>(best, second), at);
        if (lane >> of_vector == v) mine = score;
      }
      const uint32_t keep = best_groups(mine, p.G, p.kept, lane);
#pragma unroll
      for (int v = 0; v < VPL / 4; ++v) {
        const int g = (v << of_vector) + local;
        if (!((keep >> (g & 31)) & 1u)) {
#pragma unroll
          for (int i = 0; i < 4; ++i) c[4 * v + i] = -CUDART_INF_F;
        }
      }
      return;
    }
  }
#pragma unroll
  for (int r = 0; r < VPL; ++r) {
    const int e = element_of<V>(r, lane);
    if (e < p.E) row[e] = c[r];
  }
  __syncwarp();
  float best = -CUDART_INF_F, second = -CUDART_INF_F;
  if (lane < p.G)
    for (int i = 0; i < p.per; ++i) top_two(best, second, row[lane * p.per + i], -CUDART_INF_F);
  const uint32_t keep = best_groups(group_score<SIG>(best, second), p.G, p.kept, lane);
#pragma unroll
  for (int r = 0; r < VPL; ++r) {
    const int e = element_of<V>(r, lane);
    if (e < p.E && !((keep >> (e * p.per_inverse >> 21)) & 1u)) c[r] = -CUDART_INF_F;
  }
  __syncwarp();
}

// The K largest of a warp's choice scores one after another, equal ones by
// ascending index: lane k returns the k-th expert or -1.
template <int VPL, int V>
__device__ __noinline__ int choose_in_turn(float (&c)[VPL], int K, int lane) {
  int mine = -1;
  for (int k = 0; k < K; ++k) {
    float best = -CUDART_INF_F;
    int at = 0x7fffffff;
#pragma unroll
    for (int r = 0; r < VPL; ++r) {
      if (c[r] > best) {
        best = c[r];
        at = element_of<V>(r, lane);
      }
    }
    const float top = warp_max(best);
    if (top == -CUDART_INF_F) break;
    const int win = __reduce_min_sync(kFull, best == top ? at : 0x7fffffff);
#pragma unroll
    for (int r = 0; r < VPL; ++r)
      if (element_of<V>(r, lane) == win) c[r] = -CUDART_INF_F;
    if (lane == k) mine = win;
  }
  return mine;
}

// A set of the registers 0 .. VPL - 1.
template <int VPL>
struct RegisterSet {
  using Bits = std::conditional_t<(VPL > 32), unsigned long long, uint32_t>;
  Bits bits = 0;
  __device__ __forceinline__ void add(int r, bool in) { bits |= in ? Bits(1) << r : Bits(0); }
  __device__ __forceinline__ int first() const {
    if constexpr (VPL > 32) return __ffsll(bits) - 1;
    return __ffs(bits) - 1;
  }
  __device__ __forceinline__ void drop_first() { bits &= bits - 1; }
};

// What a warp's lanes share while they choose: candidates, one a lane.
struct Candidates {
  int expert[32];
  unsigned long long key[32];
};

// Order of choice as one number: the higher score first, then the lower
// index.  -0 and +0 are equal scores.
__device__ __forceinline__ unsigned long long choice_key(float c, int e) {
  const uint32_t u = __float_as_uint(c + 0.0f);
  const uint32_t hi = u ^ (uint32_t(int32_t(u) >> 31) | 0x80000000u);
  return static_cast<unsigned long long>(hi) << 32 | uint32_t(~e);
}

// A lane's share of a token's choice: expert e, with logit l, takes `rank`;
// e = -1 where the rank stays empty, rank >= K where the lane has none.
struct Chosen {
  int e, rank;
  float l;
};

// Chooses the K largest of a warp's choice scores c, `best` the lane's
// largest; -inf and NaN are never chosen.  The K-th largest of the lanes'
// largest (equal ones taken together) is a bound that at least K scores
// reach, where K can be chosen at all; with scores spread over the lanes few
// more do.  Those become candidates, one a lane, that each count the
// candidates before them.  More than 32 candidates (many equal scores, K
// near 32) are chosen in turn.
template <int VPL, int V, bool BF16, bool SIG>
__device__ __forceinline__ Chosen choose(const RouteParams& p, const float (&c)[VPL], float best,
                                         const void* logits, int64_t offset, int lane,
                                         Candidates& cand) {
  float bound = -CUDART_INF_F;
#pragma unroll 4
  for (int k = 0; k < p.K; ++k) {
    bound = warp_max(best);
    best = best == bound ? -CUDART_INF_F : best;
  }
  bound = fmaxf(bound, -3.402823466e38f);
  RegisterSet<VPL> mine;
#pragma unroll
  for (int r = 0; r < VPL; ++r) mine.add(r, c[r] >= bound);
  const uint32_t before = lanemask_lt();
  int n = 0;
  for (;;) {
    const uint32_t who = __ballot_sync(kFull, mine.bits != 0);
    if (who == 0) break;
    const int at = n + __popc(who & before);
    if (mine.bits != 0 && at < 32) cand.expert[at] = element_of<V>(mine.first(), lane);
    mine.drop_first();
    n += __popc(who);
  }
  __syncwarp();
  Chosen out = {-1, lane, 0.0f};
  if (n > 32) {
    float left[VPL];      // a copy: c itself then stays in registers
#pragma unroll
    for (int r = 0; r < VPL; ++r) left[r] = c[r];
    out.e = choose_in_turn<VPL, V>(left, p.K, lane);
    if (out.e >= 0) out.l = load_one<BF16>(logits, offset + out.e);
    return out;
  }
  unsigned long long key = 0;
  if (lane < n) {
    out.e = cand.expert[lane];
    out.l = load_one<BF16>(logits, offset + out.e);
    float score = out.l;
    if constexpr (SIG) score = sigmoid(out.l) + (p.bias != nullptr ? p.bias[out.e] : 0.0f);
    key = choice_key(score, out.e);
  }
  cand.key[lane] = key;      // the rest come after any candidate
  __syncwarp();
  int rank = 0;
  for (int i = 0; i < n; i += 4) {
#pragma unroll
    for (int j = 0; j < 4; ++j) rank += cand.key[i + j] > key ? 1 : 0;
  }
  __syncwarp();
  if (lane < n) out.rank = rank;
  return out;
}

// Floats of a row of E in shared memory: whole vectors of four.
__host__ __device__ __forceinline__ int padded_row(int E) { return (E + 3) & ~3; }

// A lane's values of a row of E floats in shared memory (16-byte aligned).
template <int VPL, int V>
__device__ __forceinline__ void read_row(const float* row, int E, int lane, float (&v)[VPL]) {
#pragma unroll
  for (int r = 0; r < VPL; r += V) {
    const int e = element_of<V>(r, lane);
    if constexpr (V == 4) {
      float4 f = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      if (e < E) f = *reinterpret_cast<const float4*>(row + e);
      v[r] = f.x;
      v[r + 1] = f.y;
      v[r + 2] = f.z;
      v[r + 3] = f.w;
    } else {
      v[r] = e < E ? row[e] : 0.0f;
    }
  }
}

// One token, given its logits: choice and gate weights.  Leaves the scores in
// `s` with their total and the row's maximum; softmax needs those only for
// statistics (STATS) or for weights that are not renormalised.  Returns the
// lane's chosen expert or -1.
template <int VPL, int V, bool BF16, bool SIG, bool STATS>
__device__ __forceinline__ int route_token(const RouteParams& p, int t, int lane, float* row,
                                           Candidates& cand, const float* bias,
                                           const float (&x)[VPL], float (&s)[VPL], float* total,
                                           float* top) {
  float best, scale = p.scale;
  const int64_t offset = int64_t(t) * p.ld;
  Chosen mine;
  if constexpr (SIG) {
    *total = scores<VPL, SIG>(x, s, top);
    float c[VPL];
    if (p.bias != nullptr) {
      read_row<VPL, V>(bias, p.E, lane, c);
    } else {
#pragma unroll
      for (int r = 0; r < VPL; ++r) c[r] = 0.0f;
    }
#pragma unroll
    for (int r = 0; r < VPL; ++r) c[r] = x[r] == -CUDART_INF_F ? -CUDART_INF_F : s[r] + c[r];
    if (p.G > 1) keep_groups<VPL, V, SIG>(p, c, row, lane);
    best = c[0];
#pragma unroll
    for (int r = 1; r < VPL; ++r) best = fmaxf(best, c[r]);
    mine = choose<VPL, V, BF16, SIG>(p, c, best, p.logits, offset, lane, cand);
  } else {
    best = x[0];
#pragma unroll
    for (int r = 1; r < VPL; ++r) best = fmaxf(best, x[r]);
    *top = warp_max(best);
    if (STATS || !p.renorm) {
      *total = soft_scores<VPL>(x, s, *top);
      if (!p.renorm) scale = scale / *total;
      if (*total != *total) scale = *total;
    } else {
      bool nan = false;
#pragma unroll
      for (int r = 0; r < VPL; ++r) nan |= x[r] != x[r];
      if (__any_sync(kFull, nan)) scale = CUDART_NAN_F;
    }
    if (p.G > 1) {
      float c[VPL];
#pragma unroll
      for (int r = 0; r < VPL; ++r) c[r] = x[r];
      keep_groups<VPL, V, SIG>(p, c, row, lane);
      best = c[0];
#pragma unroll
      for (int r = 1; r < VPL; ++r) best = fmaxf(best, c[r]);
      mine = choose<VPL, V, BF16, SIG>(p, c, best, p.logits, offset, lane, cand);
    } else {
      mine = choose<VPL, V, BF16, SIG>(p, x, best, p.logits, offset, lane, cand);
    }
  }
  const bool taken = mine.e >= 0 && mine.rank < p.K;
  float w = 0.0f;
  if (taken) w = SIG ? sigmoid(mine.l) : soft_score(mine.l, *top);
  if (p.renorm) {
    const float sum = warp_sum(w);
    scale = sum == 0.0f ? 0.0f : scale / sum;
  }
  if (mine.rank < p.K) {
    const int64_t at = int64_t(t) * p.K + mine.rank;
    p.idx[at] = mine.e;
    p.w[at] = taken ? w * scale : 0.0f;
  }
  return taken ? mine.e : -1;
}

__device__ __forceinline__ void route_masked(const RouteParams& p, int t, int lane) {
  if (lane < p.K) {
    p.idx[int64_t(t) * p.K + lane] = -1;
    p.w[int64_t(t) * p.K + lane] = 0.0f;
  }
}

// Logits that a warp loads ahead of the token it works on: the next token's,
// where two rows fit its registers.
template <int VPL>
constexpr bool kAhead = VPL <= 16;

template <int VPL, int V, bool BF16, bool SIG>
__global__ void __launch_bounds__(kRouteThreads) route_kernel(RouteParams p) {
  extern __shared__ __align__(16) float smem[];
  __shared__ Candidates cands[kRouteWarps];
  pdl_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const float* bias = smem;      // [E] padded to whole vectors, then the warps' rows
  float* row = smem + (warp + 1) * padded_row(p.E);
  if (SIG && p.bias != nullptr) {
    for (int e = threadIdx.x; e < p.E; e += kRouteThreads) smem[e] = p.bias[e];
    __syncthreads();
  }
  const int stride = gridDim.x * kRouteWarps;
  float x[VPL], s[VPL], total, top;
  int t = blockIdx.x * kRouteWarps + warp;
  if (kAhead<VPL> && t < p.T) load_row<VPL, V, BF16>(p.logits, int64_t(t) * p.ld, p.E, lane, x);
  for (; t < p.T; t += stride) {
    float next[VPL];
    if constexpr (kAhead<VPL>) {
      const int u = t + stride;
      if (u < p.T) load_row<VPL, V, BF16>(p.logits, int64_t(u) * p.ld, p.E, lane, next);
    } else {
      load_row<VPL, V, BF16>(p.logits, int64_t(t) * p.ld, p.E, lane, x);
    }
    if (p.mask != nullptr && p.mask[t] == 0)
      route_masked(p, t, lane);
    else
      route_token<VPL, V, BF16, SIG, false>(p, t, lane, row, cands[warp], bias, x, s, &total,
                                            &top);
    if constexpr (kAhead<VPL>) {
#pragma unroll
      for (int r = 0; r < VPL; ++r) x[r] = next[r];
    }
  }
}

// First sequence whose end lies past token t (the last one otherwise).
__device__ __forceinline__ int sequence_of(const int32_t* seq_start, int B, int t) {
  int lo = 0, hi = B - 1;
  while (lo < hi) {
    const int mid = (lo + hi) / 2;
    if (seq_start[mid + 1] > t)
      hi = mid;
    else
      lo = mid + 1;
  }
  return lo;
}

// ep_route_balance, first kernel.  A CTA owns the tokens [c * R, (c + 1) * R)
// and walks the sequences they belong to; the sums of (CTA c, sequence b) go
// to partial row c + b, which no other pair uses (both only grow along the
// tokens).
template <int VPL>
constexpr int kBalanceThreads = VPL <= 16 ? 512 : 256;
template <int VPL>
constexpr int kBalanceCtasPerSm = VPL <= 8 ? 2 : 1;

template <int VPL, int V, bool BF16, bool SIG>
__global__ void __launch_bounds__(kBalanceThreads<VPL>, kBalanceCtasPerSm<VPL>)
balance_kernel(RouteParams p) {
  constexpr int kThreads = kBalanceThreads<VPL>, kWarps = kThreads / 32;
  extern __shared__ __align__(16) float smem[];
  const int width = padded_row(p.E);
  float* probs = smem;                                          // [kWarps][width]
  float* bias = smem + kWarps * width;                          // [width]
  int* counts = reinterpret_cast<int*>(bias + width);           // [width]
  __shared__ Candidates cands[kWarps];
  __shared__ float warp_z[kWarps];
  __shared__ int warp_n[kWarps];
  pdl_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  float* row = probs + warp * width;
  if (blockIdx.x == 0 && threadIdx.x == 0) *p.done = 0;
  for (int e = threadIdx.x; e < p.E; e += kThreads) counts[e] = 0;
  if (SIG && p.bias != nullptr)
    for (int e = threadIdx.x; e < p.E; e += kThreads) bias[e] = p.bias[e];
  __syncthreads();
  const int first = blockIdx.x * p.tokens_per_cta;
  const int last = min(p.T, first + p.tokens_per_cta);
  int b = p.B > 1 ? sequence_of(p.seq_start, p.B, first) : 0;
  for (int t = first; t < last;) {
    while (b < p.B - 1 && p.seq_start[b + 1] <= t) ++b;
    const int end = b < p.B - 1 ? min(last, p.seq_start[b + 1]) : last;
    float sum[VPL], z = 0.0f;
    int n = 0;
#pragma unroll
    for (int r = 0; r < VPL; ++r) sum[r] = 0.0f;
    float x[VPL], s[VPL], total, top;
    int u = t + warp;
    if (kAhead<VPL> && u < end) load_row<VPL, V, BF16>(p.logits, int64_t(u) * p.ld, p.E, lane, x);
    for (; u < end; u += kWarps) {
      float next[VPL];
      if constexpr (kAhead<VPL>) {
        if (u + kWarps < end)
          load_row<VPL, V, BF16>(p.logits, int64_t(u + kWarps) * p.ld, p.E, lane, next);
      } else {
        load_row<VPL, V, BF16>(p.logits, int64_t(u) * p.ld, p.E, lane, x);
      }
      if (p.mask != nullptr && p.mask[u] == 0) {
        route_masked(p, u, lane);
      } else {
        const int mine = route_token<VPL, V, BF16, SIG, true>(p, u, lane, row, cands[warp], bias,
                                                              x, s, &total, &top);
        if (mine >= 0) atomicAdd(&counts[mine], 1);
        // total is 0 only where no expert is in service: the token adds nothing
        const float inv = total == 0.0f ? 0.0f : fast_reciprocal(total);
#pragma unroll
        for (int r = 0; r < VPL; ++r) sum[r] = fmaf(s[r], inv, sum[r]);
        ++n;
        if (!SIG && total != 0.0f) {
          const float lse = top + __logf(total);
          z += lse * lse;
        }
      }
      if constexpr (kAhead<VPL>) {
#pragma unroll
        for (int r = 0; r < VPL; ++r) x[r] = next[r];
      }
    }
    __syncwarp();
#pragma unroll
    for (int r = 0; r < VPL; ++r) {
      const int e = element_of<V>(r, lane);
      if (e < p.E) row[e] = sum[r];
    }
    if (lane == 0) {
      warp_z[warp] = z;
      warp_n[warp] = n;
    }
    __syncthreads();
    const int64_t part = int64_t(blockIdx.x) + b;
    for (int e = threadIdx.x; e < p.E; e += kThreads) {
      float acc = 0.0f;
#pragma unroll
      for (int v = 0; v < kWarps; ++v) acc += probs[v * width + e];
      p.part_prob[part * p.E + e] = acc;
      p.part_count[part * p.E + e] = counts[e];
      counts[e] = 0;
    }
    if (threadIdx.x == 0) {
      float zs = 0.0f;
      int ns = 0;
      for (int v = 0; v < kWarps; ++v) {
        zs += warp_z[v];
        ns += warp_n[v];
      }
      p.part_z[part] = zs;
      p.part_tokens[part] = ns;
    }
    __syncthreads();
    t = end;
  }
}

constexpr int kSumExperts = 8;       // of a CTA of the second kernel: a 32-byte sector of a row
constexpr int kSumRows = 32;         // partial rows it adds at a time
constexpr int kSumThreads = kSumExperts * kSumRows;

struct BalanceParams {
  const int32_t* seq_start;
  int T, E, K, B, tokens_per_cta;
  const float* part_prob;
  const int32_t* part_count;
  const int32_t* part_tokens;
  const float* part_z;
  int32_t* expert_count;   // [B, E]
  float* expert_prob;      // [B, E]
  int32_t* seq_tokens;     // [B + 2]
  float* dots;             // [B, gridDim.y]: a CTA's sum of count * prob / n
  float* seq_z;            // [B]
  unsigned* done;          // CTAs that have finished
  float* loss;             // [2]
};

// Sum over a block, in a fixed order, in every thread.  The block is whole
// warps, at most 32 of them.
template <typename T>
__device__ T block_sum(T v, T* scratch) {
#pragma unroll
  for (int d = 16; d; d >>= 1) v += __shfl_xor_sync(kFull, v, d);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) scratch[threadIdx.x >> 5] = v;
  __syncthreads();
  T s = T(0);
  for (int i = 0; i < int(blockDim.x >> 5); ++i) s += scratch[i];
  return s;
}

// Second kernel: CTA (b, i) adds up the partial rows of sequence b for the
// experts from kSumExperts i on, kSumRows rows at a time, in a fixed order;
// the CTA that finishes last forms the losses from what all have written.
__global__ void __launch_bounds__(kSumThreads) balance_sum_kernel(BalanceParams p) {
  __shared__ float probs[kSumRows][kSumExperts];
  __shared__ int counts[kSumRows][kSumExperts];
  __shared__ float fscratch[32];
  __shared__ int iscratch[32];
  __shared__ bool is_last;
  pdl_wait();
  const int b = blockIdx.x, lane = threadIdx.x % kSumExperts, part = threadIdx.x / kSumExperts;
  int e = blockIdx.y * kSumExperts + lane;
  const int lo = b == 0 ? 0 : min(max(p.seq_start[b], 0), p.T);
  const int hi = b == p.B - 1 ? p.T : min(max(p.seq_start[b + 1], 0), p.T);
  int c0 = 0, c1 = 0;
  if (hi > lo) {
    c0 = lo / p.tokens_per_cta;
    c1 = (hi - 1) / p.tokens_per_cta + 1;
  }
  float prob = 0.0f, z = 0.0f;
  int count = 0, n = 0;
  if (e < p.E) {
    const float* fp = p.part_prob + int64_t(c0 + b) * p.E + e;
    const int32_t* ip = p.part_count + int64_t(c0 + b) * p.E + e;
#pragma unroll 8
    for (int c = part; c < c1 - c0; c += kSumRows) {
      prob += fp[int64_t(c) * p.E];
      count += ip[int64_t(c) * p.E];
    }
  }
  for (int c = c0 + threadIdx.x; c < c1; c += kSumThreads) {
    n += p.part_tokens[c + b];
    z += p.part_z[c + b];
  }
  probs[part][lane] = prob;
  counts[part][lane] = count;
  n = block_sum(n, iscratch);
  z = block_sum(z, fscratch);
  if (threadIdx.x < 32) {      // lanes from kSumExperts on add nothing
    prob = 0.0f;
    count = 0;
    e = blockIdx.y * kSumExperts + threadIdx.x;
    const float inv_n = n > 0 ? 1.0f / float(n) : 0.0f;
    if (threadIdx.x < kSumExperts) {
#pragma unroll
      for (int r = 0; r < kSumRows; ++r) {
        prob += probs[r][threadIdx.x];
        count += counts[r][threadIdx.x];
      }
      prob *= inv_n;
      if (e < p.E) {
        p.expert_prob[int64_t(b) * p.E + e] = prob;
        p.expert_count[int64_t(b) * p.E + e] = count;
      }
    }
    const float dot = warp_sum(float(count) * inv_n * prob);
    if (threadIdx.x == 0) {
      p.dots[int64_t(b) * gridDim.y + blockIdx.y] = dot;
      if (blockIdx.y == 0) {
        p.seq_tokens[b] = n;
        p.seq_z[b] = z;
      }
      __threadfence();
      is_last = atomicAdd(p.done, 1u) == gridDim.x * gridDim.y - 1;
    }
  }
  __syncthreads();
  if (!is_last) return;
  __threadfence();
  float loss = 0.0f;
  int full = 0;
  n = 0;
  z = 0.0f;
  for (int64_t i = threadIdx.x; i < int64_t(p.B) * gridDim.y; i += kSumThreads)
    loss += __ldcg(p.dots + i);
  for (int i = threadIdx.x; i < p.B; i += kSumThreads) {
    const int m = __ldcg(p.seq_tokens + i);
    n += m;
    full += m > 0 ? 1 : 0;
    z += __ldcg(p.seq_z + i);
  }
  loss = block_sum(loss, fscratch);
  z = block_sum(z, fscratch);
  n = block_sum(n, iscratch);
  full = block_sum(full, iscratch);
  if (threadIdx.x == 0) {
    p.seq_tokens[p.B] = n;
    p.seq_tokens[p.B + 1] = full;
    p.loss[0] = full > 0 ? loss * (float(p.E) / float(p.K)) / float(full) : 0.0f;
    p.loss[1] = n > 0 ? z / float(n) : 0.0f;
  }
}

struct RouteBackwardParams {
  const void* logits;
  int64_t ld;
  const uint8_t* mask;
  int T, E, K, B, tokens_per_cta;
  bool renorm;
  float scale;
  const int64_t* idx;        // [T, K]
  const float* grad_w;       // [T, K] or null
  const int32_t* seq_start;
  const int32_t* expert_count;   // [B, E] or null (no losses)
  const int32_t* seq_tokens;     // [B + 2]
  const float* grad_loss;        // [2]
  void* grad;                // [T, ld_grad]
  int64_t ld_grad;
};

template <int VPL, int V, bool BF16>
__device__ __forceinline__ void store_row(void* base, int64_t offset, int E, int lane,
                                          const float (&g)[VPL]) {
#pragma unroll
  for (int r = 0; r < VPL; r += V) {
    const int e = element_of<V>(r, lane);
    if (e >= E) continue;
    if constexpr (V == 1) {
      if constexpr (BF16)
        static_cast<__nv_bfloat16*>(base)[offset + e] = __float2bfloat16_rn(g[r]);
      else
        static_cast<float*>(base)[offset + e] = g[r];
    } else {
      if constexpr (BF16) {
        *reinterpret_cast<uint2*>(static_cast<uint16_t*>(base) + offset + e) =
            make_uint2(pack_bf16x2(g[r], g[r + 1]), pack_bf16x2(g[r + 2], g[r + 3]));
      } else {
        *reinterpret_cast<float4*>(static_cast<float*>(base) + offset + e) =
            make_float4(g[r], g[r + 1], g[r + 2], g[r + 3]);
      }
    }
  }
}

// dL/dlogits of a token, all of it recomputed from its logits:
//   dq_e = g0 c_be E / (K n_b^2 B')       balance loss by the normalised score
//   ds_k = scale dw_k, or scale / S (dw_k - sum_j dw_j s_j / S)   gate weight
//   softmax:  g = dq + ds,  dl = s (g - sum s g + g1 2 lse / N)
//   sigmoid:  u = (dq - sum q dq) / sum s + ds,  dl = u s (1 - s)
template <int VPL, int V, bool BF16, bool SIG>
__global__ void __launch_bounds__(kRouteThreads) route_backward_kernel(RouteBackwardParams p) {
  extern __shared__ __align__(16) float smem[];
  pdl_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  float* row = smem + warp * padded_row(p.E);
  for (int e = lane; e < p.E; e += 32) row[e] = 0.0f;
  __syncwarp();
  const int first = blockIdx.x * p.tokens_per_cta;
  const int last = min(p.T, first + p.tokens_per_cta);
  float dq[VPL];
#pragma unroll
  for (int r = 0; r < VPL; ++r) dq[r] = 0.0f;
  float dlse = 0.0f;
  const bool losses = p.expert_count != nullptr;
  if (losses && !SIG) {
    const int n = p.seq_tokens[p.B];
    dlse = n > 0 ? p.grad_loss[1] * 2.0f / float(n) : 0.0f;
  }
  int b = -1;
  // a token's logits, choice and gate gradient are loaded a token ahead
  float x[VPL], s[VPL], top, dw = 0.0f;
  int64_t choice = -1;
  const bool selects = p.grad_w != nullptr && lane < p.K;
  const auto load_choice = [&](int t, int64_t& e, float& g) {
    e = p.idx[int64_t(t) * p.K + lane];
    g = p.grad_w[int64_t(t) * p.K + lane];
  };
  int t = first + warp;
  if (t < last) {
    if constexpr (kAhead<VPL>) load_row<VPL, V, BF16>(p.logits, int64_t(t) * p.ld, p.E, lane, x);
    if (selects) load_choice(t, choice, dw);
  }
  for (; t < last; t += kRouteWarps) {
    float next[VPL], next_dw = 0.0f;
    int64_t next_choice = -1;
    if (t + kRouteWarps < last) {
      if constexpr (kAhead<VPL>)
        load_row<VPL, V, BF16>(p.logits, int64_t(t + kRouteWarps) * p.ld, p.E, lane, next);
      if (selects) load_choice(t + kRouteWarps, next_choice, next_dw);
    }
    if constexpr (!kAhead<VPL>)
      load_row<VPL, V, BF16>(p.logits, int64_t(t) * p.ld, p.E, lane, x);
    float g[VPL];
    if (p.mask != nullptr && p.mask[t] == 0) {
#pragma unroll
      for (int r = 0; r < VPL; ++r) g[r] = 0.0f;
    } else {
      if (losses) {
        const int was = b;
        if (b < 0)
          b = p.B > 1 ? sequence_of(p.seq_start, p.B, t) : 0;
        else
          while (b < p.B - 1 && p.seq_start[b + 1] <= t) ++b;
        if (b != was) {
          const int n = p.seq_tokens[b], full = p.seq_tokens[p.B + 1];
          const float each = n > 0 && full > 0 ? p.grad_loss[0] * (float(p.E) / float(p.K)) /
                                                     (float(n) * float(n) * float(full))
                                               : 0.0f;
#pragma unroll
          for (int r = 0; r < VPL; ++r) {
            const int e = element_of<V>(r, lane);
            dq[r] = e < p.E ? each * float(p.expert_count[int64_t(b) * p.E + e]) : 0.0f;
          }
        }
      }
      // gate weights: lane k holds selection k
      const int mine = choice >= 0 && choice < p.E ? int(choice) : -1;
      const float l = mine >= 0 ? load_one<BF16>(p.logits, int64_t(t) * p.ld + mine) : 0.0f;
      const float total = scores<VPL, SIG>(x, s, &top);
      const float inv = total == 0.0f ? 0.0f : fast_reciprocal(total);
      if (p.grad_w != nullptr) {
        float ds = 0.0f, sk = 0.0f;
        if (mine >= 0) {
          sk = SIG ? sigmoid(l) : soft_score(l, top) * inv;
          ds = dw * p.scale;
        }
        if (p.renorm) {
          const float sum = warp_sum(sk);
          const float is = sum == 0.0f ? 0.0f : fast_reciprocal(sum);
          const float mean = warp_sum(ds * sk) * is;
          ds = (ds - mean) * is;
        }
        if (mine >= 0) row[mine] = ds;
        __syncwarp();
        read_row<VPL, V>(row, p.E, lane, g);
        __syncwarp();
        if (mine >= 0) row[mine] = 0.0f;
      } else {
#pragma unroll
        for (int r = 0; r < VPL; ++r) g[r] = 0.0f;
      }
      float dot = 0.0f;
#pragma unroll
      for (int r = 0; r < VPL; ++r) {
        if constexpr (SIG) {
          dot = fmaf(s[r], dq[r], dot);
        } else {
          s[r] *= inv;
          g[r] += dq[r];
          dot = fmaf(s[r], g[r], dot);
        }
      }
      dot = warp_sum(dot);
      if constexpr (SIG) {
        dot *= inv;
#pragma unroll
        for (int r = 0; r < VPL; ++r)
          g[r] = fmaf(dq[r] - dot, inv, g[r]) * (s[r] * (1.0f - s[r]));
      } else {
        const float z = total != 0.0f ? dlse * (top + __logf(total)) : 0.0f;
#pragma unroll
        for (int r = 0; r < VPL; ++r) g[r] = s[r] * (g[r] - (dot - z));
      }
    }
    store_row<VPL, V, BF16>(p.grad, int64_t(t) * p.ld_grad, p.E, lane, g);
    __syncwarp();
    choice = next_choice;
    dw = next_dw;
    if constexpr (kAhead<VPL>) {
#pragma unroll
      for (int r = 0; r < VPL; ++r) x[r] = next[r];
    }
  }
}

// ---- host -----------------------------------------------------------------

bool aligned(const void* p) { return p != nullptr && (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool aligned_or_null(const void* p) { return p == nullptr || aligned(p); }

bool router_ok(const ep_router_config* c) {
  if (c == nullptr) return false;
  if (c->num_experts < 1 || c->num_experts > 2048) return false;
  if (c->num_topk < 1 || c->num_topk > 32 || c->num_topk > c->num_experts) return false;
  if (c->score != EP_SCORE_SOFTMAX && c->score != EP_SCORE_SIGMOID) return false;
  if (c->num_groups < 1 || c->num_groups > kMaxGroups) return false;
  if (c->num_experts % c->num_groups != 0) return false;
  if (c->topk_groups < 1 || c->topk_groups > c->num_groups) return false;
  if (int64_t(c->num_experts / c->num_groups) * c->topk_groups < c->num_topk) return false;
  if (c->renormalize != 0 && c->renormalize != 1) return false;
  if (c->logits_bf16 != 0 && c->logits_bf16 != 1) return false;
  return c->route_scale == c->route_scale;   // not NaN
}

constexpr int kMaxSequences = 1 << 20;

// CTAs of the per-token kernels over `tokens` tokens: at most four an SM
// (32 warps), each warp with a token at least.
constexpr int kRouteCtasPerSm = 4;
int route_ctas(int tokens) {
  const int want = (tokens + kRouteWarps - 1) / kRouteWarps;
  const int most = device_info().sm_count * kRouteCtasPerSm;
  return want < most ? want : most;
}

// Calls f.template operator()<VPL, V, BF16, SIG>() for the smallest VPL that
// holds E logits in a warp.  Rows whose vectors of four are aligned load
// those; narrow rows keep more lanes busy with single loads.
template <typename F>
cudaError_t with_shape(int E, int64_t ld, bool bf16, bool sig, F&& f) {
  const bool vec = E >= 128 && E <= 512 && E % 4 == 0 && ld % 4 == 0;
  int vpl = vec ? 4 : 1;
  while (vpl * 32 < E) vpl *= 2;
#define EP_SHAPE(N, W)                                                    \
  if (vpl == N && vec == (W == 4)) {                                      \
    if (bf16) return sig ? f.template operator()<N, W, true, true>()      \
                         : f.template operator()<N, W, true, false>();    \
    return sig ? f.template operator()<N, W, false, true>()               \
               : f.template operator()<N, W, false, false>();             \
  }
  EP_SHAPE(1, 1) EP_SHAPE(2, 1) EP_SHAPE(4, 1) EP_SHAPE(8, 1) EP_SHAPE(16, 1)
  EP_SHAPE(32, 1) EP_SHAPE(64, 1)
  EP_SHAPE(4, 4) EP_SHAPE(8, 4) EP_SHAPE(16, 4)
#undef EP_SHAPE
  return cudaErrorInvalidValue;
}

// Raises a kernel's dynamic shared-memory limit where `bytes` needs it (48 KiB
// with the static arrays, which are under 8, need no leave).
template <typename... P>
cudaError_t allow_smem(void (*kernel)(P...), size_t bytes) {
  if (bytes <= 40 * 1024) return cudaSuccess;
  return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, int(bytes));
}

struct LaunchRoute {
  RouteParams p;
  int ctas;
  cudaStream_t stream;
  template <int VPL, int V, bool BF16, bool SIG>
  cudaError_t operator()() const {
    const size_t rows = p.G > 1 ? kRouteWarps + 1 : SIG ? 1 : 0;
    const size_t smem = sizeof(float) * rows * padded_row(p.E);
    auto* kernel = route_kernel<VPL, V, BF16, SIG>;
    const cudaError_t e = allow_smem(kernel, smem);
    if (e != cudaSuccess) return e;
    return launch_pdl(kernel, dim3(ctas), dim3(kRouteThreads), smem, stream, p);
  }
};

// CTAs of the second kernel along the experts.
int sum_ctas(int E) { return (E + kSumExperts - 1) / kSumExperts; }

struct LaunchBalance {
  RouteParams p;
  BalanceParams q;      // of the second kernel
  cudaStream_t stream;
  template <int VPL, int V, bool BF16, bool SIG>
  cudaError_t operator()() {
    constexpr int kThreads = kBalanceThreads<VPL>, kWarps = kThreads / 32;
    // each warp with a token at least; no tokens: one CTA still clears `done`
    const int want = (p.T + kWarps - 1) / kWarps;
    const int most = device_info().sm_count * kBalanceCtasPerSm<VPL>;
    const int ctas = want < most ? (want > 1 ? want : 1) : most;
    p.tokens_per_cta = q.tokens_per_cta = p.T > 0 ? (p.T + ctas - 1) / ctas : 1;
    const int used = p.T > 0 ? (p.T + p.tokens_per_cta - 1) / p.tokens_per_cta : 1;
    const size_t smem = sizeof(float) * (kWarps + 2) * padded_row(p.E);
    auto* kernel = balance_kernel<VPL, V, BF16, SIG>;
    cudaError_t e = allow_smem(kernel, smem);
    if (e != cudaSuccess) return e;
    e = launch_pdl(kernel, dim3(used), dim3(kThreads), smem, stream, p);
    if (e != cudaSuccess) return e;
    return launch_pdl(balance_sum_kernel, dim3(p.B, sum_ctas(p.E)), dim3(kSumThreads), 0, stream,
                      q);
  }
};

struct LaunchBackward {
  RouteBackwardParams p;
  int ctas;
  cudaStream_t stream;
  template <int VPL, int V, bool BF16, bool SIG>
  cudaError_t operator()() const {
    const size_t smem = sizeof(float) * kRouteWarps * padded_row(p.E);
    auto* kernel = route_backward_kernel<VPL, V, BF16, SIG>;
    const cudaError_t e = allow_smem(kernel, smem);
    if (e != cudaSuccess) return e;
    return launch_pdl(kernel, dim3(ctas), dim3(kRouteThreads), smem, stream, p);
  }
};

// Tokens per CTA of the kernels that give each CTA a run of tokens.
int run_length(int T) {
  const int ctas = route_ctas(T);
  return ctas > 0 ? (T + ctas - 1) / ctas : 1;
}

struct BalanceWorkspace {
  float* prob;
  int32_t* count;
  int32_t* tokens;
  float* z;
  float* dots;
  float* seq_z;
  unsigned* done;
  int64_t bytes;
};

// The first kernel has at most two CTAs an SM, whatever T.
BalanceWorkspace carve(void* base, int E, int B) {
  const int64_t rows = int64_t(device_info().sm_count) * 2 + B;
  char* at = static_cast<char*>(base);
  auto take = [&](int64_t n) {
    char* p = at;
    at += (n * 4 + 15) / 16 * 16;
    return p;
  };
  BalanceWorkspace w;
  w.prob = reinterpret_cast<float*>(take(rows * E));
  w.count = reinterpret_cast<int32_t*>(take(rows * E));
  w.tokens = reinterpret_cast<int32_t*>(take(rows));
  w.z = reinterpret_cast<float*>(take(rows));
  w.dots = reinterpret_cast<float*>(take(int64_t(B) * sum_ctas(E)));
  w.done = reinterpret_cast<unsigned*>(take(1));
  w.seq_z = reinterpret_cast<float*>(take(B));
  w.bytes = at - static_cast<char*>(base);
  return w;
}

int32_t status(cudaError_t e) { return note_cuda(e) == cudaSuccess ? EP_OK : EP_ERR_CUDA; }

// Checks shared by the two forward entry points.
bool route_args(const ep_router_config* cfg, int32_t T, const void* d_logits, int64_t ld,
                const float* d_bias, const uint8_t* d_mask, int64_t* d_idx, float* d_w,
                RouteParams* p) {
  if (!router_ok(cfg) || T < 0 || ld < cfg->num_experts) return false;
  if (d_bias != nullptr && cfg->score != EP_SCORE_SIGMOID) return false;
  if (!aligned_or_null(d_bias) || !aligned_or_null(d_mask)) return false;
  if (T > 0 && (!aligned(d_logits) || !aligned(d_idx) || !aligned(d_w))) return false;
  *p = RouteParams{};
  p->logits = d_logits;
  p->ld = ld;
  p->bias = d_bias;
  p->mask = d_mask;
  p->T = T;
  p->E = cfg->num_experts;
  p->K = cfg->num_topk;
  p->G = cfg->num_groups;
  p->kept = cfg->topk_groups;
  if (p->kept == p->G) p->G = p->kept = 1;
  p->per = p->E / p->G;
  p->per_log2 = -1;
  for (int i = 2; i <= 7; ++i)
    if (p->per == 1 << i) p->per_log2 = i;
  // floor(2^21 / per) + 1 is off by under 2^-21 of e < 2^11, less than the
  // 1 / per that the quotient is from the next whole number (per <= 2^10)
  p->per_inverse = (1u << 21) / uint32_t(p->per) + 1u;
  p->renorm = cfg->renormalize != 0;
  p->scale = cfg->route_scale;
  p->idx = d_idx;
  p->w = d_w;
  p->B = 1;
  return true;
}

}  // namespace
}  // namespace ep

using namespace ep;

extern "C" {

int32_t ep_route(const ep_router_config* cfg, int32_t num_tokens, const void* d_logits,
                 int64_t ld_logits, const float* d_bias, const uint8_t* d_token_mask,
                 int64_t* d_topk_idx, float* d_topk_weights, void* stream) {
  LaunchRoute l;
  if (!route_args(cfg, num_tokens, d_logits, ld_logits, d_bias, d_token_mask, d_topk_idx,
                  d_topk_weights, &l.p))
    return EP_ERR_INVALID_ARG;
  if (num_tokens == 0) return EP_OK;
  l.ctas = route_ctas(num_tokens);
  l.stream = static_cast<cudaStream_t>(stream);
  return status(with_shape(l.p.E, ld_logits, cfg->logits_bf16 != 0,
                           cfg->score == EP_SCORE_SIGMOID, l));
}

int64_t ep_route_workspace_bytes(const ep_router_config* cfg, int32_t num_seqs) {
  if (!router_ok(cfg) || num_seqs < 1 || num_seqs > kMaxSequences) return -1;
  return carve(nullptr, cfg->num_experts, num_seqs).bytes;
}

int32_t ep_route_balance(const ep_router_config* cfg, int32_t num_tokens, const void* d_logits,
                         int64_t ld_logits, const float* d_bias, const uint8_t* d_token_mask,
                         int32_t num_seqs, const int32_t* d_seq_start, int64_t* d_topk_idx,
                         float* d_topk_weights, int32_t* d_expert_count, float* d_expert_prob,
                         int32_t* d_seq_tokens, float* d_loss, void* d_workspace,
                         void* stream) {
  LaunchBalance l;
  if (!route_args(cfg, num_tokens, d_logits, ld_logits, d_bias, d_token_mask, d_topk_idx,
                  d_topk_weights, &l.p))
    return EP_ERR_INVALID_ARG;
  if (num_seqs < 1 || num_seqs > kMaxSequences) return EP_ERR_INVALID_ARG;
  if (num_seqs > 1 && d_seq_start == nullptr) return EP_ERR_INVALID_ARG;
  if (!aligned_or_null(d_seq_start) || !aligned(d_expert_count) || !aligned(d_expert_prob) ||
      !aligned(d_seq_tokens) || !aligned(d_loss) || !aligned(d_workspace))
    return EP_ERR_INVALID_ARG;
  const BalanceWorkspace w = carve(d_workspace, l.p.E, num_seqs);
  l.stream = static_cast<cudaStream_t>(stream);
  l.p.seq_start = d_seq_start;
  l.p.B = num_seqs;
  l.p.part_prob = w.prob;
  l.p.part_count = w.count;
  l.p.part_tokens = w.tokens;
  l.p.part_z = w.z;
  l.p.done = w.done;
  l.q.seq_start = d_seq_start;
  l.q.T = num_tokens;
  l.q.E = l.p.E;
  l.q.K = l.p.K;
  l.q.B = num_seqs;
  l.q.part_prob = w.prob;
  l.q.part_count = w.count;
  l.q.part_tokens = w.tokens;
  l.q.part_z = w.z;
  l.q.expert_count = d_expert_count;
  l.q.expert_prob = d_expert_prob;
  l.q.seq_tokens = d_seq_tokens;
  l.q.dots = w.dots;
  l.q.seq_z = w.seq_z;
  l.q.done = w.done;
  l.q.loss = d_loss;
  return status(with_shape(l.p.E, ld_logits, cfg->logits_bf16 != 0,
                           cfg->score == EP_SCORE_SIGMOID, l));
}

int32_t ep_route_backward(const ep_router_config* cfg, int32_t num_tokens, const void* d_logits,
                          int64_t ld_logits, const uint8_t* d_token_mask,
                          const int64_t* d_topk_idx, const float* d_grad_w, int32_t num_seqs,
                          const int32_t* d_seq_start, const int32_t* d_expert_count,
                          const int32_t* d_seq_tokens, const float* d_grad_loss,
                          void* d_grad_logits, int64_t ld_grad, void* stream) {
  if (!router_ok(cfg) || num_tokens < 0) return EP_ERR_INVALID_ARG;
  if (ld_logits < cfg->num_experts || ld_grad < cfg->num_experts) return EP_ERR_INVALID_ARG;
  if (num_seqs < 1 || num_seqs > kMaxSequences) return EP_ERR_INVALID_ARG;
  if (num_tokens > 0 && (!aligned(d_logits) || !aligned(d_grad_logits)))
    return EP_ERR_INVALID_ARG;
  const void* optional[] = {d_token_mask, d_topk_idx, d_grad_w, d_seq_start,
                            d_expert_count, d_seq_tokens, d_grad_loss};
  for (const void* o : optional)
    if (!aligned_or_null(o)) return EP_ERR_INVALID_ARG;
  // gate weights need the choice; the losses need all three of their inputs
  if (d_grad_w != nullptr && d_topk_idx == nullptr) return EP_ERR_INVALID_ARG;
  const int set = (d_expert_count != nullptr) + (d_seq_tokens != nullptr) +
                  (d_grad_loss != nullptr);
  if (set != 0 && set != 3) return EP_ERR_INVALID_ARG;
  if (set == 3 && num_seqs > 1 && d_seq_start == nullptr) return EP_ERR_INVALID_ARG;
  if (num_tokens == 0) return EP_OK;
  LaunchBackward l;
  l.p = RouteBackwardParams{};
  l.p.logits = d_logits;
  l.p.ld = ld_logits;
  l.p.mask = d_token_mask;
  l.p.T = num_tokens;
  l.p.E = cfg->num_experts;
  l.p.K = cfg->num_topk;
  l.p.B = num_seqs;
  l.p.tokens_per_cta = run_length(num_tokens);
  l.p.renorm = cfg->renormalize != 0;
  l.p.scale = cfg->route_scale;
  l.p.idx = d_topk_idx;
  l.p.grad_w = d_grad_w;
  l.p.seq_start = d_seq_start;
  l.p.expert_count = d_expert_count;
  l.p.seq_tokens = d_seq_tokens;
  l.p.grad_loss = d_grad_loss;
  l.p.grad = d_grad_logits;
  l.p.ld_grad = ld_grad;
  l.ctas = (num_tokens + l.p.tokens_per_cta - 1) / l.p.tokens_per_cta;
  l.stream = static_cast<cudaStream_t>(stream);
  // both rows have to allow vectors for either to use them
  const int64_t ld = ld_logits % 4 == 0 ? ld_grad : ld_logits;
  return status(with_shape(l.p.E, ld, cfg->logits_bf16 != 0, cfg->score == EP_SCORE_SIGMOID, l));
}

}  // extern "C"

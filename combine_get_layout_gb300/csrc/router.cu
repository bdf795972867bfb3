// The router gate on the GPU: scores, grouped top-K choice and gate weights
// (ep_route), the same with the balance and z losses (ep_route_balance), and
// the gradient of both by the logits (ep_route_backward).
//
// A tile of 8, 16 or 32 lanes of a warp owns one token at a time and holds
// its E logits in registers, so that a token's row is read once and every
// sum over experts is a few shuffles; narrow tiles (few experts) put several
// tokens in a warp, which shares the instructions that do not depend on the
// number of experts.  The statistics of the losses are summed in registers
// over a CTA's run of tokens, then once per (CTA, sequence), in a fixed
// order: no floating-point atomics, so the same inputs give the same bits.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <math_constants.h>

#include <atomic>
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

// A tile of `L` lanes with `N` fp32 or bf16 logits each, loaded in vectors of
// `V` neighbours (1 or 4).
template <int L, int N, int V, bool BF16>
struct Shape {
  static constexpr int kLanes = L, kValues = N, kVec = V;
  static constexpr bool kBf16 = BF16;
  static constexpr int kTiles = 32 / L;             // tokens of a warp
  static constexpr int kRuns = 32 / L < N ? 32 / L : N;   // of a lane's logits, see choose()
  static constexpr int kSlots = L == 8 ? 2 : 1;     // candidates a lane
  static constexpr int kCandidates = L * kSlots;    // of a token
  // logits that are loaded a token ahead: where two rows fit the registers
  static constexpr bool kAhead = N <= 16;
  // Expert of register r of lane l of the tile.
  static __device__ __forceinline__ int expert(int r, int l) { return (r / V * L + l) * V + r % V; }
};

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

// ---- rows -----------------------------------------------------------------

template <class S>
__device__ __forceinline__ float load_one(const void* base, int64_t at) {
  if constexpr (S::kBf16)
    return __uint_as_float(uint32_t(static_cast<const uint16_t*>(base)[at]) << 16);
  else
    return static_cast<const float*>(base)[at];
}

// A token's logits in registers, -inf past the last expert and, where !have,
// throughout.
template <class S>
__device__ __forceinline__ void load_row(const void* base, int64_t offset, int E, int l, bool have,
                                         float (&x)[S::kValues]) {
  const int limit = have ? E : 0;
#pragma unroll
  for (int r = 0; r < S::kValues; r += S::kVec) {
    const int e = S::expert(r, l);
#pragma unroll
    for (int i = 0; i < S::kVec; ++i) x[r + i] = -CUDART_INF_F;
    if (e >= limit) continue;
    if constexpr (S::kVec == 1) {
      x[r] = load_one<S>(base, offset + e);
    } else if constexpr (S::kBf16) {
      const uint2 v =
          *reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(base) + offset + e);
      x[r] = bf16_lo(v.x);
      x[r + 1] = bf16_hi(v.x);
      x[r + 2] = bf16_lo(v.y);
      x[r + 3] = bf16_hi(v.y);
    } else {
      const float4 v = *reinterpret_cast<const float4*>(static_cast<const float*>(base) + offset + e);
      x[r] = v.x;
      x[r + 1] = v.y;
      x[r + 2] = v.z;
      x[r + 3] = v.w;
    }
  }
}

template <class S>
__device__ __forceinline__ void store_row(void* base, int64_t offset, int E, int l,
                                          const float (&g)[S::kValues]) {
#pragma unroll
  for (int r = 0; r < S::kValues; r += S::kVec) {
    const int e = S::expert(r, l);
    if (e >= E) continue;
    if constexpr (S::kVec == 1) {
      if constexpr (S::kBf16)
        static_cast<__nv_bfloat16*>(base)[offset + e] = __float2bfloat16_rn(g[r]);
      else
        static_cast<float*>(base)[offset + e] = g[r];
    } else if constexpr (S::kBf16) {
      *reinterpret_cast<uint2*>(static_cast<uint16_t*>(base) + offset + e) =
          make_uint2(pack_bf16x2(g[r], g[r + 1]), pack_bf16x2(g[r + 2], g[r + 3]));
    } else {
      *reinterpret_cast<float4*>(static_cast<float*>(base) + offset + e) =
          make_float4(g[r], g[r + 1], g[r + 2], g[r + 3]);
    }
  }
}

// Floats of a row of E in shared memory: whole vectors of four.
__host__ __device__ __forceinline__ int padded_row(int E) { return (E + 3) & ~3; }

// A lane's values of a row of E floats in shared memory (16-byte aligned).
template <class S>
__device__ __forceinline__ void read_row(const float* row, int E, int l, float (&v)[S::kValues]) {
#pragma unroll
  for (int r = 0; r < S::kValues; r += S::kVec) {
    const int e = S::expert(r, l);
    if constexpr (S::kVec == 4) {
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

// ---- tiles ----------------------------------------------------------------

template <int L>
__device__ __forceinline__ float tile_sum(float v) {
#pragma unroll
  for (int d = L / 2; d; d >>= 1) v += __shfl_xor_sync(kFull, v, d);
  return v;
}

// A choice bias as the kernels keep it: NaN takes its expert out of the choice,
// as -inf does, so that no choice score is NaN.
__device__ __forceinline__ float clean_bias(float b) { return fmaxf(b, -CUDART_INF_F); }

// Largest of a tile's values; a NaN counts only where all are NaN.
template <int L>
__device__ __forceinline__ float tile_max(float v) {
  if constexpr (L == 32) {
    float m;
    asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(m) : "f"(v));
    return m;
  } else {
#pragma unroll
    for (int d = L / 2; d; d >>= 1) v = fmaxf(v, __shfl_xor_sync(kFull, v, d));
    return v;
  }
}

// The larger and the smaller, or NaN if either is.
__device__ __forceinline__ float max_or_nan(float a, float b) {
  float m;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(m) : "f"(a), "f"(b));
  return m;
}

__device__ __forceinline__ float min_or_nan(float a, float b) {
  float m;
  asm("min.NaN.f32 %0, %1, %2;" : "=f"(m) : "f"(a), "f"(b));
  return m;
}

// Bits of a ballot that belong to this lane's tile, from bit 0.
template <int L>
__device__ __forceinline__ uint32_t tile_bits(uint32_t ballot, int lane) {
  if constexpr (L == 32)
    return ballot;
  else
    return ballot >> (lane & ~(L - 1)) & ((1u << L) - 1u);
}

// ---- scores ---------------------------------------------------------------

constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

// 2^x and 1 / x to 2^-22 of the value, or 0 below 2^-126.
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

// exp(d) for -128 <= d <= 88.  t = d log2 e is rounded to up to 2^-17 of an
// exponent near 128, so that 2^t would be off by up to 4e-6 of its value;
// d - t ln 2 is what the rounding left out, and exp of it 1 + itself.
__device__ __forceinline__ float exponential(float d) {
  const float t = d * kLog2e, e = fast_exp2(t);
  return fmaf(e, fmaf(-t, kLn2, d), e);
}

// a / b for 0 <= a <= b, given 1 / b to within a few roundings: the product,
// and its residual as one correction (Newton's step for a quotient).  a / a
// is 1: the correction of 1 - 2^-24 or 1 + 2^-23 rounds to it.
__device__ __forceinline__ float quotient(float a, float b, float inv_b) {
  const float q = a * inv_b;
  return fmaf(fmaf(-q, b, a), inv_b, q);
}

// Under 2^-126 (x below -87.3) it is 0.
__device__ __forceinline__ float sigmoid(float x) {
  const float d = min_or_nan(max_or_nan(-x, -128.0f), 88.0f);
  return fast_reciprocal(1.0f + exponential(d));
}

// exp(l - top), 0 under 2^-126; the difference first, so that no size of
// logit overflows.
__device__ __forceinline__ float soft_score(float l, float top) {
  return exponential(max_or_nan(l - top, -128.0f));
}

template <int N>
__device__ __forceinline__ float largest(const float (&x)[N]) {
  float m = x[0];
#pragma unroll
  for (int r = 1; r < N; ++r) m = fmaxf(m, x[r]);
  return m;
}

// Softmax scores of a token before their division: s = exp(x - top), top the
// row's maximum; returns their total.  -inf scores 0, and so does all of a
// row of nothing else.
template <class S>
__device__ __forceinline__ float soft_scores(const float (&x)[S::kValues], float (&s)[S::kValues],
                                             float top) {
  const float base = top == -CUDART_INF_F ? 0.0f : top;
  float total = 0.0f;
#pragma unroll
  for (int r = 0; r < S::kValues; ++r) {
    s[r] = soft_score(x[r], base);
    total += s[r];
  }
  return tile_sum<S::kLanes>(total);
}

// Scores of a token, as soft_scores or sigmoid has them, their total, and
// (softmax) the row's maximum.
template <class S, bool SIG>
__device__ __forceinline__ float scores(const float (&x)[S::kValues], float (&s)[S::kValues],
                                        float* top) {
  if constexpr (SIG) {
    float total = 0.0f;
#pragma unroll
    for (int r = 0; r < S::kValues; ++r) {
      s[r] = sigmoid(x[r]);      // exp2(+inf) = inf, its reciprocal 0
      total += s[r];
    }
    *top = 0.0f;
    return tile_sum<S::kLanes>(total);
  } else {
    *top = tile_max<S::kLanes>(largest(x));
    return soft_scores<S>(x, s, *top);
  }
}

// ---- groups ---------------------------------------------------------------

// The `kept` best of G groups by the scores that lanes l < G hold, as a bit
// mask; equal scores go to the lower group, -inf is never kept.  No NaN
// reaches this.
template <class S>
__device__ __forceinline__ uint32_t best_groups(float score, int G, int kept, int lane) {
  const int l = lane % S::kLanes;
  if constexpr (S::kLanes == 32) {      // a maximum is one instruction: one after another
    uint32_t keep = 0;
    float left = l < G ? score : -CUDART_INF_F;
    for (int i = 0; i < kept; ++i) {
      const float top = tile_max<32>(left);
      const uint32_t first = __ballot_sync(kFull, left == top);
      const uint32_t one = first & (0u - first);
      keep |= one;
      if (one >> l & 1u) left = -CUDART_INF_F;
    }
    // groups of no score answer last, if at all
    return keep & __ballot_sync(kFull, l < G && score > -CUDART_INF_F);
  } else {
    int before = 0;
    for (int g = 0; g < G; ++g) {
      const float o = __shfl_sync(kFull, score, g, S::kLanes);
      before += o > score || (o == score && g < l) ? 1 : 0;
    }
    const bool in = l < G && before < kept && score > -CUDART_INF_F;
    return tile_bits<S::kLanes>(__ballot_sync(kFull, in), lane);
  }
}

// Adds (b, s) of another set to a running (best, second).
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
// experts up to four a lane are whole aligned runs of the lanes of one
// vector (V = 4), and reduce by shuffles; other sizes go through the tile's
// shared scratch of E floats.
template <class S, bool SIG>
__device__ __forceinline__ void keep_groups(const RouteParams& p, float (&c)[S::kValues], float* row,
                                            int lane) {
  constexpr int L = S::kLanes;
  const int l = lane % L;
  if constexpr (!SIG) {      // a NaN is not chosen; sigmoid choice scores have none
#pragma unroll
    for (int r = 0; r < S::kValues; ++r) c[r] = fmaxf(c[r], -CUDART_INF_F);
  }
  if constexpr (S::kVec == 4) {
    constexpr int kLog = L == 8 ? 3 : L == 16 ? 4 : 5;
    if (p.per_log2 > 0 && p.per_log2 - 2 <= kLog) {
      // a group is 2^span lanes of a vector, a vector 2^(kLog - span) groups
      const int span = p.per_log2 - 2, of_vector = kLog - span;
      const int at = (l & ((1 << of_vector) - 1)) << span;      // where group l begins
      float mine = -CUDART_INF_F;
#pragma unroll
      for (int v = 0; v < S::kValues / 4; ++v) {
        const float hi0 = fmaxf(c[4 * v], c[4 * v + 1]), lo0 = fminf(c[4 * v], c[4 * v + 1]);
        const float hi1 = fmaxf(c[4 * v + 2], c[4 * v + 3]);
        const float lo1 = fminf(c[4 * v + 2], c[4 * v + 3]);
        float best = hi0, second = lo0;
        top_two(best, second, hi1, lo1);
#pragma unroll
        for (int i = 0; i < kLog; ++i) {
          if (i >= span) break;
          const float b = __shfl_xor_sync(kFull, best, 1 << i);
          if constexpr (SIG) {
            const float s = __shfl_xor_sync(kFull, second, 1 << i);
            top_two(best, second, b, s);
          } else {
            best = fmaxf(best, b);
          }
        }
        const float score = __shfl_sync(kFull, group_score<SIG>(best, second), at, L);
        if (l >> of_vector == v) mine = score;
      }
      const uint32_t keep = best_groups<S>(mine, p.G, p.kept, lane);
#pragma unroll
      for (int v = 0; v < S::kValues / 4; ++v) {
        const int g = (v << of_vector) + (l >> span);
        if (!((keep >> (g & 31)) & 1u)) {
#pragma unroll
          for (int i = 0; i < 4; ++i) c[4 * v + i] = -CUDART_INF_F;
        }
      }
      return;
    }
  }
#pragma unroll
  for (int r = 0; r < S::kValues; ++r) {
    const int e = S::expert(r, l);
    if (e < p.E) row[e] = c[r];
  }
  __syncwarp();
  float best = -CUDART_INF_F, second = -CUDART_INF_F;
  if (l < p.G)
    for (int i = 0; i < p.per; ++i) top_two(best, second, row[l * p.per + i], -CUDART_INF_F);
  const uint32_t keep = best_groups<S>(group_score<SIG>(best, second), p.G, p.kept, lane);
#pragma unroll
  for (int r = 0; r < S::kValues; ++r) {
    const int e = S::expert(r, l);
    if (e < p.E && !((keep >> (e * p.per_inverse >> 21)) & 1u)) c[r] = -CUDART_INF_F;
  }
  __syncwarp();
}

// ---- choice ---------------------------------------------------------------

// The K largest of a tile's choice scores one after another, equal ones by
// ascending index: lane k of the tile returns the k-th expert or -1.
template <class S>
__device__ __noinline__ int choose_in_turn(float (&c)[S::kValues], int K, int l) {
  int mine = -1;
  for (int k = 0; k < K; ++k) {
    float best = -CUDART_INF_F;
    int at = 0x7fffffff;
#pragma unroll
    for (int r = 0; r < S::kValues; ++r) {
      if (c[r] > best) {
        best = c[r];
        at = S::expert(r, l);
      }
    }
    const float top = tile_max<S::kLanes>(best);
    int win = best == top && top > -CUDART_INF_F ? at : 0x7fffffff;
#pragma unroll
    for (int d = S::kLanes / 2; d; d >>= 1) win = min(win, __shfl_xor_sync(kFull, win, d));
#pragma unroll
    for (int r = 0; r < S::kValues; ++r)
      if (S::expert(r, l) == win) c[r] = -CUDART_INF_F;
    if (l == k && top > -CUDART_INF_F) mine = win;
  }
  return mine;
}

// A set of the registers 0 .. N - 1.
template <int N>
struct RegisterSet {
  using Bits = std::conditional_t<(N > 32), unsigned long long, uint32_t>;
  Bits bits = 0;
  __device__ __forceinline__ void add(int r, bool in) { bits |= in ? Bits(1) << r : Bits(0); }
  __device__ __forceinline__ int first() const {
    if constexpr (N > 32) return __ffsll(bits) - 1;
    return __ffs(bits) - 1;
  }
  __device__ __forceinline__ void drop_first() { bits &= bits - 1; }
};

// What a tile's lanes share while they choose.
template <class S>
struct __align__(16) Candidates {
  unsigned long long key[S::kCandidates];
  int expert[S::kCandidates];
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
template <class S>
struct Chosen {
  int e[S::kSlots], rank[S::kSlots];
  float l[S::kSlots];
};

// Chooses the K largest of a tile's choice scores c; -inf and NaN are never
// chosen.  A lane's scores are taken as kRuns runs, 32 runs a token, and the
// K-th largest of the runs' maxima (equal ones of different lanes taken
// together) is a bound that at least K scores reach, where K can be chosen
// at all; with the best scores spread over the runs few more do.  Those
// become candidates that each count the candidates before them.  More than
// kCandidates (many equal scores, K near the lanes) are chosen in turn.
template <class S, bool SIG>
__device__ __forceinline__ Chosen<S> choose(const RouteParams& p, const float (&c)[S::kValues],
                                            int64_t offset, int lane, Candidates<S>& cand) {
  constexpr int L = S::kLanes, kRun = S::kValues / S::kRuns;
  const int l = lane % L;
  float top[S::kRuns];      // the runs' maxima, in descending order
#pragma unroll
  for (int i = 0; i < S::kRuns; ++i) {
    top[i] = -CUDART_INF_F;
#pragma unroll
    for (int r = 0; r < kRun; ++r) top[i] = fmaxf(top[i], c[i * kRun + r]);
  }
  const auto order = [&](int a, int b) {
    const float hi = fmaxf(top[a], top[b]);
    top[b] = fminf(top[a], top[b]);
    top[a] = hi;
  };
  if constexpr (S::kRuns == 2) order(0, 1);
  if constexpr (S::kRuns == 4) {
    order(0, 1);
    order(2, 3);
    order(0, 2);
    order(1, 3);
    order(1, 2);
  }
  float bound = -CUDART_INF_F;
#pragma unroll 4
  for (int k = 0; k < p.K; ++k) {
    bound = tile_max<L>(top[0]);
    const bool drop = top[0] == bound;
#pragma unroll
    for (int i = 0; i < S::kRuns - 1; ++i) top[i] = drop ? top[i + 1] : top[i];
    top[S::kRuns - 1] = drop ? -CUDART_INF_F : top[S::kRuns - 1];
  }
  bound = fmaxf(bound, -3.402823466e38f);
  RegisterSet<S::kValues> mine;
#pragma unroll
  for (int r = 0; r < S::kValues; ++r) mine.add(r, c[r] >= bound);
  const uint32_t before = (1u << l) - 1u;
  int n = 0;
  for (;;) {
    const uint32_t all = __ballot_sync(kFull, mine.bits != 0);
    if (all == 0) break;
    const uint32_t who = tile_bits<L>(all, lane);
    const int at = n + __popc(who & before);
    if (mine.bits != 0 && at < S::kCandidates) cand.expert[at] = S::expert(mine.first(), l);
    mine.drop_first();
    n += __popc(who);
  }
  __syncwarp();
  Chosen<S> out;
#pragma unroll
  for (int i = 0; i < S::kSlots; ++i) {
    out.e[i] = -1;
    out.rank[i] = l + i * L;
    out.l[i] = 0.0f;
  }
  if (__any_sync(kFull, n > S::kCandidates)) {
    float left[S::kValues];      // a copy: c itself then stays in registers
#pragma unroll
    for (int r = 0; r < S::kValues; ++r) left[r] = c[r];
    out.e[0] = choose_in_turn<S>(left, p.K, l);
    if (out.e[0] >= 0) out.l[0] = load_one<S>(p.logits, offset + out.e[0]);
    return out;
  }
  unsigned long long key[S::kSlots];
#pragma unroll
  for (int i = 0; i < S::kSlots; ++i) {
    key[i] = 0;      // past the candidates: after all of them
    if (l + i * L < n) {
      const int e = cand.expert[l + i * L];
      out.e[i] = e;
      out.l[i] = load_one<S>(p.logits, offset + e);
      float score = out.l[i];
      if constexpr (SIG) score = sigmoid(score) + (p.bias != nullptr ? p.bias[e] : 0.0f);
      key[i] = choice_key(score, e);
    }
    cand.key[l + i * L] = key[i];
  }
  __syncwarp();
  int rank[S::kSlots] = {};
  for (int j = 0; j < n; j += 4) {
    const ulonglong2 a = *reinterpret_cast<const ulonglong2*>(cand.key + j);
    const ulonglong2 b = *reinterpret_cast<const ulonglong2*>(cand.key + j + 2);
#pragma unroll
    for (int i = 0; i < S::kSlots; ++i)
      rank[i] += (a.x > key[i] ? 1 : 0) + (a.y > key[i] ? 1 : 0) + (b.x > key[i] ? 1 : 0) +
                 (b.y > key[i] ? 1 : 0);
  }
  __syncwarp();
#pragma unroll
  for (int i = 0; i < S::kSlots; ++i)
    if (l + i * L < n) out.rank[i] = rank[i];
  return out;
}

// ---- a token --------------------------------------------------------------

// One token of each tile, given its logits: choice and gate weights, written
// where `live`.  Leaves the scores in `s` with their total and the row's
// maximum; softmax needs those only for statistics (STATS) or for weights
// that are not renormalised.  Returns the choice, e = -1 for what is not
// taken.
template <class S, bool SIG, bool STATS>
__device__ __forceinline__ Chosen<S> route_token(const RouteParams& p, int t, bool live, int lane,
                                                 float* row, Candidates<S>& cand,
                                                 const float* bias, const float (&x)[S::kValues],
                                                 float (&s)[S::kValues], float* total,
                                                 float* top) {
  constexpr int L = S::kLanes;
  const int l = lane % L;
  const int64_t offset = int64_t(t) * p.ld;
  float divisor = 1.0f;      // of the chosen scores
  float c[S::kValues];
  if constexpr (SIG) {
    *total = scores<S, SIG>(x, s, top);
    if (p.bias != nullptr) {
      read_row<S>(bias, p.E, l, c);
    } else {
#pragma unroll
      for (int r = 0; r < S::kValues; ++r) c[r] = 0.0f;
    }
#pragma unroll
    for (int r = 0; r < S::kValues; ++r)
      c[r] = x[r] > -CUDART_INF_F ? s[r] + c[r] : -CUDART_INF_F;      // NaN too
  } else {
    *top = tile_max<L>(largest(x));
    if (STATS || !p.renorm) {
      *total = soft_scores<S>(x, s, *top);
      if (!p.renorm || *total != *total) divisor = *total;
    } else {
      // NaN where a logit is (a +inf makes its own weight and so all NaN).
      // Not a sum: finite logits' may overflow, and meet -inf.
      float any = x[0];
#pragma unroll
      for (int r = 1; r < S::kValues; ++r) any = max_or_nan(any, x[r]);
      if (tile_bits<L>(__ballot_sync(kFull, any != any), lane) != 0) divisor = CUDART_NAN_F;
    }
#pragma unroll
    for (int r = 0; r < S::kValues; ++r) c[r] = x[r];
  }
  if (p.G > 1) keep_groups<S, SIG>(p, c, row, lane);
  Chosen<S> out = choose<S, SIG>(p, c, offset, lane, cand);
  float w[S::kSlots], sum = 0.0f;
#pragma unroll
  for (int i = 0; i < S::kSlots; ++i) {
    const bool taken = out.e[i] >= 0 && out.rank[i] < p.K;
    w[i] = 0.0f;
    if (taken) w[i] = SIG ? sigmoid(out.l[i]) : soft_score(out.l[i], *top);
    sum += w[i];
    if (!taken) out.e[i] = -1;
  }
  if (p.renorm) {
    sum = tile_sum<L>(sum);
    if (divisor == divisor) divisor = sum;      // the mark of a row with a NaN stays
  }
  const float inv = fast_reciprocal(divisor);
#pragma unroll
  for (int i = 0; i < S::kSlots; ++i) {
    if (live && out.rank[i] < p.K) {
      const int64_t at = int64_t(t) * p.K + out.rank[i];
      p.idx[at] = out.e[i];
      p.w[at] = out.e[i] >= 0 && divisor != 0.0f ? quotient(w[i], divisor, inv) * p.scale : 0.0f;
    }
  }
  return out;
}

// ep_route.  A tile goes through tokens with the next row on its way.
//
// What bounds it: instructions, about 400 a token of 256 experts by softmax
// with top-8 (300 of them with top-1: loads, scores, reductions, addresses)
// and 690 by sigmoid with groups, at 2.5 a cycle and SM with 28 warps.  16384
// tokens, bf16: 8.3 us, where the bytes would take 1.5; 128 tokens 3.1 us
// and one 2.7, of which an empty launch is about 1.7.
//
// CTAs that shall share an SM, for the register limit: 32 or 24 warps with
// the widths of common layers.
template <class S>
constexpr int kRouteShare = S::kValues <= 8 ? 4 : S::kValues <= 16 ? 3 : 1;

template <class S, bool SIG>
__global__ void __launch_bounds__(kRouteThreads, kRouteShare<S>) route_kernel(RouteParams p) {
  extern __shared__ __align__(16) float smem[];
  __shared__ Candidates<S> cands[kRouteWarps * S::kTiles];
  pdl_wait();
  const int lane = threadIdx.x & 31, l = lane % S::kLanes;
  const int tile = threadIdx.x / S::kLanes;      // of the CTA
  constexpr int kCtaTiles = kRouteWarps * S::kTiles;
  const float* bias = smem;      // [E] padded to whole vectors, then the tiles' rows
  float* row = smem + (tile + 1) * padded_row(p.E);
  if (SIG && p.bias != nullptr) {
    for (int e = threadIdx.x; e < p.E; e += kRouteThreads) smem[e] = clean_bias(p.bias[e]);
    __syncthreads();
  }
  const int stride = gridDim.x * kCtaTiles;
  const auto load = [&](int t, float (&x)[S::kValues]) {
    const bool have = t < p.T && (p.mask == nullptr || p.mask[t] != 0);
    load_row<S>(p.logits, int64_t(t) * p.ld, p.E, l, have, x);
  };
  float x[S::kValues], s[S::kValues], total, top;
  // a warp's tiles go through the same number of tokens
  int t = blockIdx.x * kCtaTiles + tile, first = t - tile % S::kTiles;
  if constexpr (S::kAhead) load(t, x);
  for (; first < p.T; t += stride, first += stride) {
    float next[S::kValues];
    if constexpr (S::kAhead)
      load(t + stride, next);
    else
      load(t, x);
    route_token<S, SIG, false>(p, t, t < p.T, lane, row, cands[tile], bias, x, s, &total, &top);
    if constexpr (S::kAhead) {
#pragma unroll
      for (int r = 0; r < S::kValues; ++r) x[r] = next[r];
    }
  }
}

// First sequence whose end lies past token t (the last one otherwise), by a
// whole warp for one t: 32 ends at a time, so that two rounds of loads serve
// a thousand sequences.
__device__ __forceinline__ int sequence_of(const int32_t* seq_start, int B, int t, int lane) {
  int lo = 0, n = B - 1;      // the answer is among lo .. lo + n
  while (n > 0) {
    const int step = n / 32 + 1, i = lane * step;
    const bool past = i + step - 1 >= n || seq_start[lo + i + step] > t;
    const int skip = __ffs(__ballot_sync(kFull, past)) - 1;      // the last lane always answers
    lo += skip * step;
    n = min(step - 1, n - skip * step);
  }
  return lo;
}

// ---- balance --------------------------------------------------------------

template <class S>
constexpr int kBalanceThreads = S::kValues <= 16 ? 512 : 256;

// ep_route_balance, first kernel: what bounds it is what bounds ep_route, and
// the flush of a CTA's sums.  16384 tokens by 256 experts, sigmoid, groups, 4
// sequences: 23.0 us for both kernels (745 instructions a token), the bytes
// 2.8; 4096 by softmax 10.5; 8191 by 64 in 37 ragged sequences 10.6.  One CTA
// of 512 threads an SM, with the registers it likes.  Measured with one
// rounding an exponential less, when this took 22.3, 10.1 and 10.3 us: two at
// 64 registers 23.4, 10.4 and 10.8; 768 threads 21.4, 10.7 and 11.6; two of
// 256 threads 23.0, 11.1 and 10.9.
// About 4 us are the second kernel and its launch; starting it early
// (launch_dependents) measured no better.
//
// A CTA owns the tokens [c * R, (c + 1) * R)
// and walks the sequences they belong to; the sums of (CTA c, sequence b) go
// to partial row c + b, which no other pair uses (both only grow along the
// tokens).
template <class S, bool SIG>
__global__ void __launch_bounds__(kBalanceThreads<S>, 1)
balance_kernel(RouteParams p) {
  constexpr int kThreads = kBalanceThreads<S>, kWarps = kThreads / 32;
  constexpr int kCtaTiles = kThreads / S::kLanes;
  extern __shared__ __align__(16) float smem[];
  const int width = padded_row(p.E);
  float* rows = smem;                                           // [kCtaTiles][width]
  float* bias = smem + kCtaTiles * width;                       // [width]
  int* counts = reinterpret_cast<int*>(bias + width);           // [width]
  __shared__ Candidates<S> cands[kCtaTiles];
  __shared__ float warp_z[kWarps];
  __shared__ int warp_n[kWarps];
  pdl_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, l = lane % S::kLanes;
  const int tile = threadIdx.x / S::kLanes;
  float* row = rows + tile * width;
  if (blockIdx.x == 0 && threadIdx.x == 0) *p.done = 0;
  for (int e = threadIdx.x; e < p.E; e += kThreads) counts[e] = 0;
  if (SIG && p.bias != nullptr)
    for (int e = threadIdx.x; e < p.E; e += kThreads) bias[e] = clean_bias(p.bias[e]);
  __syncthreads();
  const int first = blockIdx.x * p.tokens_per_cta;
  const int last = min(p.T, first + p.tokens_per_cta);
  int b = p.B > 1 ? sequence_of(p.seq_start, p.B, first, lane) : 0;
  float sum[S::kValues], z = 0.0f;
  int n = 0;
#pragma unroll
  for (int r = 0; r < S::kValues; ++r) sum[r] = 0.0f;
  float x[S::kValues], s[S::kValues], total, top;
  bool have, next_have = false;
  const auto load = [&](int u, bool& have, float (&x)[S::kValues]) {
    have = u < last && (p.mask == nullptr || p.mask[u] != 0);
    load_row<S>(p.logits, int64_t(u) * p.ld, p.E, l, have, x);
  };
  if constexpr (S::kAhead) load(first + tile, have, x);
  for (int t = first; t < last; t += kCtaTiles) {
    const int u = t + tile;
    float next[S::kValues];
    if constexpr (S::kAhead)
      load(u + kCtaTiles, next_have, next);
    else
      load(u, have, x);
    const Chosen<S> mine = route_token<S, SIG, true>(p, u, u < last, lane, row, cands[tile], bias,
                                                     x, s, &total, &top);
    // all tiles' tokens are routed; the sequences they lie in, one by one
    const int block_end = min(last, t + kCtaTiles);
    for (int from = t; from < block_end;) {
      while (b < p.B - 1 && p.seq_start[b + 1] <= from) ++b;
      const int end = b < p.B - 1 ? min(last, p.seq_start[b + 1]) : last;
      if (have && u >= from && u < end) {
#pragma unroll
        for (int i = 0; i < S::kSlots; ++i)
          if (mine.e[i] >= 0) atomicAdd(&counts[mine.e[i]], 1);
        // total is 0 only where no expert is in service: the token adds nothing
        const float inv = total == 0.0f ? 0.0f : fast_reciprocal(total);
#pragma unroll
        for (int r = 0; r < S::kValues; ++r) sum[r] = fmaf(s[r], inv, sum[r]);
        if (l == 0) {
          ++n;
          if (!SIG && total != 0.0f) {
            const float lse = top + __logf(total);
            z += lse * lse;
          }
        }
      }
      from = end;
      if (end > block_end) continue;      // the sequence goes on in the next tokens
      // the tiles of a warp, then the warps in order.  A warp's sums go to the
      // row of its first tile: other rows may still hold the choice scores of
      // groups of warps that have not come here yet.
      __syncwarp();
#pragma unroll
      for (int d = 16; d >= S::kLanes; d >>= 1) {
#pragma unroll
        for (int r = 0; r < S::kValues; ++r) sum[r] += __shfl_xor_sync(kFull, sum[r], d);
      }
      z = tile_sum<32>(z);
      n = __reduce_add_sync(kFull, n);
#pragma unroll
      for (int r = 0; r < S::kValues; ++r) {
        const int e = S::expert(r, l);
        if (lane < S::kLanes && e < p.E) rows[warp * S::kTiles * width + e] = sum[r];
        sum[r] = 0.0f;
      }
      if (lane == 0) {
        warp_z[warp] = z;
        warp_n[warp] = n;
      }
      z = 0.0f;
      n = 0;
      __syncthreads();
      const int64_t part = int64_t(blockIdx.x) + b;
      for (int e = threadIdx.x; e < p.E; e += kThreads) {
        float acc = 0.0f;
#pragma unroll
        for (int v = 0; v < kWarps; ++v) acc += rows[v * S::kTiles * width + e];
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
    }
    if constexpr (S::kAhead) {
#pragma unroll
      for (int r = 0; r < S::kValues; ++r) x[r] = next[r];
      have = next_have;
    }
  }
}

constexpr int kSumThreads = 256;     // of a CTA of the second kernel
// Experts of such a CTA: 8 (a 32-byte sector of a row; 32 partial rows at a
// time) where sequences have many partial rows, 64 (four at a time) where
// they have few, so that many sequences make fewer CTAs: 4096 tokens of 64
// sequences by 256 experts 17.7 and 11.8 us.
constexpr int kSumExperts = 8, kSumExpertsMany = 64;

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

// Second kernel: CTA (b, i) adds up the partial rows of sequence b for the
// experts from EX i on, kSumThreads / EX rows at a time, in a fixed order;
// the first warp of the CTA that finishes last forms the losses from what all
// have written.  Latency alone: a handful of dependent loads, sums and one
// atomic.
template <int EX>
__global__ void __launch_bounds__(kSumThreads) balance_sum_kernel(BalanceParams p) {
  constexpr int kWarps = kSumThreads / 32, kRows = kSumThreads / EX;
  constexpr int kSums = EX < 32 ? kWarps : kRows;      // of an expert, through shared memory
  __shared__ float probs[kSums][EX], zs[kWarps];
  __shared__ int counts[kSums][EX], ns[kWarps];
  pdl_wait();
  const int b = blockIdx.x, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int part = threadIdx.x / EX, first = blockIdx.y * EX, e = first + threadIdx.x % EX;
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
    for (int c = part; c < c1 - c0; c += kRows) {
      prob += fp[int64_t(c) * p.E];
      count += ip[int64_t(c) * p.E];
    }
  }
  for (int c = c0 + threadIdx.x; c < c1; c += kSumThreads) {
    n += p.part_tokens[c + b];
    z += p.part_z[c + b];
  }
  // the rows of a warp, then the warps
#pragma unroll
  for (int d = EX; d < 32; d <<= 1) {
    prob += __shfl_xor_sync(kFull, prob, d);
    count += __shfl_xor_sync(kFull, count, d);
  }
  z = tile_sum<32>(z);
  n = __reduce_add_sync(kFull, n);
  if constexpr (EX < 32) {
    if (lane < EX) {
      probs[warp][lane] = prob;
      counts[warp][lane] = count;
    }
  } else {
    probs[part][threadIdx.x % EX] = prob;
    counts[part][threadIdx.x % EX] = count;
  }
  if (lane == 0) {
    zs[warp] = z;
    ns[warp] = n;
  }
  __syncthreads();
  if (warp != 0) return;
  z = tile_sum<32>(lane < kWarps ? zs[lane] : 0.0f);
  n = __reduce_add_sync(kFull, lane < kWarps ? ns[lane] : 0);
  const float inv_n = n > 0 ? 1.0f / float(n) : 0.0f;
  float dot = 0.0f;
#pragma unroll
  for (int i = lane; i < EX; i += 32) {
    prob = 0.0f;
    count = 0;
#pragma unroll
    for (int w = 0; w < kSums; ++w) {
      prob += probs[w][i];
      count += counts[w][i];
    }
    prob *= inv_n;
    if (first + i < p.E) {
      p.expert_prob[int64_t(b) * p.E + first + i] = prob;
      p.expert_count[int64_t(b) * p.E + first + i] = count;
    }
    dot += float(count) * inv_n * prob;
  }
  dot = tile_sum<32>(dot);
  unsigned before = 0;
  if (lane == 0) {
    p.dots[int64_t(b) * gridDim.y + blockIdx.y] = dot;
    if (blockIdx.y == 0) {
      p.seq_tokens[b] = n;
      p.seq_z[b] = z;
    }
    __threadfence();
    before = atomicAdd(p.done, 1u);
  }
  before = __shfl_sync(kFull, before, 0);
  if (before != gridDim.x * gridDim.y - 1) return;
  __threadfence();
  // every term is there: 32 at a time, in a fixed order
  float loss = 0.0f;
  int full = 0;
  n = 0;
  z = 0.0f;
  const int64_t dots = int64_t(p.B) * gridDim.y;
  for (int64_t i = lane; i < dots; i += 32 * 16) {
    float v[16];      // all on their way at once
#pragma unroll
    for (int j = 0; j < 16; ++j) v[j] = i + 32 * j < dots ? __ldcg(p.dots + i + 32 * j) : 0.0f;
#pragma unroll
    for (int j = 0; j < 16; ++j) loss += v[j];
  }
#pragma unroll 4
  for (int i = lane; i < p.B; i += 32) {
    const int m = __ldcg(p.seq_tokens + i);
    n += m;
    full += m > 0 ? 1 : 0;
    z += __ldcg(p.seq_z + i);
  }
  loss = tile_sum<32>(loss);
  z = tile_sum<32>(z);
  n = __reduce_add_sync(kFull, n);
  full = __reduce_add_sync(kFull, full);
  if (lane == 0) {
    p.seq_tokens[p.B] = n;
    p.seq_tokens[p.B + 1] = full;
    p.loss[0] = full > 0 ? loss * (float(p.E) / float(p.K)) / float(full) : 0.0f;
    p.loss[1] = n > 0 ? z / float(n) : 0.0f;
  }
}

// ---- backward -------------------------------------------------------------

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

// dL/dlogits of a token, all of it recomputed from its logits:
//   dq_e = g0 c_be E / (K n_b^2 B')       balance loss by the normalised score
//   ds_k = scale dw_k, or scale / S (dw_k - sum_j dw_j s_j / S)   gate weight
//   softmax:  g = dq + ds,  dl = s (g - sum s g + g1 2 lse / N)
//   sigmoid:  u = (dq - sum q dq) / sum s + ds,  dl = u s (1 - s)
// The next token's logits, choice and gate gradient are loaded ahead.
//
// What bounds it: instructions again, about 460 a token of 256 experts; 16384
// tokens, bf16, sigmoid: 9.4 us (bytes: 2.8), 4096, fp32, softmax: 4.0 (1.3).
template <class S, bool SIG>
__global__ void __launch_bounds__(kRouteThreads, kRouteShare<S>)
route_backward_kernel(RouteBackwardParams p) {
  extern __shared__ __align__(16) float smem[];
  pdl_wait();
  constexpr int L = S::kLanes, kCtaTiles = kRouteThreads / L;
  const int lane = threadIdx.x & 31, l = lane % L, tile = threadIdx.x / L;
  float* row = smem + tile * padded_row(p.E);      // ds of the chosen, else 0
  for (int e = l; e < p.E; e += L) row[e] = 0.0f;
  __syncwarp();
  const int first = blockIdx.x * p.tokens_per_cta;
  const int last = min(p.T, first + p.tokens_per_cta);
  float dq[S::kValues];
#pragma unroll
  for (int r = 0; r < S::kValues; ++r) dq[r] = 0.0f;
  float dlse = 0.0f;
  const bool losses = p.expert_count != nullptr;
  if (losses && !SIG) {
    const int n = p.seq_tokens[p.B];
    dlse = n > 0 ? p.grad_loss[1] * 2.0f / float(n) : 0.0f;
  }
  struct Token {
    float x[S::kValues], dw;
    int choice;      // of lane k of the tile: its k-th, or -1
    bool have;
  };
  const auto load = [&](int t, Token& k) {
    k.have = t < last && (p.mask == nullptr || p.mask[t] != 0);
    load_row<S>(p.logits, int64_t(t) * p.ld, p.E, l, k.have, k.x);
    k.choice = -1;
    k.dw = 0.0f;
    if (p.grad_w != nullptr && k.have && l < p.K) {
      const int64_t e = p.idx[int64_t(t) * p.K + l];
      k.choice = e >= 0 && e < p.E ? int(e) : -1;
      k.dw = p.grad_w[int64_t(t) * p.K + l];
    }
  };
  Token now, next;
  int t = first + tile, warp_first = t - tile % S::kTiles;
  int b = losses && p.B > 1 ? sequence_of(p.seq_start, p.B, warp_first, lane) : 0, was = -1;
  if constexpr (S::kAhead) load(t, now);
  for (; warp_first < last; t += kCtaTiles, warp_first += kCtaTiles) {
    if constexpr (S::kAhead)
      load(t + kCtaTiles, next);
    else
      load(t, now);
    if (losses && t < last) {
      while (b < p.B - 1 && p.seq_start[b + 1] <= t) ++b;
      if (b != was) {
        was = b;
        const int n = p.seq_tokens[b], full = p.seq_tokens[p.B + 1];
        const float each = n > 0 && full > 0 ? p.grad_loss[0] * (float(p.E) / float(p.K)) /
                                                   (float(n) * float(n) * float(full))
                                             : 0.0f;
#pragma unroll
        for (int r = 0; r < S::kValues; ++r) {
          const int e = S::expert(r, l);
          dq[r] = e < p.E ? each * float(p.expert_count[int64_t(b) * p.E + e]) : 0.0f;
        }
      }
    }
    __syncwarp();
    const int mine = now.choice;
    const float logit =
        mine >= 0 ? load_one<S>(p.logits, int64_t(t) * p.ld + mine) : 0.0f;
    float s[S::kValues], g[S::kValues], top;
    const float total = scores<S, SIG>(now.x, s, &top);
    const float inv = total == 0.0f ? 0.0f : fast_reciprocal(total);
    if (p.grad_w != nullptr) {
      float ds = 0.0f, sk = 0.0f;
      if (mine >= 0) {
        sk = SIG ? sigmoid(logit) : soft_score(logit, top) * inv;
        ds = now.dw * p.scale;
      }
      if (p.renorm) {
        const float sum = tile_sum<L>(sk);
        const float is = sum == 0.0f ? 0.0f : fast_reciprocal(sum);
        // a single choice weighs exactly 1, and passes nothing on
        const float mean = tile_sum<L>(ds * quotient(sk, sum, is));
        ds = (ds - mean) * is;
      }
      if (mine >= 0) row[mine] = ds;
      __syncwarp();
      read_row<S>(row, p.E, l, g);
      __syncwarp();
      if (mine >= 0) row[mine] = 0.0f;
    } else {
#pragma unroll
      for (int r = 0; r < S::kValues; ++r) g[r] = 0.0f;
    }
    float dot = 0.0f;
#pragma unroll
    for (int r = 0; r < S::kValues; ++r) {
      if constexpr (SIG) {
        dot = fmaf(s[r], dq[r], dot);
      } else {
        s[r] *= inv;
        g[r] += dq[r];
        dot = fmaf(s[r], g[r], dot);
      }
    }
    dot = tile_sum<L>(dot);
    if constexpr (SIG) {
      dot *= inv;
#pragma unroll
      for (int r = 0; r < S::kValues; ++r)
        g[r] = fmaf(dq[r] - dot, inv, g[r]) * (s[r] * (1.0f - s[r]));
    } else {
      const float z = total != 0.0f ? dlse * (top + __logf(total)) : 0.0f;
#pragma unroll
      for (int r = 0; r < S::kValues; ++r) g[r] = s[r] * (g[r] - (dot - z));
    }
    // a padding token's row was taken as -inf: all its scores are 0, but not
    // their products with a coefficient that is not finite
    if (!now.have) {
#pragma unroll
      for (int r = 0; r < S::kValues; ++r) g[r] = 0.0f;
    }
    if (t < last) store_row<S>(p.grad, int64_t(t) * p.ld_grad, p.E, l, g);
    if constexpr (S::kAhead) now = next;
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
constexpr int kMaxTokens = 1 << 30;      // token numbers and strides stay under 2^31

// CTAs of a per-token kernel over `tokens` tokens, `tiles` of them at a time
// in a CTA: at most `share` CTAs an SM, each tile with a token at least.
int route_ctas(int tokens, int tiles, int share) {
  const int want = (tokens + tiles - 1) / tiles;
  const int most = device_info().sm_count * share;
  return want < most ? want : most;
}

// Tokens a CTA when `tokens` are dealt to at most `ctas` CTAs in runs.
int run_length(int tokens, int ctas) { return ctas > 0 ? (tokens + ctas - 1) / ctas : 1; }

// Calls f.template operator()<Shape, SIG>() with the tile that suits E, K, G
// and the number of tokens T.  Few tokens (a warp each at most) take a whole
// warp, which is done soonest; many take narrow tiles where these measured
// faster: 8 lanes up to 64 experts (ep_route of 8192 tokens by 64: 3.0 us, by
// whole warps 4.6), 16 up to 128 (4.2, 5.3), but not 16 at 256 (11.1, 8.0 at
// 16384 tokens: the same instructions a token less a third, yet half the
// tokens in flight and longer chains of shuffles).  A tile needs a lane for
// each group and rank, and candidates for K and a few more.  Rows whose
// vectors of four logits are aligned are loaded as those.
template <bool BF16, typename F>
cudaError_t with_shape(int T, int E, int K, int G, int64_t ld, bool sig, F&& f) {
  const bool vec = E % 4 == 0 && ld % 4 == 0;
  const bool many = T > device_info().sm_count * 32;
#define EP_SHAPE(L, N, V)                                                 \
  return sig ? f.template operator()<Shape<L, N, V, BF16>, true>()        \
             : f.template operator()<Shape<L, N, V, BF16>, false>()
  if (many && vec && E <= 64 && K <= 8 && G <= 8) {
    if (E <= 32) EP_SHAPE(8, 4, 4);
    EP_SHAPE(8, 8, 4);
  }
  if (many && vec && E <= 128 && K <= 10 && G <= 16) EP_SHAPE(16, 8, 4);
  if (E <= 32) EP_SHAPE(32, 1, 1);
  if (E <= 64) EP_SHAPE(32, 2, 1);
  if (E <= 128) EP_SHAPE(32, 4, 1);
  if (E <= 256) {
    if (vec) EP_SHAPE(32, 8, 4);
    EP_SHAPE(32, 8, 1);
  }
  if (E <= 512) {
    if (vec) EP_SHAPE(32, 16, 4);
    EP_SHAPE(32, 16, 1);
  }
  EP_SHAPE(32, 64, 1);
#undef EP_SHAPE
}

template <typename F>
cudaError_t with_shape(const ep_router_config* cfg, int T, int G, int64_t ld, F&& f) {
  const bool sig = cfg->score == EP_SCORE_SIGMOID;
  return cfg->logits_bf16 ? with_shape<true>(T, cfg->num_experts, cfg->num_topk, G, ld, sig, f)
                          : with_shape<false>(T, cfg->num_experts, cfg->num_topk, G, ld, sig, f);
}

// Raises a kernel's dynamic shared-memory limit where `bytes` needs it (48 KiB
// with the static arrays, which are under 13, need no leave): once per kernel
// and device, to what the most experts need, because host threads that launch
// the same kernel with other numbers of experts share the limit.
constexpr size_t kMostSmem = 10 * 2048 * sizeof(float);      // the balance kernel's rows

template <auto kKernel, class S, int kRows>
cudaError_t allow_smem(size_t bytes) {
  static_assert(kRows * S::kLanes * S::kValues * sizeof(float) <= kMostSmem);
  if (bytes <= 32 * 1024) return cudaSuccess;
  static std::atomic<uint64_t> raised{0};      // a bit a device
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 64 && (raised.load(std::memory_order_acquire) >> dev & 1)) return cudaSuccess;
  e = cudaFuncSetAttribute(kKernel, cudaFuncAttributeMaxDynamicSharedMemorySize, int(kMostSmem));
  if (e == cudaSuccess && dev < 64) raised.fetch_or(uint64_t(1) << dev, std::memory_order_release);
  return e;
}

struct LaunchRoute {
  RouteParams p;
  cudaStream_t stream;
  template <class S, bool SIG>
  cudaError_t operator()() const {
    constexpr int kCtaTiles = kRouteThreads / S::kLanes;
    const size_t rows = p.G > 1 ? kCtaTiles + 1 : SIG ? 1 : 0;
    const size_t smem = sizeof(float) * rows * padded_row(p.E);
    constexpr auto* kernel = route_kernel<S, SIG>;
    const cudaError_t e = allow_smem<kernel, S, kCtaTiles + 1>(smem);
    if (e != cudaSuccess) return e;
    return launch_pdl(kernel, dim3(route_ctas(p.T, kCtaTiles, kRouteShare<S>)),
                      dim3(kRouteThreads), smem, stream, p);
  }
};

// CTAs of the second kernel along the experts, at most.
int sum_ctas(int E) { return (E + kSumExperts - 1) / kSumExperts; }

struct LaunchBalance {
  RouteParams p;
  BalanceParams q;      // of the second kernel
  cudaStream_t stream;
  template <class S, bool SIG>
  cudaError_t operator()() {
    constexpr int kThreads = kBalanceThreads<S>, kCtaTiles = kThreads / S::kLanes;
    const int ctas = route_ctas(p.T, kCtaTiles, 1);
    p.tokens_per_cta = q.tokens_per_cta = run_length(p.T, ctas);
    // no tokens: one CTA still clears `done`
    const int used = p.T > 0 ? (p.T + p.tokens_per_cta - 1) / p.tokens_per_cta : 1;
    const size_t smem = sizeof(float) * (kCtaTiles + 2) * padded_row(p.E);
    constexpr auto* kernel = balance_kernel<S, SIG>;
    cudaError_t e = allow_smem<kernel, S, kCtaTiles + 2>(smem);
    if (e != cudaSuccess) return e;
    e = launch_pdl(kernel, dim3(used), dim3(kThreads), smem, stream, p);
    if (e != cudaSuccess) return e;
    if (used < 16 * int64_t(p.B))
      return launch_pdl(balance_sum_kernel<kSumExpertsMany>,
                        dim3(p.B, (p.E + kSumExpertsMany - 1) / kSumExpertsMany),
                        dim3(kSumThreads), 0, stream, q);
    return launch_pdl(balance_sum_kernel<kSumExperts>, dim3(p.B, sum_ctas(p.E)),
                      dim3(kSumThreads), 0, stream, q);
  }
};

struct LaunchBackward {
  RouteBackwardParams p;
  cudaStream_t stream;
  template <class S, bool SIG>
  cudaError_t operator()() {
    constexpr int kCtaTiles = kRouteThreads / S::kLanes;
    p.tokens_per_cta = run_length(p.T, route_ctas(p.T, kCtaTiles, kRouteShare<S>));
    const size_t smem = sizeof(float) * kCtaTiles * padded_row(p.E);
    constexpr auto* kernel = route_backward_kernel<S, SIG>;
    const cudaError_t e = allow_smem<kernel, S, kCtaTiles + 1>(smem);
    if (e != cudaSuccess) return e;
    return launch_pdl(kernel, dim3((p.T + p.tokens_per_cta - 1) / p.tokens_per_cta),
                      dim3(kRouteThreads), smem, stream, p);
  }
};

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

// The first kernel has at most one CTA an SM, whatever T.
BalanceWorkspace carve(void* base, int E, int B) {
  const int64_t rows = int64_t(device_info().sm_count) + B;
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
  if (!router_ok(cfg) || T < 0 || T > kMaxTokens || ld < cfg->num_experts) return false;
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
  l.stream = static_cast<cudaStream_t>(stream);
  return status(with_shape(cfg, num_tokens, l.p.G, ld_logits, l));
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
  return status(with_shape(cfg, num_tokens, l.p.G, ld_logits, l));
}

int32_t ep_route_backward(const ep_router_config* cfg, int32_t num_tokens, const void* d_logits,
                          int64_t ld_logits, const uint8_t* d_token_mask,
                          const int64_t* d_topk_idx, const float* d_grad_w, int32_t num_seqs,
                          const int32_t* d_seq_start, const int32_t* d_expert_count,
                          const int32_t* d_seq_tokens, const float* d_grad_loss,
                          void* d_grad_logits, int64_t ld_grad, void* stream) {
  if (!router_ok(cfg) || num_tokens < 0 || num_tokens > kMaxTokens) return EP_ERR_INVALID_ARG;
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
  l.stream = static_cast<cudaStream_t>(stream);
  // both rows have to allow vectors for either to use them
  const int64_t ld = ld_logits % 4 == 0 ? ld_grad : ld_logits;
  return status(with_shape(cfg, num_tokens, 1, ld, l));
}

}  // extern "C"

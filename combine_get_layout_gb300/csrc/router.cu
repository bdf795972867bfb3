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
  bool renorm;
  float scale;
  int64_t* idx;              // [T, K]
  float* w;                  // [T, K]
  // balance
  const int32_t* seq_start;  // [B + 1] or null (B = 1)
  int B;
  int tokens_per_cta, ctas;
  float* part_prob;          // [ctas + B, E]
  int32_t* part_count;       // [ctas + B, E]
  int32_t* part_tokens;      // [ctas + B]
  float* part_z;             // [ctas + B]
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

// Order-preserving 32-bit key of a float; -0 and +0 share one key.
__device__ __forceinline__ uint32_t order_key(float f) {
  const uint32_t u = __float_as_uint(f + 0.0f);
  return u ^ (uint32_t(int32_t(u) >> 31) | 0x80000000u);
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int d = 16; d; d >>= 1) v += __shfl_xor_sync(kFull, v, d);
  return v;
}

__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
  for (int d = 16; d; d >>= 1) v = fmaxf(v, __shfl_xor_sync(kFull, v, d));
  return v;
}

__device__ __forceinline__ float sigmoid(float x) { return 1.0f / (1.0f + expf(-x)); }

// Scores of a token: s = exp(x - max) / sum (softmax) or sigmoid(x).  Leaves
// the scores in `s`; returns their total over the experts (softmax: the sum
// of exponentials) and the row's maximum.  A row with no finite maximum
// below has all-zero scores.
template <int VPL, bool SIG>
__device__ __forceinline__ float scores(const float (&x)[VPL], float (&s)[VPL], float* top) {
  float total = 0.0f;
  if constexpr (SIG) {
#pragma unroll
    for (int r = 0; r < VPL; ++r) {
      s[r] = x[r] == -CUDART_INF_F ? 0.0f : sigmoid(x[r]);
      total += s[r];
    }
    *top = 0.0f;
    return warp_sum(total);
  } else {
    float m = x[0];
#pragma unroll
    for (int r = 1; r < VPL; ++r) m = fmaxf(m, x[r]);
    m = warp_max(m);
    *top = m;
#pragma unroll
    for (int r = 0; r < VPL; ++r) {
      // an expert out of service, and a row with none in service, score 0
      s[r] = x[r] == -CUDART_INF_F ? 0.0f : expf(x[r] - m);
      total += s[r];
    }
    return warp_sum(total);
  }
}

// Clears the choice scores of every group but the `kept` best.  `row` is
// this warp's shared scratch of E floats.
template <int VPL, int V, bool SIG>
__device__ void keep_groups(float (&c)[VPL], float* row, int E, int G, int kept, int lane) {
#pragma unroll
  for (int r = 0; r < VPL; ++r) {
    const int e = element_of<V>(r, lane);
    if (e < E) row[e] = c[r];
  }
  __syncwarp();
  const int per = E / G;
  float best = -CUDART_INF_F, second = -CUDART_INF_F;
  if (lane < G) {
    for (int i = 0; i < per; ++i) {
      const float v = row[lane * per + i];
      second = fmaxf(second, fminf(best, v));
      best = fmaxf(best, v);
    }
  }
  // sigmoid: the two best scores' sum, an expert out of service adding none
  float mine = best;
  if (SIG && second > -CUDART_INF_F) mine += second;
  const uint32_t key = lane < G ? order_key(mine) : 0u;
  int beaten_by = 0;
  for (int g = 0; g < G; ++g) {
    const uint32_t other = __shfl_sync(kFull, key, g);
    beaten_by += (other > key || (other == key && g < lane)) ? 1 : 0;
  }
  const uint32_t keep = __ballot_sync(kFull, lane < G ? beaten_by < kept : false);
#pragma unroll
  for (int r = 0; r < VPL; ++r) {
    const int e = element_of<V>(r, lane);
    if (e < E && !((keep >> (e / per)) & 1u)) c[r] = -CUDART_INF_F;
  }
  __syncwarp();
}

// The K largest of a warp's choice scores, in descending order, equal ones
// by ascending index: lane k returns the k-th index, or -1 when fewer than
// k + 1 experts can be chosen.
template <int VPL, int V>
__device__ __forceinline__ int choose(float (&c)[VPL], int K, int lane) {
  int mine = -1;
  for (int k = 0; k < K; ++k) {
    float best = c[0];
    int at = element_of<V>(0, lane);
#pragma unroll
    for (int r = 1; r < VPL; ++r) {
      if (c[r] > best) {
        best = c[r];
        at = element_of<V>(r, lane);
      }
    }
    const uint32_t key = order_key(best);
    const uint32_t top = __reduce_max_sync(kFull, key);
    if (top == order_key(-CUDART_INF_F)) break;
    const int win = int(__reduce_min_sync(kFull, key == top ? uint32_t(at) : 0xffffffffu));
#pragma unroll
    for (int r = 0; r < VPL; ++r)
      if (element_of<V>(r, lane) == win) c[r] = -CUDART_INF_F;
    if (lane == k) mine = win;
  }
  return mine;
}

// One token: choice and gate weights, and the normalised scores in `s`.
// Returns the expert of lane k < K.
template <int VPL, int V, bool BF16, bool SIG>
__device__ __forceinline__ int route_token(const RouteParams& p, int t, int lane, float* row,
                                           float (&s)[VPL], float* total, float* top) {
  float x[VPL];
  load_row<VPL, V, BF16>(p.logits, int64_t(t) * p.ld, p.E, lane, x);
  *total = scores<VPL, SIG>(x, s, top);
  float c[VPL];
#pragma unroll
  for (int r = 0; r < VPL; ++r) {
    c[r] = x[r];
    if (SIG) {
      const int e = element_of<V>(r, lane);
      const float b = p.bias != nullptr && e < p.E ? p.bias[e] : 0.0f;
      c[r] = x[r] == -CUDART_INF_F ? -CUDART_INF_F : s[r] + b;
    }
    if (c[r] != c[r]) c[r] = -CUDART_INF_F;   // a NaN is not chosen
  }
  if (p.G > 1) keep_groups<VPL, V, SIG>(c, row, p.E, p.G, p.kept, lane);
  const int mine = choose<VPL, V>(c, p.K, lane);
  float w = 0.0f;
  if (mine >= 0) {
    const float l = load_one<BF16>(p.logits, int64_t(t) * p.ld + mine);
    w = SIG ? sigmoid(l) : expf(l - *top) / *total;
  }
  if (p.renorm) {
    const float sum = warp_sum(w);
    w = sum == 0.0f ? 0.0f : w / sum;
  }
  if (lane < p.K) {
    p.idx[int64_t(t) * p.K + lane] = mine;
    p.w[int64_t(t) * p.K + lane] = w * p.scale;
  }
  return mine;
}

__device__ __forceinline__ void route_masked(const RouteParams& p, int t, int lane) {
  if (lane < p.K) {
    p.idx[int64_t(t) * p.K + lane] = -1;
    p.w[int64_t(t) * p.K + lane] = 0.0f;
  }
}

template <int VPL, int V, bool BF16, bool SIG>
__global__ void __launch_bounds__(kRouteThreads) route_kernel(RouteParams p) {
  extern __shared__ float smem[];
  pdl_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  float* row = smem + warp * p.E;
  float s[VPL], total, top;
  for (int t = blockIdx.x * kRouteWarps + warp; t < p.T; t += gridDim.x * kRouteWarps) {
    if (p.mask != nullptr && p.mask[t] == 0) {
      route_masked(p, t, lane);
      continue;
    }
    route_token<VPL, V, BF16, SIG>(p, t, lane, row, s, &total, &top);
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
template <int VPL, int V, bool BF16, bool SIG>
__global__ void __launch_bounds__(kRouteThreads) balance_kernel(RouteParams p) {
  extern __shared__ float smem[];
  float* probs = smem;                                         // [kRouteWarps][E]
  int* counts = reinterpret_cast<int*>(smem + kRouteWarps * p.E);   // [E]
  __shared__ float warp_z[kRouteWarps];
  __shared__ int warp_n[kRouteWarps];
  pdl_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  float* row = probs + warp * p.E;
  for (int e = threadIdx.x; e < p.E; e += kRouteThreads) counts[e] = 0;
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
    for (int u = t + warp; u < end; u += kRouteWarps) {
      if (p.mask != nullptr && p.mask[u] == 0) {
        route_masked(p, u, lane);
        continue;
      }
      float s[VPL], total, top;
      const int mine = route_token<VPL, V, BF16, SIG>(p, u, lane, row, s, &total, &top);
      if (mine >= 0) atomicAdd(&counts[mine], 1);
      // total is 0 only where no expert is in service: the token adds nothing
      const float inv = total == 0.0f ? 0.0f : 1.0f / total;
#pragma unroll
      for (int r = 0; r < VPL; ++r) sum[r] += s[r] * inv;
      ++n;
      if (!SIG && total != 0.0f) {
        const float lse = top + logf(total);
        z += lse * lse;
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
    for (int e = threadIdx.x; e < p.E; e += kRouteThreads) {
      float acc = 0.0f;
#pragma unroll
      for (int v = 0; v < kRouteWarps; ++v) acc += probs[v * p.E + e];
      p.part_prob[part * p.E + e] = acc;
      p.part_count[part * p.E + e] = counts[e];
      counts[e] = 0;
    }
    if (threadIdx.x == 0) {
      float zs = 0.0f;
      int ns = 0;
      for (int v = 0; v < kRouteWarps; ++v) {
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

struct BalanceParams {
  const int32_t* seq_start;
  int T, E, K, B, tokens_per_cta, ctas;
  const float* part_prob;
  const int32_t* part_count;
  const int32_t* part_tokens;
  const float* part_z;
  int32_t* expert_count;   // [B, E]
  float* expert_prob;      // [B, E]
  int32_t* seq_tokens;     // [B + 2]
  float* seq_loss;         // [B] workspace: sum over e of count * prob
  float* seq_z;            // [B] workspace
  float* loss;             // [2]
};

// Sum over a block of kRouteThreads, in a fixed order, in every thread.
__device__ float block_sum(float v, float* scratch) {
  v = warp_sum(v);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) scratch[threadIdx.x >> 5] = v;
  __syncthreads();
  float s = 0.0f;
  for (int i = 0; i < kRouteWarps; ++i) s += scratch[i];
  return s;
}

// Second kernel: one CTA a sequence adds up its partial rows in order.
__global__ void __launch_bounds__(kRouteThreads) balance_sum_kernel(BalanceParams p) {
  __shared__ float scratch[kRouteWarps];
  pdl_wait();
  const int b = blockIdx.x;
  const int lo = b == 0 ? 0 : min(max(p.seq_start[b], 0), p.T);
  const int hi = b == p.B - 1 ? p.T : min(max(p.seq_start[b + 1], 0), p.T);
  int c0 = 0, c1 = 0;
  if (hi > lo) {
    c0 = lo / p.tokens_per_cta;
    c1 = (hi - 1) / p.tokens_per_cta + 1;
  }
  int n = 0;
  float z = 0.0f;
  for (int c = c0; c < c1; ++c) {
    n += p.part_tokens[c + b];
    z += p.part_z[c + b];
  }
  const float inv_n = n > 0 ? 1.0f / float(n) : 0.0f;
  float dot = 0.0f;
  for (int e = threadIdx.x; e < p.E; e += kRouteThreads) {
    float prob = 0.0f;
    int count = 0;
    for (int c = c0; c < c1; ++c) {
      prob += p.part_prob[int64_t(c + b) * p.E + e];
      count += p.part_count[int64_t(c + b) * p.E + e];
    }
    prob *= inv_n;
    p.expert_prob[int64_t(b) * p.E + e] = prob;
    p.expert_count[int64_t(b) * p.E + e] = count;
    dot += float(count) * inv_n * prob;
  }
  dot = block_sum(dot, scratch);
  if (threadIdx.x == 0) {
    p.seq_tokens[b] = n;
    p.seq_loss[b] = dot * (float(p.E) / float(p.K));
    p.seq_z[b] = z;
  }
}

// Third kernel: the losses over all sequences.
__global__ void __launch_bounds__(kRouteThreads) balance_loss_kernel(BalanceParams p) {
  __shared__ float scratch[kRouteWarps];
  pdl_wait();
  float loss = 0.0f, z = 0.0f;
  int n = 0, full = 0;
  for (int b = threadIdx.x; b < p.B; b += kRouteThreads) {
    loss += p.seq_loss[b];
    z += p.seq_z[b];
    n += p.seq_tokens[b];
    full += p.seq_tokens[b] > 0 ? 1 : 0;
  }
  loss = block_sum(loss, scratch);
  z = block_sum(z, scratch);
  __shared__ int totals[2];
  if (threadIdx.x < 2) totals[threadIdx.x] = 0;
  __syncthreads();
  atomicAdd(&totals[0], n);
  atomicAdd(&totals[1], full);
  __syncthreads();
  if (threadIdx.x == 0) {
    p.seq_tokens[p.B] = totals[0];
    p.seq_tokens[p.B + 1] = totals[1];
    p.loss[0] = totals[1] > 0 ? loss / float(totals[1]) : 0.0f;
    p.loss[1] = totals[0] > 0 ? z / float(totals[0]) : 0.0f;
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
  extern __shared__ float smem[];
  pdl_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  float* row = smem + warp * p.E;
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
  for (int t = first + warp; t < last; t += kRouteWarps) {
    float g[VPL];
    const int64_t out = int64_t(t) * p.ld_grad;
    if (p.mask != nullptr && p.mask[t] == 0) {
#pragma unroll
      for (int r = 0; r < VPL; ++r) g[r] = 0.0f;
      store_row<VPL, V, BF16>(p.grad, out, p.E, lane, g);
      continue;
    }
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
    float x[VPL], s[VPL], top;
    load_row<VPL, V, BF16>(p.logits, int64_t(t) * p.ld, p.E, lane, x);
    const float total = scores<VPL, SIG>(x, s, &top);
    const float inv = total == 0.0f ? 0.0f : 1.0f / total;
    // gate weights: lane k holds selection k
    int mine = -1;
    float ds = 0.0f, sk = 0.0f;
    if (p.grad_w != nullptr) {
      if (lane < p.K) {
        const int64_t e = p.idx[int64_t(t) * p.K + lane];
        mine = e >= 0 && e < p.E ? int(e) : -1;
      }
      if (mine >= 0) {
        const float l = load_one<BF16>(p.logits, int64_t(t) * p.ld + mine);
        sk = SIG ? sigmoid(l) : expf(l - top) * inv;
        ds = p.grad_w[int64_t(t) * p.K + lane] * p.scale;
      }
      if (p.renorm) {
        const float sum = warp_sum(sk);
        const float is = sum == 0.0f ? 0.0f : 1.0f / sum;
        const float mean = warp_sum(ds * sk) * is;
        if (mine >= 0) ds = (ds - mean) * is;
      }
      if (mine >= 0) row[mine] = ds;
      __syncwarp();
    }
    float dot = 0.0f;
#pragma unroll
    for (int r = 0; r < VPL; ++r) {
      const int e = element_of<V>(r, lane);
      g[r] = e < p.E ? row[e] : 0.0f;
      if constexpr (!SIG) {
        s[r] *= inv;
        g[r] += dq[r];
        dot += s[r] * g[r];
      } else {
        dot += s[r] * inv * dq[r];
      }
    }
    dot = warp_sum(dot);
    const float z = !SIG && total != 0.0f ? dlse * (top + logf(total)) : 0.0f;
#pragma unroll
    for (int r = 0; r < VPL; ++r) {
      if constexpr (SIG)
        g[r] = (g[r] + (dq[r] - dot) * inv) * s[r] * (1.0f - s[r]);
      else
        g[r] = s[r] * (g[r] - dot + z);
    }
    store_row<VPL, V, BF16>(p.grad, out, p.E, lane, g);
    if (p.grad_w != nullptr) {
      __syncwarp();
      if (mine >= 0) row[mine] = 0.0f;
      __syncwarp();
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

// CTAs of the per-token kernels over `tokens` tokens: at most eight an SM
// (2048 threads), each warp with a token at least.
int route_ctas(int tokens) {
  const int want = (tokens + kRouteWarps - 1) / kRouteWarps;
  const int most = device_info().sm_count * 8;
  return want < most ? want : most;
}

// Calls f.template operator()<VPL, V, BF16, SIG>() for the smallest VPL that
// holds E logits in a warp.  Rows whose vectors of four are aligned load
// those; narrow rows keep more lanes busy with single loads.
template <typename F>
cudaError_t with_shape(int E, int64_t ld, bool bf16, bool sig, F&& f) {
  const bool vec = E >= 128 && E % 4 == 0 && ld % 4 == 0;
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
  EP_SHAPE(4, 4) EP_SHAPE(8, 4) EP_SHAPE(16, 4) EP_SHAPE(32, 4) EP_SHAPE(64, 4)
#undef EP_SHAPE
  return cudaErrorInvalidValue;
}

// Raises a kernel's dynamic shared-memory limit where `bytes` needs it.
template <typename... P>
cudaError_t allow_smem(void (*kernel)(P...), size_t bytes) {
  if (bytes <= 48 * 1024) return cudaSuccess;
  return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, int(bytes));
}

struct LaunchRoute {
  RouteParams p;
  int ctas;
  cudaStream_t stream;
  template <int VPL, int V, bool BF16, bool SIG>
  cudaError_t operator()() const {
    const size_t smem = p.G > 1 ? sizeof(float) * kRouteWarps * p.E : 0;
    auto* kernel = route_kernel<VPL, V, BF16, SIG>;
    const cudaError_t e = allow_smem(kernel, smem);
    if (e != cudaSuccess) return e;
    return launch_pdl(kernel, dim3(ctas), dim3(kRouteThreads), smem, stream, p);
  }
};

struct LaunchBalance {
  RouteParams p;
  cudaStream_t stream;
  template <int VPL, int V, bool BF16, bool SIG>
  cudaError_t operator()() const {
    const size_t smem = sizeof(float) * (kRouteWarps + 1) * p.E;
    auto* kernel = balance_kernel<VPL, V, BF16, SIG>;
    const cudaError_t e = allow_smem(kernel, smem);
    if (e != cudaSuccess) return e;
    return launch_pdl(kernel, dim3(p.ctas), dim3(kRouteThreads), smem, stream, p);
  }
};

struct LaunchBackward {
  RouteBackwardParams p;
  int ctas;
  cudaStream_t stream;
  template <int VPL, int V, bool BF16, bool SIG>
  cudaError_t operator()() const {
    const size_t smem = sizeof(float) * kRouteWarps * p.E;
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
  float* seq_loss;
  float* seq_z;
  int64_t bytes;
};

// ctas <= sm_count * 8, so that the size does not depend on T.
BalanceWorkspace carve(void* base, int E, int B) {
  const int64_t rows = int64_t(device_info().sm_count) * 8 + B;
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
  w.seq_loss = reinterpret_cast<float*>(take(B));
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
  l.p.tokens_per_cta = run_length(num_tokens);
  l.p.ctas = (num_tokens + l.p.tokens_per_cta - 1) / l.p.tokens_per_cta;
  l.p.part_prob = w.prob;
  l.p.part_count = w.count;
  l.p.part_tokens = w.tokens;
  l.p.part_z = w.z;
  if (num_tokens > 0) {
    const cudaError_t e = with_shape(l.p.E, ld_logits, cfg->logits_bf16 != 0,
                                     cfg->score == EP_SCORE_SIGMOID, l);
    if (note_cuda(e) != cudaSuccess) return EP_ERR_CUDA;
  }
  BalanceParams q;
  q.seq_start = d_seq_start;
  q.T = num_tokens;
  q.E = l.p.E;
  q.K = l.p.K;
  q.B = num_seqs;
  q.tokens_per_cta = l.p.tokens_per_cta;
  q.ctas = l.p.ctas;
  q.part_prob = w.prob;
  q.part_count = w.count;
  q.part_tokens = w.tokens;
  q.part_z = w.z;
  q.expert_count = d_expert_count;
  q.expert_prob = d_expert_prob;
  q.seq_tokens = d_seq_tokens;
  q.seq_loss = w.seq_loss;
  q.seq_z = w.seq_z;
  q.loss = d_loss;
  cudaError_t e = launch_pdl(balance_sum_kernel, dim3(num_seqs), dim3(kRouteThreads), 0,
                             l.stream, q);
  if (e == cudaSuccess)
    e = launch_pdl(balance_loss_kernel, dim3(1), dim3(kRouteThreads), 0, l.stream, q);
  return status(e);
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

// The gated activation between an expert's two products, with its input kept
// in 8 bits for the backward pass (ep_act_save, ep_act_backward).
//
// a = silu(g) u.  The forward pass reads h = [g, u] once and writes a beside
// E4M3 codes of h in blocks of 128 columns; the backward pass reads those and
// the gradient of a, and writes the gradient of h and a again.  A few
// operations a byte: memory bounds both.
//
// A warp takes four blocks of g and the same four of u of one row: 8 lanes a
// block, 16 columns a lane, so that a block's maximum is three shuffles.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "../../include/ep.h"
#include "ep_internal.h"
#include "fp8_quant.cuh"

namespace ep {
namespace {

constexpr int kThreads = 256;
constexpr int kBlock = 128;
constexpr int kSpan = 512;        // columns of g a warp takes at a time

struct ActParams {
  int E, I, cap;
  int spans;                      // kSpan pieces of a row
  const int32_t *start, *end;
  const uint8_t* h;               // bf16 (save)
  const uint8_t* grad_a;          // bf16 (backward)
  uint8_t *a, *grad_h;            // bf16
  uint8_t* q;
  float* scale;
};

// Rows of the experts before each one, in shared memory: table[E + 1].
__device__ void count_rows(const ActParams& p, int* table) {
  const int lane = threadIdx.x % 32;
  for (int e = threadIdx.x; e < p.E; e += kThreads) {
    const int s = min(max(__ldg(p.start + e), 0), p.cap);
    table[e + 1] = max(min(__ldg(p.end + e), p.cap) - s, 0);
  }
  __syncthreads();
  if (threadIdx.x < 32) {
    int64_t sum = 0;
    for (int e0 = 0; e0 < p.E; e0 += 32) {
      int64_t v = e0 + lane < p.E ? table[e0 + lane + 1] : 0;
#pragma unroll
      for (int o = 1; o < 32; o *= 2) {
        const int64_t u = __shfl_up_sync(0xffffffffu, v, o);
        if (lane >= o) v += u;
      }
      if (e0 + lane < p.E) table[e0 + lane + 1] = int(min(sum + v, int64_t(INT32_MAX)));
      sum += __shfl_sync(0xffffffffu, v, 31);
    }
    if (lane == 0) table[0] = 0;
  }
  __syncthreads();
}

// The buffer row of the r-th row of all experts.
__device__ __forceinline__ int64_t row_of(const ActParams& p, const int* table, int r) {
  int lo = 0, hi = p.E;
  while (hi - lo > 1) {
    const int mid = (lo + hi) / 2;
    if (table[mid] <= r)
      lo = mid;
    else
      hi = mid;
  }
  return min(max(__ldg(p.start + lo), 0), p.cap) + (r - table[lo]);
}

__device__ __forceinline__ void unpack(uint4 v, float* f) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = bf16_lo(w[i]);
    f[2 * i + 1] = bf16_hi(w[i]);
  }
}

__device__ __forceinline__ uint4 pack(const float* f) {
  return make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]),
                    pack_bf16x2(f[6], f[7]));
}

// Eight E4M3 values times their scale.
__device__ __forceinline__ void unpack8(uint2 v, float scale, float* f) {
  const uint32_t w[2] = {v.x, v.y};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint16_t two = uint16_t(w[i / 2] >> (16 * (i % 2)));
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(two));
    float a, b;
    asm("{\n\t.reg .f16 l, u;\n\tmov.b32 {l, u}, %2;\n\tcvt.f32.f16 %0, l;\n\tcvt.f32.f16 %1, u;\n\t}"
        : "=f"(a), "=f"(b)
        : "r"(h));
    f[2 * i] = a * scale;
    f[2 * i + 1] = b * scale;
  }
}

__device__ __forceinline__ uint4 load16(const uint8_t* p, bool there) {
  return there ? ld_stream_u4(p) : make_uint4(0, 0, 0, 0);
}

__global__ void __launch_bounds__(kThreads) act_save_kernel(const ActParams p) {
  extern __shared__ int table[];
  pdl_wait();
  count_rows(p, table);
  const int lane = threadIdx.x % 32;
  const int64_t items = int64_t(table[p.E]) * p.spans;
  const int blocks = (p.I + kBlock - 1) / kBlock;
  const int64_t step = int64_t(gridDim.x) * (kThreads / 32);
  for (int64_t i = int64_t(blockIdx.x) * (kThreads / 32) + threadIdx.x / 32; i < items; i += step) {
    const int r = int(i / p.spans);
    const int c = int(i - int64_t(r) * p.spans) * kSpan + lane * 16;     // first column
    const int64_t row = row_of(p, table, r);
    const bool lo = c < p.I, hi = c + 8 < p.I;
    const uint8_t* g = p.h + (row * 2 * p.I + c) * 2;
    const uint8_t* u = g + int64_t(p.I) * 2;
    const uint4 g0 = load16(g, lo), g1 = load16(g + 16, hi);
    const uint4 u0 = load16(u, lo), u1 = load16(u + 16, hi);
    float x[16], y[16];
    unpack(g0, x);
    unpack(g1, x + 8);
    unpack(u0, y);
    unpack(u1, y + 8);
#pragma unroll
    for (int j = 0; j < 16; ++j) y[j] *= x[j] / (1.0f + expf(-x[j]));
    uint8_t* a = p.a + (row * p.I + c) * 2;
    if (lo) *reinterpret_cast<uint4*>(a) = pack(y);
    if (hi) *reinterpret_cast<uint4*>(a + 16) = pack(y + 8);
    uint4 gq, uq;
    float gs, us;
    quantize_group16(g0, g1, &gq, &gs);
    quantize_group16(u0, u1, &uq, &us);
    uint8_t* q = p.q + row * 2 * p.I + c;
    if (lo) {
      *reinterpret_cast<uint2*>(q) = make_uint2(gq.x, gq.y);
      *reinterpret_cast<uint2*>(q + p.I) = make_uint2(uq.x, uq.y);
    }
    if (hi) {
      *reinterpret_cast<uint2*>(q + 8) = make_uint2(gq.z, gq.w);
      *reinterpret_cast<uint2*>(q + p.I + 8) = make_uint2(uq.z, uq.w);
    }
    if (lo && lane % 8 == 0) {
      float* s = p.scale + row * 2 * blocks + c / kBlock;
      s[0] = gs;
      s[blocks] = us;
    }
  }
}

__global__ void __launch_bounds__(kThreads) act_backward_kernel(const ActParams p) {
  extern __shared__ int table[];
  pdl_wait();
  count_rows(p, table);
  const int lane = threadIdx.x % 32;
  const int64_t items = int64_t(table[p.E]) * p.spans;
  const int blocks = (p.I + kBlock - 1) / kBlock;
  const int64_t step = int64_t(gridDim.x) * (kThreads / 32);
  for (int64_t i = int64_t(blockIdx.x) * (kThreads / 32) + threadIdx.x / 32; i < items; i += step) {
    const int r = int(i / p.spans);
    const int c0 = int(i - int64_t(r) * p.spans) * kSpan;
    const int64_t row = row_of(p, table, r);
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      // eight columns a lane
      const int c = c0 + half * (kSpan / 2) + lane * 8;
      if (c >= p.I) continue;
      const uint8_t* q = p.q + row * 2 * p.I + c;
      const float* s = p.scale + row * 2 * blocks + c / kBlock;
      float g[8], u[8], d[8], dg[8], du[8], a[8];
      const uint2 gq = __ldg(reinterpret_cast<const uint2*>(q));
      const uint2 uq = __ldg(reinterpret_cast<const uint2*>(q + p.I));
      unpack(ld_stream_u4(p.grad_a + (row * p.I + c) * 2), d);
      unpack8(gq, __ldg(s), g);
      unpack8(uq, __ldg(s + blocks), u);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float t = 1.0f / (1.0f + expf(-g[j]));
        const float act = g[j] * t;
        dg[j] = d[j] * u[j] * t * (1.0f + g[j] * (1.0f - t));
        du[j] = d[j] * act;
        a[j] = act * u[j];
      }
      uint8_t* h = p.grad_h + (row * 2 * p.I + c) * 2;
      *reinterpret_cast<uint4*>(h) = pack(dg);
      *reinterpret_cast<uint4*>(h + int64_t(p.I) * 2) = pack(du);
      if (p.a != nullptr) *reinterpret_cast<uint4*>(p.a + (row * p.I + c) * 2) = pack(a);
    }
  }
}

bool aligned(const void* p) { return p != nullptr && reinterpret_cast<uintptr_t>(p) % 16 == 0; }

bool sizes_ok(int32_t E, int32_t I, int32_t cap, int32_t num_rows) {
  return E >= 1 && E <= 2048 && I >= 8 && I <= (1 << 19) && I % 8 == 0 && cap >= 0 &&
         num_rows >= 0;
}

int32_t launch(void (*kernel)(ActParams), const ActParams& p, int num_rows, void* stream) {
  const int64_t items = int64_t(num_rows) * p.spans;
  const int64_t most = int64_t(device_info().sm_count) * 8;
  const int64_t ctas = (items + kThreads / 32 - 1) / (kThreads / 32);
  return note_cuda(launch_pdl(kernel, dim3(unsigned(ctas < most ? ctas : most)), dim3(kThreads),
                              sizeof(int) * (p.E + 1), static_cast<cudaStream_t>(stream), p)) ==
                 cudaSuccess
             ? EP_OK
             : EP_ERR_CUDA;
}

ActParams params(int32_t E, int32_t I, int32_t cap, const int32_t* start, const int32_t* end) {
  ActParams p = {};
  p.E = E;
  p.I = I;
  p.cap = cap;
  p.spans = (I + kSpan - 1) / kSpan;
  p.start = start;
  p.end = end;
  return p;
}

}  // namespace
}  // namespace ep

using namespace ep;

extern "C" {

int32_t ep_act_save(int32_t num_experts, int32_t width, int32_t cap, int32_t num_rows,
                    const void* d_h, const int32_t* d_expert_start, const int32_t* d_expert_end,
                    void* d_a, uint8_t* d_q, float* d_scale, void* stream) {
  if (!sizes_ok(num_experts, width, cap, num_rows)) return EP_ERR_INVALID_ARG;
  if (!aligned(d_expert_start) || !aligned(d_expert_end)) return EP_ERR_INVALID_ARG;
  if (cap > 0 && (!aligned(d_h) || !aligned(d_a) || !aligned(d_q) || !aligned(d_scale)))
    return EP_ERR_INVALID_ARG;
  if (cap == 0 || num_rows == 0) return EP_OK;
  ActParams p = params(num_experts, width, cap, d_expert_start, d_expert_end);
  p.h = static_cast<const uint8_t*>(d_h);
  p.a = static_cast<uint8_t*>(d_a);
  p.q = d_q;
  p.scale = d_scale;
  return launch(act_save_kernel, p, num_rows, stream);
}

int32_t ep_act_backward(int32_t num_experts, int32_t width, int32_t cap, int32_t num_rows,
                        const void* d_grad_a, const uint8_t* d_q, const float* d_scale,
                        const int32_t* d_expert_start, const int32_t* d_expert_end,
                        void* d_grad_h, void* d_a, void* stream) {
  if (!sizes_ok(num_experts, width, cap, num_rows)) return EP_ERR_INVALID_ARG;
  if (!aligned(d_expert_start) || !aligned(d_expert_end)) return EP_ERR_INVALID_ARG;
  if (cap > 0 &&
      (!aligned(d_grad_a) || !aligned(d_q) || !aligned(d_scale) || !aligned(d_grad_h)))
    return EP_ERR_INVALID_ARG;
  if (d_a != nullptr && !aligned(d_a)) return EP_ERR_INVALID_ARG;
  if (cap == 0 || num_rows == 0) return EP_OK;
  ActParams p = params(num_experts, width, cap, d_expert_start, d_expert_end);
  p.grad_a = static_cast<const uint8_t*>(d_grad_a);
  p.q = const_cast<uint8_t*>(d_q);
  p.scale = const_cast<float*>(d_scale);
  p.grad_h = static_cast<uint8_t*>(d_grad_h);
  p.a = static_cast<uint8_t*>(d_a);
  return launch(act_backward_kernel, p, num_rows, stream);
}

}  // extern "C"

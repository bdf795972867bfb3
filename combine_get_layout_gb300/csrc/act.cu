// The gated activation between an expert's two products, with its input kept
// in 8 bits for the backward pass (ep_act_save, ep_act_backward).
//
// a = silu(g) u.  The forward pass reads h = [g, u] once and writes a beside
// E4M3 codes of h in blocks of 128 columns; the backward pass reads those and
// the gradient of a, and writes the gradient of h and a again.  A few
// operations a byte: memory bounds both.
//
// A warp walks along a row, 256 columns of g and the same of u in a step, 8
// adjacent columns a lane, so that every access of a warp is one contiguous
// piece; 16 lanes hold one block of 128, whose maximum is four shuffles.  The
// loads of a warp's next step are issued before the present one is computed.
//
// 32768 rows of 2 x 2048: save 94.5 us (541 MB, 5.7 TB/s; two issue slots of
// three are taken), backward 107 us (675 MB, 6.3 TB/s).
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "../../include/ep.h"
#include "ep_internal.h"
#include "fp8_quant.cuh"
#include "segments.cuh"

namespace ep {
namespace {

constexpr int kThreads = 256;
constexpr int kCtasPerSm = 4;     // 64 registers a thread
constexpr int kBlock = 128;
constexpr int kStep = 256;        // columns of g a warp takes in one step

struct ActParams {
  int E, I, cap;
  int parts, part;                // a row is walked in `parts` of `part` columns
  const int32_t *start, *end;
  const uint8_t* h;               // bf16 (save)
  const uint8_t* grad_a;          // bf16 (backward)
  uint8_t *a, *grad_h;            // bf16
  uint8_t* q;
  float* scale;
};

// Rows of the experts before each one: table[E + 1] in shared memory.
__device__ __forceinline__ void count_rows(const ActParams& p, int* table) {
  __shared__ int64_t partial[kThreads / 32];
  count_experts(p.E, table, partial, [&](int e) {
    int first, rows;
    clip_segment(p.start, p.end, p.cap, e, first, rows);
    return rows;
  });
}

// A warp's walk over the parts of all experts' rows, a step at a time.
struct Walk {
  int64_t r = 0;         // row among the experts' rows
  int64_t row = 0;       // in the buffers
  int part, col, end;    // part of it, first column of the step, end of the part
  int e = -1;
  int first;             // buffer row of the expert's first

  __device__ __forceinline__ bool enter(const ActParams& p, const int* table) {
    if (r >= table[p.E]) return false;
    if (e < 0 || r < table[e] || r >= table[e + 1]) {
      e = expert_of(table, p.E, r);
      int rows;
      clip_segment(p.start, p.end, p.cap, e, first, rows);
    }
    row = int64_t(first) + (r - table[e]);
    col = part * p.part;
    end = min(col + p.part, p.I);
    return true;
  }
  __device__ __forceinline__ bool begin(const ActParams& p, const int* table) {
    const int at = blockIdx.x * (kThreads / 32) + threadIdx.x / 32;
    r = at / p.parts;
    part = at % p.parts;
    return enter(p, table);
  }
  __device__ __forceinline__ bool next(const ActParams& p, const int* table) {
    col += kStep;
    if (col < end) return true;
    const int at = part + gridDim.x * (kThreads / 32);
    r += at / p.parts;
    part = at % p.parts;
    return enter(p, table);
  }
};

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
    asm("{\n\t.reg .f16 l, u;\n\tmov.b32 {l, u}, %2;\n\t"
        "cvt.f32.f16 %0, l;\n\tcvt.f32.f16 %1, u;\n\t}"
        : "=f"(a), "=f"(b)
        : "r"(h));
    f[2 * i] = a * scale;
    f[2 * i + 1] = b * scale;
  }
}

// 1 / (1 + exp(-x)) by the hardware's exponential and reciprocal: within
// (2 + |x|) 2^-22 of itself, far inside the rounding to bf16 behind it, at a
// quarter of the instructions that expf and a division take (which bound the
// kernels).  Below 2^-126 it is 0.
__device__ __forceinline__ float sigmoid(float x) {
  float e, r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(x * -1.44269504088896340736f));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.0f + e));
  return r;
}

// What lanes past a row's end hold: NaN, which no maximum takes from a block
// that has a value, and which leaves a block of NaN alone one.
constexpr uint32_t kNoValue = 0x7fff7fff;

// A block of zeros and NaN has a maximum of 0, and 0 in all its codes as in a
// dispatch; its scale is -0 (no other block's is), by which the backward pass
// knows it: it reads as NaN.
constexpr uint32_t kNanAmongZeros = 0x80000000;

__device__ __forceinline__ float kept_scale(float s) {
  return __float_as_uint(s) == kNanAmongZeros ? __uint_as_float(0x7fffffff) : s;
}

__device__ __forceinline__ bool any_nan(const float* f) {
  bool nan = false;
#pragma unroll
  for (int j = 0; j < 8; ++j) nan |= f[j] != f[j];
  return nan;
}

// The larger of two pairs of magnitudes; NaN is not larger.
__device__ __forceinline__ uint32_t max2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

// The larger of the magnitudes of eight values, in both halves.
__device__ __forceinline__ uint32_t most8(uint4 v) {
  constexpr uint32_t kMagnitude = 0x7fff7fff;
  const uint32_t m = max2(max2(v.x & kMagnitude, v.y & kMagnitude),
                          max2(v.z & kMagnitude, v.w & kMagnitude));
  return max2(m, __byte_perm(m, m, 0x1032));
}

// The codes of eight values f (packed: v) of a block with this maximum, and
// the block's scale: amax / 448 and the codes of the quotients as in
// quantize_group16, but for a block of NaN alone: its maximum, and so its
// scale and codes, are NaN.
__device__ __forceinline__ uint2 quantize8(uint4 v, const float* f, float amax, float* scale) {
  // |a| / 448 by its reciprocal and one exact remainder is the IEEE quotient
  // for every bf16 value from 2^-90 on (all were compared)
  constexpr float kPart = 1.0f / 448.0f;
  if (amax >= 0x1p-90f && amax <= 0x1.fffffep127f) {
    const float q0 = amax * kPart;
    const float s = fmaf(fmaf(-q0, 448.0f, amax), kPart, q0);
    *scale = s;
    // scaled_quotient's, the signs from the values (a quotient of -0 is -0)
    const float y = __frcp_rn(s);
    uint32_t c[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float a = f[2 * j], b = f[2 * j + 1];
      const float qa = a * y, qb = b * y;
      c[j] = pack_e4m3x2(fmaf(fmaf(-qa, s, a), y, qa), fmaf(fmaf(-qb, s, b), y, qb));
    }
    constexpr uint32_t kSigns = 0x80808080;
    return make_uint2(__byte_perm(c[0], c[1], 0x5410) | (__byte_perm(v.x, v.y, 0x7531) & kSigns),
                      __byte_perm(c[2], c[3], 0x5410) | (__byte_perm(v.z, v.w, 0x7531) & kSigns));
  }
  // (amax itself: 0, or NaN; lanes past a row's end come here too, and divide
  // nothing)
  *scale = amax;
  if (amax == 0.0f) return make_uint2(0, 0);
  if (amax != amax) return make_uint2(0x7f7f7f7f, 0x7f7f7f7f);
  const float s = __fdiv_rn(amax, 448.0f);
  *scale = s;
  uint32_t c[4];
#pragma unroll
  for (int j = 0; j < 4; ++j)
    c[j] = pack_e4m3x2(__fdiv_rn(f[2 * j], s), __fdiv_rn(f[2 * j + 1], s));
  return make_uint2(c[0] | c[1] << 16, c[2] | c[3] << 16);
}

__global__ void __launch_bounds__(kThreads, kCtasPerSm) act_save_kernel(const ActParams p) {
  extern __shared__ int table[];
  pdl_wait();
  count_rows(p, table);
  const int lane = threadIdx.x % 32;
  const int blocks = (p.I + kBlock - 1) / kBlock;
  Walk w;
  uint4 g, u;
  const uint8_t* h = nullptr;      // of the row
  const auto load = [&] {
    const int c = w.col + lane * 8;
    g = u = make_uint4(kNoValue, kNoValue, kNoValue, kNoValue);
    if (c < w.end) {
      g = ld_stream_u4(h + c * 2);
      u = ld_stream_u4(h + (c + p.I) * 2);
    }
  };
  bool there = w.begin(p, table);
  int64_t row = w.row;
  if (there) {
    h = p.h + row * 4 * p.I;
    load();
  }
  while (there) {
    const uint4 gv = g, uv = u;
    uint8_t* const a = p.a + row * 2 * p.I;
    uint8_t* const q = p.q + row * 2 * p.I;
    float* const s = p.scale + row * 2 * blocks;
    const int c = w.col + lane * 8;
    const bool in = c < w.end;
    there = w.next(p, table);
    if (there) {
      if (w.row != row) h = p.h + w.row * 4 * p.I;
      load();
    }
    row = w.row;
    // both maxima in one word
    uint32_t m = __byte_perm(most8(gv), most8(uv), 0x5410);
#pragma unroll
    for (int o = 8; o >= 1; o >>= 1) m = max2(m, __shfl_xor_sync(0xffffffffu, m, o));
    float x[8], y[8], x_scale, y_scale;
    unpack(gv, x);
    unpack(uv, y);
    const uint2 xq = quantize8(gv, x, bf16_lo(m), &x_scale);
    const uint2 yq = quantize8(uv, y, bf16_hi(m), &y_scale);
    // (one vote a step where no block is 0)
    if (__any_sync(0xffffffffu, (m & 0xffffu) == 0 || m >> 16 == 0)) {
      const uint32_t block = 0xffffu << (lane & 16);
      const uint32_t x_nan = __ballot_sync(0xffffffffu, in && any_nan(x)) & block;
      const uint32_t y_nan = __ballot_sync(0xffffffffu, in && any_nan(y)) & block;
      if ((m & 0xffffu) == 0 && x_nan != 0) x_scale = __uint_as_float(kNanAmongZeros);
      if (m >> 16 == 0 && y_nan != 0) y_scale = __uint_as_float(kNanAmongZeros);
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) y[j] *= x[j] * sigmoid(x[j]);
    if (in) {
      *reinterpret_cast<uint4*>(a + c * 2) = pack(y);
      *reinterpret_cast<uint2*>(q + c) = xq;
      *reinterpret_cast<uint2*>(q + c + p.I) = yq;
      if (lane % 16 == 0) {
        s[c / kBlock] = x_scale;
        s[c / kBlock + blocks] = y_scale;
      }
    }
  }
}

__global__ void __launch_bounds__(kThreads, kCtasPerSm) act_backward_kernel(const ActParams p) {
  extern __shared__ int table[];
  pdl_wait();
  count_rows(p, table);
  const int lane = threadIdx.x % 32;
  const int blocks = (p.I + kBlock - 1) / kBlock;
  Walk w;
  uint4 d;
  uint2 gq, uq;
  float gs, us;
  const auto load = [&] {
    const int c = w.col + lane * 8;
    if (c >= w.end) return;
    const uint8_t* q = p.q + w.row * 2 * p.I + c;
    const float* s = p.scale + w.row * 2 * blocks + c / kBlock;
    d = ld_stream_u4(p.grad_a + (w.row * p.I + c) * 2);
    gq = __ldg(reinterpret_cast<const uint2*>(q));
    uq = __ldg(reinterpret_cast<const uint2*>(q + p.I));
    gs = __ldg(s);
    us = __ldg(s + blocks);
  };
  bool there = w.begin(p, table);
  if (there) load();
  while (there) {
    float x[8], y[8], da[8], dg[8];
    const uint4 dv = d;
    const uint2 gv = gq, uv = uq;
    const float g_scale = gs, u_scale = us;
    const int64_t row = w.row;
    const int c = w.col + lane * 8;
    const bool in = c < w.end;
    there = w.next(p, table);
    if (there) load();
    if (!in) continue;
    unpack(dv, da);
    unpack8(gv, kept_scale(g_scale), x);
    unpack8(uv, kept_scale(u_scale), y);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float t = sigmoid(x[j]);
      const float act = x[j] * t;
      dg[j] = da[j] * y[j] * t * (1.0f + x[j] * (1.0f - t));
      da[j] *= act;
      y[j] *= act;
    }
    uint8_t* h = p.grad_h + (row * 2 * p.I + c) * 2;
    *reinterpret_cast<uint4*>(h) = pack(dg);
    *reinterpret_cast<uint4*>(h + int64_t(p.I) * 2) = pack(da);
    if (p.a != nullptr) *reinterpret_cast<uint4*>(p.a + (row * p.I + c) * 2) = pack(y);
  }
}

bool aligned(const void* p) { return p != nullptr && reinterpret_cast<uintptr_t>(p) % 16 == 0; }

bool sizes_ok(int32_t E, int32_t I, int32_t cap, int32_t num_rows) {
  return E >= 1 && E <= 2048 && I >= 8 && I <= (1 << 19) && I % 8 == 0 && cap >= 0 &&
         num_rows >= 0;
}

int32_t launch(void (*kernel)(ActParams), ActParams p, int num_rows, void* stream) {
  // a row a warp, or its steps spread over warps where the rows are few
  const int64_t most = int64_t(device_info().sm_count) * kCtasPerSm;
  const int steps = (p.I + kStep - 1) / kStep;
  const int64_t warps = most * (kThreads / 32);
  const int64_t wanted = (warps + num_rows - 1) / num_rows;
  const int parts = int(wanted < steps ? wanted : steps);
  p.part = (steps + parts - 1) / parts * kStep;
  p.parts = (p.I + p.part - 1) / p.part;
  const int64_t items = int64_t(num_rows) * p.parts;
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

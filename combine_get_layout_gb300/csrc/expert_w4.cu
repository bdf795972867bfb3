// Experts' products with 4-bit weights (ep_expert_w4) and the packing of the
// weights (ep_w4_pack).
//
// At decode an expert has a few rows, so the cost is reading its weights
// once; a 64 x 128 tile of packed codes is 4 KiB in the order a warp loads
// it (lane after lane, 16 bytes each).  The codes become bf16 (f16 for E4M3
// rows, which f16 holds exactly) small integers in registers and are
// multiplied by the rows on the tensor cores, weights as the 16-row operand
// and up to eight rows of x as the columns: mma.m16n8k16, fp32 sums.  The
// integers are exact, and the scales multiply the fp32 sum of each group, so
// nothing is rounded before the end.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "../../include/ep.h"
#include "ep_device.cuh"
#include "ep_internal.h"

namespace ep {
namespace {

constexpr int kW4Threads = 256;
constexpr int kW4Warps = kW4Threads / 32;
constexpr int kTileRows = 64;      // packed weight rows a tile
constexpr int kBlockIn = 128;      // inputs a block
constexpr int kChunk = 8;          // rows of x a warp multiplies at once
constexpr int kWordsPerBlock = kTileRows * kBlockIn / 8;

struct W4Params {
  int E, H, N;              // N: output columns (half the weight rows when gated)
  int tiles, blocks;
  int cap;
  bool gated;
  const void* x;            // [cap, H]
  const float* x_scale;     // [cap, H / 128] (E4M3)
  const uint32_t* codes;
  const __nv_bfloat16* scales;
  const uint8_t* zeros;     // or null
  const int32_t *start, *end;
  __nv_bfloat16* out;       // [cap, N]
};

// ---- arithmetic on packed pairs -------------------------------------------------

template <bool FP8>
__device__ __forceinline__ void mma(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                    uint32_t a3, uint32_t b0, uint32_t b1) {
  if constexpr (FP8)
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  else
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// The exponent that makes a 16-bit float with integer mantissa bits: 128 + q
// in bf16 (7 mantissa bits), 1024 + q in f16 (10), both exact.
template <bool FP8>
constexpr uint32_t kOffsetBits = FP8 ? 0x64006400u : 0x43004300u;

// 16-bit float pair (offset + zero, offset + zero).
template <bool FP8>
__device__ __forceinline__ uint32_t offset_pair(uint32_t zero) {
  return kOffsetBits<FP8> + zero * 0x00010001u;
}

// Fields j and j + 4 of a word minus the zero point, as a 16-bit float pair.
template <bool FP8>
__device__ __forceinline__ uint32_t decode(uint32_t word, int j, uint32_t offset) {
  const uint32_t u = ((word >> (4 * j)) & 0x000F000Fu) | kOffsetBits<FP8>;
  uint32_t r;
  if constexpr (FP8)
    asm("sub.f16x2 %0, %1, %2;" : "=r"(r) : "r"(u), "r"(offset));
  else
    asm("sub.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(u), "r"(offset));
  return r;
}

// Two E4M3 values as an f16 pair (exact).
__device__ __forceinline__ uint32_t e4m3_pair(uint32_t two) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(uint16_t(two)));
  return r;
}

// ---- the product ----------------------------------------------------------------

// Chunks of kChunk rows before each expert, in shared memory: pre[e] of e's
// predecessors, pre[E] of all.
__device__ void count_chunks(const W4Params& p, int* pre) {
  for (int e = threadIdx.x; e < p.E; e += kW4Threads) {
    const int lo = max(0, p.start[e]), hi = min(p.cap, p.end[e]);
    pre[e] = hi > lo ? (hi - lo + kChunk - 1) / kChunk : 0;
  }
  __syncthreads();
  if (threadIdx.x < 32) {
    int carry = 0;
    for (int e0 = 0; e0 < p.E; e0 += 32) {
      const int e = e0 + threadIdx.x;
      const int mine = e < p.E ? pre[e] : 0;
      int sum = mine;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const int up = __shfl_up_sync(0xffffffffu, sum, d);
        if (int(threadIdx.x) >= d) sum += up;
      }
      if (e < p.E) pre[e] = carry + sum - mine;
      carry += __shfl_sync(0xffffffffu, sum, 31);
    }
    if (threadIdx.x == 0) pre[p.E] = carry;
  }
  __syncthreads();
}

// The expert whose chunks hold chunk c.
__device__ __forceinline__ int expert_of(const int* pre, int E, int c) {
  int lo = 0, hi = E - 1;
  while (lo < hi) {
    const int mid = (lo + hi) / 2;
    if (pre[mid + 1] > c)
      hi = mid;
    else
      lo = mid + 1;
  }
  return lo;
}

// One warp: a tile of 64 packed weight rows by a chunk of up to 8 rows of x.
// Lane (g = lane / 4, q = lane % 4) holds packed rows 8 g .. 8 g + 7 (piece
// 2 r + h is row g + 8 h of the r-th 16-row operand) and columns 2 q, 2 q + 1.
template <bool FP8, int GROUP, bool ZEROS>
__global__ void __launch_bounds__(kW4Threads) expert_w4_kernel(W4Params p) {
  extern __shared__ int pre[];
  pdl_wait();
  count_chunks(p, pre);
  const int lane = threadIdx.x & 31, g = lane >> 2, q = lane & 3;
  constexpr int kGroups = kBlockIn / GROUP;       // scale groups a block
  constexpr int kWords = GROUP / 32;              // words of a lane a group
  const int64_t items = int64_t(pre[p.E]) * p.tiles;
  const int64_t step = int64_t(gridDim.x) * kW4Warps;
  for (int64_t it = int64_t(blockIdx.x) * kW4Warps + (threadIdx.x >> 5); it < items; it += step) {
    const int chunk = int(it / p.tiles), tile = int(it % p.tiles);
    const int e = expert_of(pre, p.E, chunk);
    const int row0 = max(0, p.start[e]) + (chunk - pre[e]) * kChunk;
    const int rows = min(kChunk, min(p.cap, p.end[e]) - row0);
    const int64_t unit0 = (int64_t(e) * p.tiles + tile) * p.blocks;
    const uint4* codes = reinterpret_cast<const uint4*>(p.codes) + unit0 * (kWordsPerBlock / 4) + lane;
    const __nv_bfloat16* scales = p.scales + unit0 * kGroups * kTileRows + 8 * g;
    const uint8_t* zeros = ZEROS ? p.zeros + unit0 * kGroups * kTileRows + 8 * g : nullptr;
    float acc[4][4] = {};
    for (int kb = 0; kb < p.blocks; ++kb) {
      uint4 w[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) w[i] = ld_stream_u4(codes + kb * (kWordsPerBlock / 4) + i * 32);
      // columns: row g of the chunk, inputs 32 i + 8 q .. + 7
      uint32_t b[16] = {};
      float sx[2] = {1.0f, 1.0f};
      if constexpr (FP8) {
        if (g < rows) {
          const uint8_t* x = static_cast<const uint8_t*>(p.x) + int64_t(row0 + g) * p.H + kb * kBlockIn + 8 * q;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const uint2 v = *reinterpret_cast<const uint2*>(x + 32 * i);
            b[4 * i] = e4m3_pair(v.x);
            b[4 * i + 1] = e4m3_pair(v.x >> 16);
            b[4 * i + 2] = e4m3_pair(v.y);
            b[4 * i + 3] = e4m3_pair(v.y >> 16);
          }
        }
#pragma unroll
        for (int c = 0; c < 2; ++c)
          sx[c] = 2 * q + c < rows ? p.x_scale[int64_t(row0 + 2 * q + c) * p.blocks + kb] : 0.0f;
      } else {
        if (g < rows) {
          const __nv_bfloat16* x = static_cast<const __nv_bfloat16*>(p.x) + int64_t(row0 + g) * p.H;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int k = kb * kBlockIn + 32 * i + 8 * q;
            if (k < p.H) {
              const uint4 v = *reinterpret_cast<const uint4*>(x + k);
              b[4 * i] = v.x;
              b[4 * i + 1] = v.y;
              b[4 * i + 2] = v.z;
              b[4 * i + 3] = v.w;
            }
          }
        }
      }
#pragma unroll
      for (int s = 0; s < kGroups; ++s) {
        const int64_t at = (int64_t(kb) * kGroups + s) * kTileRows;
        const uint4 sv = *reinterpret_cast<const uint4*>(scales + at);
        const uint32_t sw[4] = {sv.x, sv.y, sv.z, sv.w};
        uint2 zv = make_uint2(0x08080808u, 0x08080808u);
        if constexpr (ZEROS) zv = *reinterpret_cast<const uint2*>(zeros + at);
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const uint32_t z = (r < 2 ? zv.x : zv.y) >> (16 * (r & 1));
          const uint32_t o0 = offset_pair<FP8>(z & 0xFFu), o1 = offset_pair<FP8>((z >> 8) & 0xFFu);
          float d[4] = {};
#pragma unroll
          for (int i = s * kWords; i < (s + 1) * kWords; ++i) {
            const uint4 lo4 = w[2 * r], hi4 = w[2 * r + 1];
            const uint32_t lo = i == 0 ? lo4.x : i == 1 ? lo4.y : i == 2 ? lo4.z : lo4.w;
            const uint32_t hi = i == 0 ? hi4.x : i == 1 ? hi4.y : i == 2 ? hi4.z : hi4.w;
            mma<FP8>(d, decode<FP8>(lo, 0, o0), decode<FP8>(hi, 0, o1), decode<FP8>(lo, 1, o0),
                     decode<FP8>(hi, 1, o1), b[4 * i], b[4 * i + 1]);
            mma<FP8>(d, decode<FP8>(lo, 2, o0), decode<FP8>(hi, 2, o1), decode<FP8>(lo, 3, o0),
                     decode<FP8>(hi, 3, o1), b[4 * i + 2], b[4 * i + 3]);
          }
          const float s0 = bf16_lo(sw[r]), s1 = bf16_hi(sw[r]);
          acc[r][0] = fmaf(d[0], s0 * sx[0], acc[r][0]);
          acc[r][1] = fmaf(d[1], s0 * sx[1], acc[r][1]);
          acc[r][2] = fmaf(d[2], s1 * sx[0], acc[r][2]);
          acc[r][3] = fmaf(d[3], s1 * sx[1], acc[r][3]);
        }
      }
    }
    // lane: packed rows 8 g + 2 r + h of columns 2 q + c in acc[r][2 h + c]
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      if (2 * q + c >= rows) continue;
      float y[8];
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        y[2 * r] = acc[r][c];
        y[2 * r + 1] = acc[r][2 + c];
      }
      __nv_bfloat16* o = p.out + int64_t(row0 + 2 * q + c) * p.N;
      if (p.gated) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int n = tile * 32 + 4 * g + i;
          if (n < p.N) o[n] = __float2bfloat16_rn(y[i] / (1.0f + expf(-y[i])) * y[i + 4]);
        }
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int n = tile * 64 + 8 * g + i;
          if (n < p.N) o[n] = __float2bfloat16_rn(y[i]);
        }
      }
    }
  }
}

// ---- packing ----------------------------------------------------------------------

// Row of W that packed row n of a tile holds, or -1 for padding.
__device__ __forceinline__ int source_row(int tile, int n, int N, bool gated) {
  if (!gated) {
    const int r = tile * 64 + n;
    return r < N ? r : -1;
  }
  const int half = N / 2, o = tile * 32 + (n >> 3) * 4 + (n & 3);
  return o < half ? ((n & 4) ? half + o : o) : -1;
}

__global__ void __launch_bounds__(256)
w4_pack_codes_kernel(int H, int N, int tiles, int blocks, bool gated, int64_t words,
                     const uint8_t* codes, uint32_t* packed) {
  pdl_wait();
  const int64_t step = int64_t(gridDim.x) * blockDim.x;
  for (int64_t at = int64_t(blockIdx.x) * blockDim.x + threadIdx.x; at < words; at += step) {
    const int i = int(at & 3), lane = int(at >> 2) & 31, piece = int(at >> 7) & 7;
    const int64_t unit = at >> 10;
    const int kb = int(unit % blocks);
    const int64_t et = unit / blocks;
    const int row = source_row(int(et % tiles), 8 * (lane >> 2) + piece, N, gated);
    const int k = kb * kBlockIn + 32 * i + 8 * (lane & 3);
    uint32_t word = 0x88888888u;
    if (row >= 0 && k < H) {   // H is a multiple of 32
      const uint8_t* src = codes + ((et / tiles) * N + row) * int64_t(H / 2) + k / 2;
      word = 0;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint32_t two = src[j];
        word |= (two & 15u) << (4 * j) | (two >> 4) << (4 * j + 16);
      }
    }
    packed[at] = word;
  }
}

__global__ void __launch_bounds__(256)
w4_pack_scales_kernel(int groups_in, int N, int tiles, int groups, bool gated, int64_t count,
                      const uint16_t* scales, const uint8_t* zeros, uint16_t* packed,
                      uint8_t* packed_zeros) {
  pdl_wait();
  const int64_t step = int64_t(gridDim.x) * blockDim.x;
  for (int64_t at = int64_t(blockIdx.x) * blockDim.x + threadIdx.x; at < count; at += step) {
    const int n = int(at & 63);
    const int64_t unit = at >> 6;
    const int s = int(unit % groups);
    const int64_t et = unit / groups;
    const int row = source_row(int(et % tiles), n, N, gated);
    const bool have = row >= 0 && s < groups_in;
    const int64_t src = ((et / tiles) * N + row) * groups_in + s;
    packed[at] = have ? scales[src] : uint16_t(0);
    if (packed_zeros != nullptr) packed_zeros[at] = have ? uint8_t(zeros[src] & 15u) : uint8_t(8);
  }
}

// ---- host ---------------------------------------------------------------------------

bool aligned(const void* p) { return p != nullptr && (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

bool w4_ok(const ep_w4_config* c) {
  if (c == nullptr) return false;
  if (c->num_experts < 1 || c->num_experts > 2048) return false;
  if (c->group_size != 32 && c->group_size != 64 && c->group_size != 128) return false;
  if (c->in_features < c->group_size || c->in_features > (1 << 20)) return false;
  if (c->in_features % c->group_size != 0) return false;
  if (c->out_features < 1 || c->out_features > (1 << 20)) return false;
  if (c->x_fp8 != 0 && c->x_fp8 != 1) return false;
  if (c->gated != 0 && c->gated != 1) return false;
  if (c->has_zeros != 0 && c->has_zeros != 1) return false;
  if (c->x_fp8 && c->in_features % kBlockIn != 0) return false;
  return !(c->gated && c->out_features % 2 != 0);
}

int w4_tiles(const ep_w4_config* c) {
  return c->gated ? (c->out_features / 2 + 31) / 32 : (c->out_features + 63) / 64;
}
int w4_blocks(const ep_w4_config* c) { return (c->in_features + kBlockIn - 1) / kBlockIn; }

// Scales (and zero points) of the packed form.
int64_t w4_scales(const ep_w4_config* c) {
  return int64_t(c->num_experts) * w4_tiles(c) * w4_blocks(c) * (kBlockIn / c->group_size) *
         kTileRows;
}

int32_t status(cudaError_t e) { return note_cuda(e) == cudaSuccess ? EP_OK : EP_ERR_CUDA; }

template <bool FP8, int GROUP, bool ZEROS>
cudaError_t launch_w4(const W4Params& p, int64_t items, cudaStream_t stream) {
  const int64_t want = (items + kW4Warps - 1) / kW4Warps;
  const int64_t most = int64_t(device_info().sm_count) * 2;
  const int grid = int(want < most ? want : most);
  return launch_pdl(expert_w4_kernel<FP8, GROUP, ZEROS>, dim3(grid), dim3(kW4Threads),
                    sizeof(int) * (p.E + 1), stream, p);
}

template <bool FP8, int GROUP>
cudaError_t launch_w4(const W4Params& p, int64_t items, cudaStream_t s) {
  return p.zeros != nullptr ? launch_w4<FP8, GROUP, true>(p, items, s)
                            : launch_w4<FP8, GROUP, false>(p, items, s);
}

template <bool FP8>
cudaError_t launch_w4(const W4Params& p, int group, int64_t items, cudaStream_t s) {
  if (group == 32) return launch_w4<FP8, 32>(p, items, s);
  if (group == 64) return launch_w4<FP8, 64>(p, items, s);
  return launch_w4<FP8, 128>(p, items, s);
}

}  // namespace
}  // namespace ep

using namespace ep;

extern "C" {

int64_t ep_w4_codes_bytes(const ep_w4_config* cfg) {
  if (!w4_ok(cfg)) return -1;
  return int64_t(cfg->num_experts) * w4_tiles(cfg) * w4_blocks(cfg) * kWordsPerBlock * 4;
}

int64_t ep_w4_scales_bytes(const ep_w4_config* cfg) {
  return w4_ok(cfg) ? w4_scales(cfg) * 2 : -1;
}

int64_t ep_w4_zeros_bytes(const ep_w4_config* cfg) {
  if (!w4_ok(cfg)) return -1;
  return cfg->has_zeros ? w4_scales(cfg) : 0;
}

int32_t ep_w4_pack(const ep_w4_config* cfg, const uint8_t* d_codes, const void* d_scales,
                   const uint8_t* d_zeros, void* d_packed_codes, void* d_packed_scales,
                   uint8_t* d_packed_zeros, void* stream) {
  if (!w4_ok(cfg)) return EP_ERR_INVALID_ARG;
  if (!aligned(d_codes) || !aligned(d_scales) || !aligned(d_packed_codes) ||
      !aligned(d_packed_scales))
    return EP_ERR_INVALID_ARG;
  if (cfg->has_zeros ? !aligned(d_zeros) || !aligned(d_packed_zeros)
                     : d_zeros != nullptr || d_packed_zeros != nullptr)
    return EP_ERR_INVALID_ARG;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const int tiles = w4_tiles(cfg), blocks = w4_blocks(cfg);
  const int64_t words = int64_t(cfg->num_experts) * tiles * blocks * kWordsPerBlock;
  const int64_t count = w4_scales(cfg);
  const int most = device_info().sm_count * 8;
  const auto grid = [&](int64_t n) { return dim3(unsigned(n / 256 + 1 < most ? n / 256 + 1 : most)); };
  cudaError_t e = launch_pdl(w4_pack_codes_kernel, grid(words), dim3(256), 0, s,
                             cfg->in_features, cfg->out_features, tiles, blocks, cfg->gated != 0,
                             words, d_codes, static_cast<uint32_t*>(d_packed_codes));
  if (e == cudaSuccess)
    e = launch_pdl(w4_pack_scales_kernel, grid(count), dim3(256), 0, s,
                   cfg->in_features / cfg->group_size, cfg->out_features, tiles,
                   blocks * (kBlockIn / cfg->group_size), cfg->gated != 0, count,
                   static_cast<const uint16_t*>(d_scales), d_zeros,
                   static_cast<uint16_t*>(d_packed_scales), d_packed_zeros);
  return status(e);
}

int32_t ep_expert_w4(const ep_w4_config* cfg, int32_t cap, int32_t num_rows, const void* d_x,
                     const float* d_x_scale, const void* d_codes, const void* d_scales,
                     const uint8_t* d_zeros, const int32_t* d_expert_start,
                     const int32_t* d_expert_end, void* d_out, void* stream) {
  if (!w4_ok(cfg) || cap < 0 || num_rows < 0) return EP_ERR_INVALID_ARG;
  if (!aligned(d_codes) || !aligned(d_scales) || !aligned(d_expert_start) ||
      !aligned(d_expert_end))
    return EP_ERR_INVALID_ARG;
  if (cfg->has_zeros ? !aligned(d_zeros) : d_zeros != nullptr) return EP_ERR_INVALID_ARG;
  if (cap > 0 && (!aligned(d_x) || !aligned(d_out))) return EP_ERR_INVALID_ARG;
  if (cfg->x_fp8 ? cap > 0 && !aligned(d_x_scale) : d_x_scale != nullptr)
    return EP_ERR_INVALID_ARG;
  if (cap == 0 || num_rows == 0) return EP_OK;
  W4Params p;
  p.E = cfg->num_experts;
  p.H = cfg->in_features;
  p.N = cfg->gated ? cfg->out_features / 2 : cfg->out_features;
  p.tiles = w4_tiles(cfg);
  p.blocks = w4_blocks(cfg);
  p.cap = cap;
  p.gated = cfg->gated != 0;
  p.x = d_x;
  p.x_scale = d_x_scale;
  p.codes = static_cast<const uint32_t*>(d_codes);
  p.scales = static_cast<const __nv_bfloat16*>(d_scales);
  p.zeros = d_zeros;
  p.start = d_expert_start;
  p.end = d_expert_end;
  p.out = static_cast<__nv_bfloat16*>(d_out);
  // an upper bound of the warps' items: an expert's last chunk may be short
  const int64_t chunks = int64_t(num_rows) / kChunk +
                         (num_rows < cfg->num_experts ? num_rows : cfg->num_experts);
  const int64_t items = chunks * p.tiles;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  return status(cfg->x_fp8 ? launch_w4<true>(p, cfg->group_size, items, s)
                           : launch_w4<false>(p, cfg->group_size, items, s));
}

}  // extern "C"

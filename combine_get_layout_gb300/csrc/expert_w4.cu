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

#include <atomic>
#include <cmath>

#include "../../include/ep.h"
#include "ep_device.cuh"
#include "ep_internal.h"

namespace ep {
namespace {

constexpr int kTileRows = 64;      // packed weight rows a tile
constexpr int kBlockIn = 128;      // inputs a block
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

// d = the same products with no sum before them.
template <bool FP8>
__device__ __forceinline__ void mma_first(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                          uint32_t a3, uint32_t b0, uint32_t b1) {
  if constexpr (FP8)
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%10,%10,%10,%10};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.0f));
  else
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%10,%10,%10,%10};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.0f));
}

// (v & mask) | bits in one instruction.
__device__ __forceinline__ uint32_t mask_or(uint32_t v, uint32_t mask, uint32_t bits) {
  uint32_t r;
  asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(r) : "r"(v), "r"(mask), "r"(bits));
  return r;
}

// A code becomes a 16-bit float without a conversion: its bits are the last
// integer bits of a mantissa whose exponent gives them weight 1.  bf16 (7
// mantissa bits) has one such place, bits 0-3 under 128; f16 (10) has bits
// 0-3 under 1024 and bits 4-7 under 64, which saves half the shifts.  The
// zero point and that offset then come off in one exact subtraction.
template <bool FP8>
__device__ __forceinline__ void decode(uint32_t word, uint32_t even, uint32_t odd,
                                       uint32_t (&pairs)[4]) {
  if constexpr (FP8) {
    const uint32_t high = word >> 8;
    pairs[0] = mask_or(word, 0x000F000Fu, 0x64006400u);
    pairs[1] = mask_or(word, 0x00F000F0u, 0x54005400u);
    pairs[2] = mask_or(high, 0x000F000Fu, 0x64006400u);
    pairs[3] = mask_or(high, 0x00F000F0u, 0x54005400u);
#pragma unroll
    for (int j = 0; j < 4; ++j)
      asm("sub.f16x2 %0, %0, %1;" : "+r"(pairs[j]) : "r"(j & 1 ? odd : even));
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      pairs[j] = mask_or(word >> (4 * j), 0x000F000Fu, 0x43004300u);
      asm("sub.bf16x2 %0, %0, %1;" : "+r"(pairs[j]) : "r"(even));
    }
  }
}

// What decode takes off the even and odd pairs of the row whose zero point
// (under 16) is byte i of z: pairs of 1024 + z and 64 + z in f16, of 128 + z
// in bf16.  One byte permutation puts the zero point and the offset's upper
// byte in both halves.
template <bool FP8>
__device__ __forceinline__ void offsets(uint32_t z, int i, uint32_t* even, uint32_t* odd) {
  *even = __byte_perm(z, FP8 ? 0x64646464u : 0x43434343u, 0x4040u + 0x0101u * i);
  *odd = __byte_perm(z << 4, 0x54545454u, 0x4040u + 0x0101u * i);
}

// Two E4M3 values as an f16 pair (exact).
__device__ __forceinline__ uint32_t e4m3_pair(uint32_t two) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(uint16_t(two)));
  return r;
}

// ---- the product ----------------------------------------------------------------

// A warp's stage in shared memory: one block (128 inputs) of its tile and
// chunk.  x rows are swizzled in units of the fragments' reads, so that the
// eight lanes (FP8: sixteen) of one shared-memory pass meet different banks.
template <bool FP8, int GROUP, bool ZEROS, int NT>
struct Stage {
  static constexpr int kGroups = kBlockIn / GROUP;
  static constexpr int kRowBytes = FP8 ? 128 : 256;
  static constexpr int kX = kTileRows * kBlockIn / 2;              // after the codes
  static constexpr int kScales = kX + 8 * NT * kRowBytes;
  static constexpr int kZeros = kScales + kGroups * kTileRows * 2;
  static constexpr int kXScale = kZeros + (ZEROS ? kGroups * kTileRows : 0);
  static constexpr int kBytes = kXScale + (FP8 ? 8 * NT * 4 : 0);
  static_assert(kBytes % 16 == 0);

  // Byte offset of 16-byte piece c of row t of x.
  static __device__ __forceinline__ int x_piece(int t, int c) {
    if constexpr (FP8) return kX + t * 128 + ((((c >> 1) ^ (t & 3)) << 1) | (c & 1)) * 16;
    return kX + t * 256 + (c ^ ((t & 1) << 2)) * 16;
  }
};

// Global -> shared, asynchronously.
template <int BYTES>
__device__ __forceinline__ void cp_async(uint32_t dst, const void* src) {
  if constexpr (BYTES == 16)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ uint4 lds16(uint32_t at) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(at));
  return v;
}
__device__ __forceinline__ uint2 lds8(uint32_t at) {
  uint2 v;
  asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(at));
  return v;
}
__device__ __forceinline__ uint32_t lds4(uint32_t at) {
  uint32_t v;
  asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(at));
  return v;
}

__device__ __forceinline__ uint32_t word_of(const uint4& v, int i) {
  return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w;
}

// Chunks of kRows rows before each expert, in shared memory: pre[e] of e's
// predecessors, pre[E] of all.  Every thread takes a run of experts, so that
// up to blockDim.x experts need one pass and two barriers.
template <int kRows>
__device__ void count_chunks(const W4Params& p, int* pre) {
  __shared__ int warp_sum[32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  const int each = (p.E + blockDim.x - 1) / blockDim.x;
  const int e0 = min(p.E, int(threadIdx.x) * each), e1 = min(p.E, e0 + each);
  int mine = 0;
  for (int e = e0; e < e1; ++e) {
    const int lo = max(0, p.start[e]), hi = min(p.cap, p.end[e]);
    const int n = hi > lo ? (hi - lo + kRows - 1) / kRows : 0;
    pre[e] = n;
    mine += n;
  }
  int sum = mine;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int up = __shfl_up_sync(0xffffffffu, sum, d);
    if (lane >= d) sum += up;
  }
  if (lane == 31) warp_sum[warp] = sum;
  __syncthreads();
  int before = sum - mine;
  for (int v = 0; v < warp; ++v) before += warp_sum[v];
  if (threadIdx.x == blockDim.x - 1) pre[p.E] = before + mine;
  for (int e = e0; e < e1; ++e) {
    const int n = pre[e];
    pre[e] = before;
    before += n;
  }
  __syncthreads();
}

// The expert whose chunks hold chunk c, by a whole warp: 32 experts' ends a
// round, so that two rounds serve a thousand experts.
__device__ __forceinline__ int expert_of(const int* pre, int E, int c, int lane) {
  int lo = 0, n = E - 1;      // the answer is among lo .. lo + n
  while (n > 0) {
    const int step = (n >> 5) + 1, i = lane * step;
    const bool past = i + step - 1 >= n || pre[lo + i + step] > c;
    const int skip = __ffs(__ballot_sync(0xffffffffu, past)) - 1;      // the last lane answers
    lo += skip * step;
    n = min(step - 1, n - skip * step);
  }
  return lo;
}

// Steps through (chunk, tile) items, tiles first, `stride` items at a time.
struct Walk {
  int chunk, tile, chunks, skip_chunks, skip_tiles;
  __device__ __forceinline__ Walk(const W4Params& p, int first, int stride, int total)
      : chunk(first / p.tiles), tile(first % p.tiles), chunks(total),
        skip_chunks(stride / p.tiles), skip_tiles(stride % p.tiles) {}
  __device__ __forceinline__ bool done() const { return chunk >= chunks; }
  __device__ __forceinline__ void advance(const W4Params& p) {
    chunk += skip_chunks;
    tile += skip_tiles;
    if (tile >= p.tiles) {
      tile -= p.tiles;
      ++chunk;
    }
  }
};

// A tile of 64 packed weight rows by a chunk of up to kRows rows of x.
struct Item {
  int expert, tile, row0, rows;
  template <int kRows>
  __device__ __forceinline__ void find(const W4Params& p, const int* pre, const Walk& at, int lane) {
    tile = at.tile;
    expert = expert_of(pre, p.E, at.chunk, lane);
    row0 = max(0, p.start[expert]) + (at.chunk - pre[expert]) * kRows;
    rows = min(kRows, min(p.cap, p.end[expert]) - row0);
  }
};

// A lane's share of the copies of an item's units, one unit after another.
// Columns past the item's rows and inputs past H are not copied: what a
// stage holds there meets only columns that are not stored, and is skipped.
template <bool FP8, int GROUP, bool ZEROS, int NT>
struct Loader {
  using St = Stage<FP8, GROUP, ZEROS, NT>;
  const char *codes, *scales, *x, *x_scale, *zeros;
  int rows;      // left of the lane's first row
  int k;         // first input of the lane's pieces of x
  int kb;

  __device__ __forceinline__ void start(const W4Params& p, const Item& it, int slice, int lane) {
    const int64_t unit = (int64_t(it.expert) * p.tiles + it.tile) * p.blocks + slice;
    codes = reinterpret_cast<const char*>(p.codes) + unit * 4096 + lane * 16;
    scales = reinterpret_cast<const char*>(p.scales) + unit * (St::kGroups * kTileRows * 2) + lane * 16;
    if constexpr (ZEROS)
      zeros = reinterpret_cast<const char*>(p.zeros) + unit * (St::kGroups * kTileRows) + lane * 16;
    const int t = FP8 ? lane >> 3 : lane >> 4, c = FP8 ? lane & 7 : lane & 15;
    rows = it.rows - t;
    k = slice * kBlockIn + c * (FP8 ? 16 : 8);
    x = static_cast<const char*>(p.x) + (int64_t(it.row0 + t) * p.H + k) * (FP8 ? 1 : 2);
    if constexpr (FP8)
      x_scale = reinterpret_cast<const char*>(p.x_scale + int64_t(it.row0 + lane) * p.blocks + slice);
    kb = slice;
  }

  __device__ __forceinline__ void copy(const W4Params& p, uint32_t stage, int lane, int split) {
#pragma unroll
    for (int i = 0; i < 8; ++i) cp_async<16>(stage + i * 512 + lane * 16, codes + i * 512);
    codes += split * 4096;
    if constexpr (FP8) {
      const int t = lane >> 3, c = lane & 7;
#pragma unroll
      for (int i = 0; i < 2 * NT; ++i)
        if (4 * i < rows) cp_async<16>(stage + St::x_piece(4 * i + t, c), x + int64_t(4 * i) * p.H);
      if (lane < 8 * NT && lane < rows + t) cp_async<4>(stage + St::kXScale + lane * 4, x_scale);
      x += split * kBlockIn;
      x_scale += split * 4;
    } else {
      const int t = lane >> 4, c = lane & 15;
#pragma unroll
      for (int i = 0; i < 4 * NT; ++i)
        if (2 * i < rows && k < p.H)
          cp_async<16>(stage + St::x_piece(2 * i + t, c), x + int64_t(4 * i) * p.H);
      x += split * kBlockIn * 2;
      k += split * kBlockIn;
    }
    if (lane < St::kGroups * 8) cp_async<16>(stage + St::kScales + lane * 16, scales);
    scales += split * (St::kGroups * kTileRows * 2);
    if constexpr (ZEROS) {
      if (lane < St::kGroups * 4) cp_async<16>(stage + St::kZeros + lane * 16, zeros);
      zeros += split * (St::kGroups * kTileRows);
    }
    kb += split;
  }
};

// acc += the unit in a stage.  Lane (g = lane / 4, q = lane % 4) holds packed
// rows 8 g .. 8 g + 7 (piece 2 r + h is row g + 8 h of the r-th 16-row
// operand) and columns 8 t + 2 q, + 1: acc[t][r][2 h + c].
template <bool FP8, int GROUP, bool ZEROS, int NT>
__device__ __forceinline__ void multiply_unit(uint32_t stage, int lane, int tiles_used, int inputs,
                                              float (&acc)[NT][4][4]) {
  using St = Stage<FP8, GROUP, ZEROS, NT>;
  constexpr int kWords = GROUP / 32;              // words of a lane a group
  const int g = lane >> 2, q = lane & 3;
  uint4 w[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) w[i] = lds16(stage + i * 512 + lane * 16);
  float sx[NT][2];
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    sx[t][0] = sx[t][1] = 1.0f;
    if constexpr (FP8) {
      const uint2 v = lds8(stage + St::kXScale + (8 * t + 2 * q) * 4);
      sx[t][0] = __uint_as_float(v.x);
      sx[t][1] = __uint_as_float(v.y);
    }
  }
#pragma unroll
  for (int s = 0; s < St::kGroups; ++s) {
    const uint4 sv = lds16(stage + St::kScales + s * 128 + g * 16);
    uint2 zv;
    if constexpr (ZEROS) zv = lds8(stage + St::kZeros + s * 64 + g * 8);
    if (!FP8 && 32 * kWords * s >= inputs) break;      // groups past H
    uint32_t even[8], odd[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      even[i] = FP8 ? 0x64086408u : 0x43084308u;      // 1032, 136
      odd[i] = 0x54805480u;                           // 72
      if constexpr (ZEROS) offsets<FP8>(i < 4 ? zv.x : zv.y, i & 3, &even[i], &odd[i]);
    }
    float d[NT][4][4];
#pragma unroll
    for (int i = s * kWords; i < (s + 1) * kWords; ++i) {
      uint32_t b[NT][4];
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        if (NT > 1 && t >= tiles_used) continue;
        if constexpr (FP8) {
          const uint2 v = lds8(stage + St::x_piece(8 * t + g, 2 * i + (q >> 1)) + (q & 1) * 8);
          b[t][0] = e4m3_pair(v.x);
          b[t][1] = e4m3_pair(v.x >> 16);
          b[t][2] = e4m3_pair(v.y);
          b[t][3] = e4m3_pair(v.y >> 16);
        } else {
          const uint4 v = lds16(stage + St::x_piece(8 * t + g, 4 * i + q));
          b[t][0] = v.x;
          b[t][1] = v.y;
          b[t][2] = v.z;
          b[t][3] = v.w;
        }
      }
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        uint32_t lo[4], hi[4];
        decode<FP8>(word_of(w[2 * r], i), even[2 * r], odd[2 * r], lo);
        decode<FP8>(word_of(w[2 * r + 1], i), even[2 * r + 1], odd[2 * r + 1], hi);
#pragma unroll
        for (int t = 0; t < NT; ++t) {
          if (NT > 1 && t >= tiles_used) continue;
          if (i == s * kWords)
            mma_first<FP8>(d[t][r], lo[0], hi[0], lo[1], hi[1], b[t][0], b[t][1]);
          else
            mma<FP8>(d[t][r], lo[0], hi[0], lo[1], hi[1], b[t][0], b[t][1]);
          mma<FP8>(d[t][r], lo[2], hi[2], lo[3], hi[3], b[t][2], b[t][3]);
        }
      }
    }
    const uint32_t sw[4] = {sv.x, sv.y, sv.z, sv.w};
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const float s0 = bf16_lo(sw[r]), s1 = bf16_hi(sw[r]);
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        if (NT > 1 && t >= tiles_used) continue;
        acc[t][r][0] = fmaf(d[t][r][0], FP8 ? s0 * sx[t][0] : s0, acc[t][r][0]);
        acc[t][r][1] = fmaf(d[t][r][1], FP8 ? s0 * sx[t][1] : s0, acc[t][r][1]);
        acc[t][r][2] = fmaf(d[t][r][2], FP8 ? s1 * sx[t][0] : s1, acc[t][r][2]);
        acc[t][r][3] = fmaf(d[t][r][3], FP8 ? s1 * sx[t][1] : s1, acc[t][r][3]);
      }
    }
  }
}

// Writes packed rows p and p + 4 (0 <= p < 4) of the lane's eight, column
// `col` of the item.
__device__ __forceinline__ void store_pair(const W4Params& p, const Item& it, int g, int i, int col,
                                           float lo, float hi) {
  if (col >= it.rows) return;
  __nv_bfloat16* o = p.out + int64_t(it.row0 + col) * p.N;
  if (p.gated) {
    const int n = it.tile * 32 + 4 * g + i;
    if (n < p.N) o[n] = __float2bfloat16_rn(lo / (1.0f + expf(-lo)) * hi);
  } else {
    const int n = it.tile * 64 + 8 * g + i;
    if (n < p.N) o[n] = __float2bfloat16_rn(lo);
    if (n + 4 < p.N) o[n + 4] = __float2bfloat16_rn(hi);
  }
}

// WARPS warps a CTA in groups of `split`: a group shares an item, warp j of
// it taking the blocks j, j + split, ...; the warps of a group add up their
// sums in shared memory.  Each warp keeps STAGES units on their way in
// shared memory of its own (cp.async, so no barrier and no flag).
template <bool FP8, int GROUP, bool ZEROS, int NT, int WARPS, int STAGES>
__global__ void __launch_bounds__(WARPS * 32) expert_w4_kernel(W4Params p, int split) {
  using St = Stage<FP8, GROUP, ZEROS, NT>;
  static_assert(St::kBytes >= NT * 2048, "a stage holds a warp's sums");
  extern __shared__ __align__(16) char smem[];
  int* const pre = reinterpret_cast<int*>(smem + WARPS * STAGES * St::kBytes);
  __shared__ uint32_t sums_at[WARPS];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const uint32_t base = smem_addr(smem) + warp * (STAGES * St::kBytes);
  pdl_wait();
  count_chunks<8 * NT>(p, pre);
  // groups are numbered across the CTAs first: a last partial round of items
  // then spreads over all SMs
  const int group = warp / split, slice = warp % split;
  Walk now(p, group * gridDim.x + blockIdx.x, gridDim.x * (WARPS / split), pre[p.E]);
  Walk ahead = now;      // the item of the unit to load next
  Loader<FP8, GROUP, ZEROS, NT> loader;
  loader.kb = p.blocks;
  const auto enter = [&] {
    Item next;
    next.find<8 * NT>(p, pre, ahead, lane);
    loader.start(p, next, slice, lane);
  };
  if (!ahead.done()) enter();
  const auto load_next = [&](uint32_t stage) {
    if (loader.kb < p.blocks) {
      loader.copy(p, stage, lane, split);
      if (loader.kb >= p.blocks) {
        ahead.advance(p);
        if (!ahead.done()) enter();
      }
    }
    cp_async_commit();
  };
#pragma unroll
  for (int i = 0; i < STAGES - 1; ++i) load_next(base + i * St::kBytes);

  uint32_t stage = base, idle = base + (STAGES - 1) * St::kBytes;
  for (; !now.done(); now.advance(p)) {
    Item it;
    it.find<8 * NT>(p, pre, now, lane);
    const int used = (it.rows + 7) >> 3;
    float acc[NT][4][4];
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int r = 0; r < 4; ++r)
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[t][r][i] = 0.0f;
    for (int kb = slice; kb < p.blocks; kb += split) {
      cp_async_wait<STAGES - 2>();
      __syncwarp();      // the unit is there, and the idle stage was read by all
      load_next(idle);
      multiply_unit<FP8, GROUP, ZEROS, NT>(stage, lane, used, p.H - kb * kBlockIn, acc);
      idle = stage;
      stage = stage == base + (STAGES - 1) * St::kBytes ? base : stage + St::kBytes;
    }
    const int g = lane >> 2, q = lane & 3;
    if (split == 1) {
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int c = 0; c < 2; ++c)
#pragma unroll
          for (int i = 0; i < 4; ++i)
            store_pair(p, it, g, i, 8 * t + 2 * q + c, acc[t][i >> 1][2 * (i & 1) + c],
                       acc[t][2 + (i >> 1)][2 * (i & 1) + c]);
      continue;
    }
    // pair (t, i, c) of a warp at [2 (8 t + 2 i + c) + half][lane] of its idle stage
    __syncwarp();
    char* const mine = smem + (idle - smem_addr(smem)) + lane * 4;
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          float* const at = reinterpret_cast<float*>(mine + (8 * t + 2 * i + c) * 256);
          at[0] = acc[t][i >> 1][2 * (i & 1) + c];
          at[32] = acc[t][2 + (i >> 1)][2 * (i & 1) + c];
        }
    if (lane == 0) sums_at[warp] = idle - smem_addr(smem);
    asm volatile("bar.sync %0, %1;" ::"r"(1 + group), "r"(32 * split) : "memory");
    for (int pair = slice; pair < 8 * used; pair += split) {
      float lo = 0.0f, hi = 0.0f;
      const char* const from = smem + pair * 256 + lane * 4;
#pragma unroll 4
      for (int v = 0; v < split; ++v) {
        const float* const at = reinterpret_cast<const float*>(from + sums_at[group * split + v]);
        lo += at[0];
        hi += at[32];
      }
      store_pair(p, it, g, (pair & 7) >> 1, 8 * (pair >> 3) + 2 * q + (pair & 1), lo, hi);
    }
    asm volatile("bar.sync %0, %1;" ::"r"(1 + group), "r"(32 * split) : "memory");
  }
  cp_async_wait<0>();
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

// Dynamic shared memory of a CTA at most (227 KiB less its static arrays), and
// what the table of chunks of 2048 experts leaves of it for the stages.
constexpr int kSmemLimit = 227 * 1024 - 256;
constexpr int kSmemBudget = kSmemLimit - 2049 * 4;

// Chunks of `size` rows that `rows` rows of E experts make, on average.
double expected_chunks(int rows, int E, int size) {
  const double active = E * (1.0 - pow(1.0 - 1.0 / E, rows));
  const double full = double(rows) / size + 0.5 * active;
  return active > full ? active : full;
}

template <bool FP8, int GROUP, bool ZEROS>
cudaError_t launch_w4(const W4Params& p, int num_rows, cudaStream_t stream) {
  constexpr int NT = 1, WARPS = 16;
  constexpr int STAGES = kSmemBudget / (WARPS * Stage<FP8, GROUP, ZEROS, NT>::kBytes);
  static_assert(STAGES >= 2);
  const double items = expected_chunks(num_rows, p.E, 8 * NT) * p.tiles;
  const int sms = device_info().sm_count;
  // Units one warp works through: rounds of items times its blocks of each,
  // and about one unit's time to add up a group's sums.
  int split = 1;
  double least = 0.0;
  for (int s = 1; s <= WARPS; s *= 2) {
    const double cost = ceil(items * s / (double(sms) * WARPS)) *
                        ((p.blocks + s - 1) / s + (s > 1 ? 1.0 : 0.0));
    if (s == 1 || cost < least) {
      split = s;
      least = cost;
    }
  }
  // an upper bound of the items: an expert's last chunk may be short
  const int64_t chunks = int64_t(num_rows) / (8 * NT) + (num_rows < p.E ? num_rows : p.E);
  const int64_t want = (chunks * p.tiles + WARPS / split - 1) / (WARPS / split);
  const int grid = int(want < sms ? want : sms);
  const size_t smem = WARPS * STAGES * Stage<FP8, GROUP, ZEROS, NT>::kBytes + sizeof(int) * (p.E + 1);
  auto* kernel = expert_w4_kernel<FP8, GROUP, ZEROS, NT, WARPS, STAGES>;
  // once per kernel and device: the limit for any number of experts
  static std::atomic<uint64_t> raised{0};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev >= 64 || !(raised.load(std::memory_order_acquire) >> dev & 1)) {
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemLimit);
    if (e != cudaSuccess) return e;
    if (dev < 64) raised.fetch_or(uint64_t(1) << dev, std::memory_order_release);
  }
  return launch_pdl(kernel, dim3(grid), dim3(WARPS * 32), smem, stream, p, split);
}

template <bool FP8, int GROUP>
cudaError_t launch_w4(const W4Params& p, int num_rows, cudaStream_t s) {
  return p.zeros != nullptr ? launch_w4<FP8, GROUP, true>(p, num_rows, s)
                            : launch_w4<FP8, GROUP, false>(p, num_rows, s);
}

template <bool FP8>
cudaError_t launch_w4(const W4Params& p, int group, int num_rows, cudaStream_t s) {
  if (group == 32) return launch_w4<FP8, 32>(p, num_rows, s);
  if (group == 64) return launch_w4<FP8, 64>(p, num_rows, s);
  return launch_w4<FP8, 128>(p, num_rows, s);
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
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  return status(cfg->x_fp8 ? launch_w4<true>(p, cfg->group_size, num_rows, s)
                           : launch_w4<false>(p, cfg->group_size, num_rows, s));
}

}  // extern "C"

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

// How a kernel takes its columns: NT tiles of eight rows of x, staged with the
// codes or read straight into registers (DIRECT).
template <bool FP8_, int GROUP_, bool ZEROS_, int NT_, bool DIRECT_>
struct Kind {
  static constexpr bool FP8 = FP8_, ZEROS = ZEROS_, DIRECT = DIRECT_;
  static constexpr int GROUP = GROUP_, NT = NT_;
  static constexpr int kChunk = 8 * NT;                      // rows of an item at most
  static constexpr int kGroups = kBlockIn / GROUP;           // scale groups a block
  static constexpr int kWords = GROUP / 32;                  // words of a lane a group

  // A warp's stage in shared memory: one unit, a block (128 inputs) of its
  // tile and chunk.  x rows are swizzled in units of the fragments' reads, so
  // that the eight lanes (FP8: sixteen) of one shared-memory pass meet
  // different banks.
  static constexpr int kRowBytes = FP8 ? 128 : 256;
  static constexpr int kX = kTileRows * kBlockIn / 2;        // after the codes
  static constexpr int kScales = kX + (DIRECT ? 0 : kChunk * kRowBytes);
  static constexpr int kZeros = kScales + kGroups * kTileRows * 2;
  static constexpr int kXScale = kZeros + (ZEROS ? kGroups * kTileRows : 0);
  static constexpr int kBytes = kXScale + (FP8 && !DIRECT ? kChunk * 4 : 0);
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
__device__ __forceinline__ uint32_t lds2(uint32_t at) {
  uint16_t v;
  asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(at));
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

// Chunks of kRows rows that rows lo .. hi - 1 make, for any 0 <= lo, hi < 2^31.
template <int kRows>
__host__ __device__ constexpr int chunks_of(int lo, int hi) {
  return hi > lo ? int((unsigned(hi) - unsigned(lo) + (kRows - 1)) / kRows) : 0;
}
static_assert(chunks_of<8>(0, 0x7fffffff) == 1 << 28 && chunks_of<16>(5, 0x7fffffff) == 1 << 27);
static_assert(chunks_of<8>(3, 3) == 0 && chunks_of<8>(4, 3) == 0 && chunks_of<8>(0, 1) == 1 &&
              chunks_of<8>(1, 9) == 1 && chunks_of<8>(1, 10) == 2);

// Chunks of kRows rows before each expert, in shared memory: pre[e] of e's
// predecessors, pre[E] of all.  Every thread takes a run of experts, so that
// up to blockDim.x experts need one pass and two barriers.
template <int kRows>
__device__ void count_chunks(const W4Params& p, int* pre) {
  __shared__ int warp_sum[32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int each = (p.E + blockDim.x - 1) / blockDim.x;
  const int e0 = min(p.E, int(threadIdx.x) * each), e1 = min(p.E, e0 + each);
  int mine = 0;
  for (int e = e0; e < e1; ++e) {
    const int lo = max(0, p.start[e]), hi = min(p.cap, p.end[e]);
    const int n = chunks_of<kRows>(lo, hi);
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

// The same for up to 32 experts, an expert a lane: every warp counts for
// itself and writes the same values, so that none waits for another (one row
// of one matrix: 5.3 -> 4.8 us).
template <int kRows>
__device__ __forceinline__ void count_few_chunks(const W4Params& p, int* pre, int lane) {
  int n = 0;
  if (lane < p.E) {
    const int lo = max(0, p.start[lane]), hi = min(p.cap, p.end[lane]);
    n = chunks_of<kRows>(lo, hi);
  }
  int end = n;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int up = __shfl_up_sync(0xffffffffu, end, d);
    if (lane >= d) end += up;
  }
  if (lane < p.E) pre[lane + 1] = end;
  if (lane == 0) pre[0] = 0;
  __syncwarp();
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
};

// Of a chunk below the total, by a whole warp.
template <int kRows>
__device__ __forceinline__ Item item_at(const W4Params& p, const int* pre, const Walk& at, int lane) {
  const int e = expert_of(pre, p.E, at.chunk, lane);
  const int row0 = max(0, p.start[e]) + (at.chunk - pre[e]) * kRows;
  return {e, at.tile, row0, min(kRows, min(p.cap, p.end[e]) - row0)};
}

// A lane's share of the copies of an item's units, one unit after another.
// Columns past the item's rows and inputs past H are not copied: what a
// stage holds there meets only columns that are not stored, and is skipped.
template <class Kd>
struct Loader {
  const char *codes, *scales, *x, *x_scale, *zeros;
  int rows;      // left of the lane's first row
  int k;         // first input of the lane's pieces of x
  int kb;

  __device__ __forceinline__ void start(const W4Params& p, const Item& it, int slice, int lane) {
    const int64_t unit = (int64_t(it.expert) * p.tiles + it.tile) * p.blocks + slice;
    codes = reinterpret_cast<const char*>(p.codes) + unit * 4096 + lane * 16;
    scales = reinterpret_cast<const char*>(p.scales) + unit * (Kd::kGroups * kTileRows * 2) + lane * 16;
    if constexpr (Kd::ZEROS)
      zeros = reinterpret_cast<const char*>(p.zeros) + unit * (Kd::kGroups * kTileRows) + lane * 16;
    if constexpr (!Kd::DIRECT) {
      const int t = Kd::FP8 ? lane >> 3 : lane >> 4, c = Kd::FP8 ? lane & 7 : lane & 15;
      rows = it.rows - t;
      k = slice * kBlockIn + c * (Kd::FP8 ? 16 : 8);
      x = static_cast<const char*>(p.x) + (int64_t(unsigned(it.row0) + t) * p.H + k) * (Kd::FP8 ? 1 : 2);
      if constexpr (Kd::FP8)
        x_scale =
            reinterpret_cast<const char*>(p.x_scale + int64_t(unsigned(it.row0) + lane) * p.blocks + slice);
    }
    kb = slice;
  }

  __device__ __forceinline__ void copy(const W4Params& p, uint32_t stage, int lane, int split) {
#pragma unroll
    for (int i = 0; i < 8; ++i) cp_async<16>(stage + i * 512 + lane * 16, codes + i * 512);
    codes += split * 4096;
    if constexpr (Kd::DIRECT) {
      // the columns go another way
    } else if constexpr (Kd::FP8) {
      const int t = lane >> 3, c = lane & 7;
#pragma unroll
      for (int i = 0; i < 2 * Kd::NT; ++i)
        if (4 * i < rows) cp_async<16>(stage + Kd::x_piece(4 * i + t, c), x + int64_t(4 * i) * p.H);
      if (lane < Kd::kChunk && lane < rows + t) cp_async<4>(stage + Kd::kXScale + lane * 4, x_scale);
      x += split * kBlockIn;
      x_scale += split * 4;
    } else {
      const int t = lane >> 4, c = lane & 15;
#pragma unroll
      for (int i = 0; i < 4 * Kd::NT; ++i)
        if (2 * i < rows && k < p.H)
          cp_async<16>(stage + Kd::x_piece(2 * i + t, c), x + int64_t(4 * i) * p.H);
      x += split * kBlockIn * 2;
      k += split * kBlockIn;
    }
    if (lane < Kd::kGroups * 8) cp_async<16>(stage + Kd::kScales + lane * 16, scales);
    scales += split * (Kd::kGroups * kTileRows * 2);
    if constexpr (Kd::ZEROS) {
      if (lane < Kd::kGroups * 4) cp_async<16>(stage + Kd::kZeros + lane * 16, zeros);
      zeros += split * (Kd::kGroups * kTileRows);
    }
    kb += split;
  }
};

// The columns of the product: lane (g, q) multiplies with inputs 32 i + 8 q
// .. + 7 (word i) of rows 8 t + g.  DIRECT (bf16) reads a unit's words into
// registers through L1, where the warps of an SM that work on other tiles of
// the same rows find them.
template <class Kd>
struct Columns {
  static_assert(!(Kd::DIRECT && Kd::FP8), "E4M3 rows are staged");
  uint4 v[Kd::DIRECT ? Kd::NT : 1][4];
  const char* x[Kd::NT];

  __device__ __forceinline__ void start(const W4Params& p, const Item& it, int slice, int lane) {
    if constexpr (Kd::DIRECT) {
      // a row past the item's reads its last one: nothing of it is stored
#pragma unroll
      for (int t = 0; t < Kd::NT; ++t)
        x[t] = static_cast<const char*>(p.x) +
               (int64_t(it.row0 + min(8 * t + (lane >> 2), it.rows - 1)) * p.H +
                slice * kBlockIn + 8 * (lane & 3)) * 2;
    }
  }

  // The next unit's, of which `inputs` lie before H; moves on by `split`.
  template <int USED>
  __device__ __forceinline__ void load(int inputs, int split) {
    if constexpr (Kd::DIRECT) {
#pragma unroll
      for (int t = 0; t < USED; ++t) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (32 * i < inputs) v[t][i] = __ldg(reinterpret_cast<const uint4*>(x[t] + 64 * i));
        x[t] += split * kBlockIn * 2;
      }
    }
  }

  // Word i as four 16-bit float pairs, inputs 2 j and 2 j + 1 in pair j.
  __device__ __forceinline__ void word(uint32_t stage, int lane, int t, int i,
                                       uint32_t (&b)[4]) const {
    const int g = lane >> 2, q = lane & 3;
    if constexpr (Kd::FP8) {
      const uint2 w = lds8(stage + Kd::x_piece(8 * t + g, 2 * i + (q >> 1)) + (q & 1) * 8);
      b[0] = e4m3_pair(w.x);
      b[1] = e4m3_pair(w.x >> 16);
      b[2] = e4m3_pair(w.y);
      b[3] = e4m3_pair(w.y >> 16);
    } else {
      uint4 w;
      if constexpr (Kd::DIRECT)
        w = v[t][i];
      else
        w = lds16(stage + Kd::x_piece(8 * t + g, 4 * i + q));
      b[0] = w.x;
      b[1] = w.y;
      b[2] = w.z;
      b[3] = w.w;
    }
  }

  // The scales of columns 8 t + 2 q and + 1.
  static __device__ __forceinline__ float2 scale(uint32_t stage, int lane, int t) {
    if constexpr (Kd::FP8) {
      const uint2 s = lds8(stage + Kd::kXScale + (8 * t + 2 * (lane & 3)) * 4);
      return make_float2(__uint_as_float(s.x), __uint_as_float(s.y));
    }
    return make_float2(1.0f, 1.0f);
  }
};

// acc += a group's sums d, rows scaled by the bf16 pair sw, columns by sx.
template <class Kd>
__device__ __forceinline__ void add_group(float (&acc)[4], const float (&d)[4], uint32_t sw,
                                          float2 sx) {
  const float s0 = bf16_lo(sw), s1 = bf16_hi(sw);
  acc[0] = fmaf(d[0], Kd::FP8 ? s0 * sx.x : s0, acc[0]);
  acc[1] = fmaf(d[1], Kd::FP8 ? s0 * sx.y : s0, acc[1]);
  acc[2] = fmaf(d[2], Kd::FP8 ? s1 * sx.x : s1, acc[2]);
  acc[3] = fmaf(d[3], Kd::FP8 ? s1 * sx.y : s1, acc[3]);
}

// d (+)= word i of weight rows lo, hi by the columns' b.
template <class Kd>
__device__ __forceinline__ void multiply_word(float (&d)[4], bool first, const uint32_t (&lo)[4],
                                              const uint32_t (&hi)[4], const uint32_t (&b)[4]) {
  if (first)
    mma_first<Kd::FP8>(d, lo[0], hi[0], lo[1], hi[1], b[0], b[1]);
  else
    mma<Kd::FP8>(d, lo[0], hi[0], lo[1], hi[1], b[0], b[1]);
  mma<Kd::FP8>(d, lo[2], hi[2], lo[3], hi[3], b[2], b[3]);
}

// What a code without a zero point carries, as decode() wants it.
template <bool FP8>
constexpr uint32_t kEven = FP8 ? 0x64086408u : 0x43084308u;      // 1024 + 8, 128 + 8
constexpr uint32_t kOdd = 0x54805480u;                           // 64 + 8

// acc += the unit in a stage, one column tile.  Lane (g = lane / 4, q = lane
// % 4) holds packed rows 8 g .. 8 g + 7 (piece 2 r + h is row g + 8 h of the
// r-th 16-row operand) and columns 2 q, 2 q + 1: acc[r][2 h + c].  The four
// operands' chains of sums run side by side.
template <class Kd>
__device__ __forceinline__ void multiply_one(uint32_t stage, int lane, int inputs,
                                             const Columns<Kd>& cols, float (&acc)[4][4]) {
  const int g = lane >> 2;
  uint4 w[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) w[i] = lds16(stage + i * 512 + lane * 16);
  const float2 sx = Columns<Kd>::scale(stage, lane, 0);
#pragma unroll
  for (int s = 0; s < Kd::kGroups; ++s) {
    if (!Kd::FP8 && Kd::GROUP * s >= inputs) break;      // groups past H
    const uint4 sv = lds16(stage + Kd::kScales + s * 128 + g * 16);
    uint2 zv;
    if constexpr (Kd::ZEROS) zv = lds8(stage + Kd::kZeros + s * 64 + g * 8);
    uint32_t even[8], odd[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      even[i] = kEven<Kd::FP8>;
      odd[i] = kOdd;
      if constexpr (Kd::ZEROS) offsets<Kd::FP8>(i < 4 ? zv.x : zv.y, i & 3, &even[i], &odd[i]);
    }
    float d[4][4];
#pragma unroll
    for (int i = s * Kd::kWords; i < (s + 1) * Kd::kWords; ++i) {
      uint32_t b[4];
      cols.word(stage, lane, 0, i, b);
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        uint32_t lo[4], hi[4];
        decode<Kd::FP8>(word_of(w[2 * r], i), even[2 * r], odd[2 * r], lo);
        decode<Kd::FP8>(word_of(w[2 * r + 1], i), even[2 * r + 1], odd[2 * r + 1], hi);
        multiply_word<Kd>(d[r], i == s * Kd::kWords, lo, hi, b);
      }
    }
    const uint32_t sw[4] = {sv.x, sv.y, sv.z, sv.w};
#pragma unroll
    for (int r = 0; r < 4; ++r) add_group<Kd>(acc[r], d[r], sw[r], sx);
  }
}

// The same for all NT column tiles: a decoded word serves each of them.  One
// operand after another, so that the sums of NT tiles fit the registers.
template <class Kd>
__device__ __forceinline__ void multiply_all(uint32_t stage, int lane, int inputs,
                                             const Columns<Kd>& cols,
                                             float (&acc)[Kd::NT][4][4]) {
  const int g = lane >> 2;
  uint32_t b[Kd::NT][4][4];
  float2 sx[Kd::NT];
#pragma unroll
  for (int t = 0; t < Kd::NT; ++t) {
#pragma unroll
    for (int i = 0; i < 4; ++i) cols.word(stage, lane, t, i, b[t][i]);
    sx[t] = Columns<Kd>::scale(stage, lane, t);
  }
#pragma unroll
  for (int r = 0; r < 4; ++r) {
    const uint4 w0 = lds16(stage + (2 * r) * 512 + lane * 16);
    const uint4 w1 = lds16(stage + (2 * r + 1) * 512 + lane * 16);
#pragma unroll
    for (int s = 0; s < Kd::kGroups; ++s) {
      if (!Kd::FP8 && Kd::GROUP * s >= inputs) break;      // groups past H
      const uint32_t sw = lds4(stage + Kd::kScales + s * 128 + g * 16 + r * 4);
      uint32_t even[2] = {kEven<Kd::FP8>, kEven<Kd::FP8>}, odd[2] = {kOdd, kOdd};
      if constexpr (Kd::ZEROS) {
        const uint32_t z = lds2(stage + Kd::kZeros + s * 64 + g * 8 + 2 * r);
        offsets<Kd::FP8>(z, 0, &even[0], &odd[0]);
        offsets<Kd::FP8>(z, 1, &even[1], &odd[1]);
      }
      float d[Kd::NT][4];
#pragma unroll
      for (int i = s * Kd::kWords; i < (s + 1) * Kd::kWords; ++i) {
        uint32_t lo[4], hi[4];
        decode<Kd::FP8>(word_of(w0, i), even[0], odd[0], lo);
        decode<Kd::FP8>(word_of(w1, i), even[1], odd[1], hi);
#pragma unroll
        for (int t = 0; t < Kd::NT; ++t)
          multiply_word<Kd>(d[t], i == s * Kd::kWords, lo, hi, b[t][i]);
      }
#pragma unroll
      for (int t = 0; t < Kd::NT; ++t) add_group<Kd>(acc[t][r], d[t], sw, sx[t]);
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
// sums in shared memory, in the order of the warps.  Each warp keeps STAGES
// units on their way in shared memory of its own (cp.async, so no barrier
// and no flag), across the ends of items too.  One CTA an SM.
//
// What bounds it.  Few rows: reading the weights.  128 tokens, 8 of 256
// experts, 4096 x 7168 gated, E4M3 rows: 3.82 GB in 562 us = 6.8 TB/s, 1.02
// of the measured copy rate.  One such token (121 MB): 25 us = 4.8 TB/s;
// its 512 items are 3.4 an SM, so that some SMs have four, and about 4 us
// are launch, table of chunks, first load and last sum.  One row by 7168 x
// 2048: 4.9 us, all latency.  Sixteen warps and not eight (659 us for the
// 128 tokens) because a unit is some 450 instructions that depend on each
// other closely: integer operations (half rate) to decode, about 230.  That
// is also what bounds many rows, with the tensor cores at a third; one
// decoding for two column tiles then pays.
template <class Kd, int WARPS, int STAGES>
__global__ void __launch_bounds__(WARPS * 32) expert_w4_kernel(W4Params p, int split) {
  constexpr int NT = Kd::NT;
  static_assert(Kd::kBytes >= NT * 2048, "a stage holds a warp's sums");
  extern __shared__ __align__(16) char smem[];
  int* const pre = reinterpret_cast<int*>(smem + WARPS * STAGES * Kd::kBytes);
  __shared__ uint32_t sums_at[WARPS];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const uint32_t base = smem_addr(smem) + warp * (STAGES * Kd::kBytes);
  pdl_wait();
  if (p.E <= 32)
    count_few_chunks<Kd::kChunk>(p, pre, lane);
  else
    count_chunks<Kd::kChunk>(p, pre);
  // groups are numbered across the CTAs first: a last partial round of items
  // then spreads over all SMs
  const int group = warp / split, slice = warp % split;
  Walk now(p, group * gridDim.x + blockIdx.x, gridDim.x * (WARPS / split), pre[p.E]);
  Walk ahead = now;      // the item of the unit to load next
  Loader<Kd> loader;
  loader.kb = p.blocks;
  const auto enter = [&] {
    loader.start(p, item_at<Kd::kChunk>(p, pre, ahead, lane), slice, lane);
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
  for (int i = 0; i < STAGES - 1; ++i) load_next(base + i * Kd::kBytes);

  Columns<Kd> cols = {};
  uint32_t stage = base, idle = base + (STAGES - 1) * Kd::kBytes;
  for (; !now.done(); now.advance(p)) {
    const Item it = item_at<Kd::kChunk>(p, pre, now, lane);
    const int used = (it.rows + 7) >> 3;
    cols.start(p, it, slice, lane);
    float acc[NT][4][4];
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int r = 0; r < 4; ++r)
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[t][r][i] = 0.0f;
    for (int kb = slice; kb < p.blocks; kb += split) {
      const int inputs = p.H - kb * kBlockIn;
      // one branch a unit: inside the products it would split the stream of
      // multiplications (measured 1.4 times slower)
      const bool all = NT > 1 && used > 1;
      if (all)
        cols.template load<NT>(inputs, split);
      else
        cols.template load<1>(inputs, split);
      cp_async_wait<STAGES - 2>();
      __syncwarp();      // the unit is there, and the idle stage was read by all
      load_next(idle);
      if (all)
        multiply_all<Kd>(stage, lane, inputs, cols, acc);
      else
        multiply_one<Kd>(stage, lane, inputs, cols, acc[0]);
      idle = stage;
      stage = stage == base + (STAGES - 1) * Kd::kBytes ? base : stage + Kd::kBytes;
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

template <class Kd>
cudaError_t launch_kind(const W4Params& p, int num_rows, cudaStream_t stream) {
  constexpr int WARPS = 16;
  // two stages; a third measured no faster, and leaves less of L1
  constexpr int STAGES = 2;
  static_assert(WARPS * STAGES * Kd::kBytes <= kSmemBudget);
  const double items = expected_chunks(num_rows, p.E, Kd::kChunk) * p.tiles;
  const int sms = device_info().sm_count;
  // Units one warp works through: rounds of items times its blocks of each,
  // and about one unit's time to add up a group's sums.  By groups of 1, 2,
  // 4, 8 and 16 warps: one token by 8 of 256 experts of 4096 x 7168 71, 45,
  // 25, 28 and 33 us; 128 such tokens 560, 578, 593, 650 and 804; one row by
  // 7168 x 2048 28, 17, 10, 7 and 5.
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
  // every SM that can have an item (an upper bound of them: an expert's last
  // chunk may be short), rather than as few as hold all groups
  const int64_t chunks = int64_t(num_rows) / Kd::kChunk + (num_rows < p.E ? num_rows : p.E);
  const int grid = int(chunks * p.tiles < sms ? chunks * p.tiles : sms);
  const size_t smem = WARPS * STAGES * Kd::kBytes + sizeof(int) * (p.E + 1);
  auto* kernel = expert_w4_kernel<Kd, WARPS, STAGES>;
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

// One column tile (8 rows) an item, or two where the experts in use have
// over seven rows on average.  64 experts of 2048 x 4096, one tile and two:
// bf16 rows 54 and 59 us at 4 rows an expert, 74 and 70 at 8, 122 and 103 at
// 16, 383 and 270 at 64; E4M3 50 and 54, 67 and 67, 113 and 99, 353 and 276.
// Two tiles of bf16 rows do not fit the stages of 16 warps and are read
// directly (staged, with 12 warps: 132 us at 16).
template <bool FP8, int GROUP, bool ZEROS>
cudaError_t launch_w4(const W4Params& p, int num_rows, cudaStream_t s) {
  const double active = p.E * (1.0 - pow(1.0 - 1.0 / p.E, num_rows));
  if (num_rows > 7.0 * active)
    return launch_kind<Kind<FP8, GROUP, ZEROS, 2, !FP8>>(p, num_rows, s);
  return launch_kind<Kind<FP8, GROUP, ZEROS, 1, false>>(p, num_rows, s);
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

// Products grouped by expert (ep_expert_mm) and their gradients
// (ep_expert_mm_backward) on the 5th-generation tensor cores.
//
// With x the rows of one expert (its segment [start, end) of the layout), W its
// matrix [N, H] and dy the gradient by the outputs:
//   forward   y  = x W^T      reduction over H    (gated: silu(y_g) * y_u)
//   by rows   dx = dy W       reduction over N
//   by W      dW = dy^T x     reduction over the segment's rows
//
// The first two put the weights on the product's M side (256 features a tile)
// and the rows on its N side: N is any multiple of 16 up to 256, so an
// expert's ragged rows cost no more than 15 idle columns, where rows on the M
// side would be rounded up to 128 or 256.  The accumulator then holds a
// feature a lane and a row a column, and the epilogue transposes it through
// shared memory.  dW is dense in both directions: 256 features of dy by 256
// of x.
//
// A pair of CTAs (cluster of two) works on a tile together: each holds half of
// the features and half of the columns in its shared memory, so that an
// operand byte is read from there half as often, and its half of the
// features' accumulator.  One persistent pair on two SMs, warps in roles: four
// read accumulators out, one issues tensor copies (TMA), one (of the first
// CTA) the products, twelve turn E4M3 rows into bf16 operands where the rows
// are in 8 bits, and one clears what a last step along the rows must not see.
// Operand tiles, 64 of the reduction each, pass through a ring of stages in
// shared memory, as many as fit for the columns that the experts' rows need;
// two accumulators alternate in tensor memory, so that one tile's epilogue
// runs beside the next one's products.
//
// E4M3 rows: the scale changes along the reduction (every 128 inputs), so it
// cannot be applied to a sum.  Forward, value * scale enters as two bf16
// parts, together within 1.4 * 2^-12 of it: the first CTA's columns are the
// first parts, the second's the others, and the epilogue adds the two sums.
// That halves the rows a tile holds, which costs nothing where the weights'
// bytes bound the product: up to some 50 rows an expert (64 experts of 4096 x
// 4096: 32 rows 335 us, in bf16 343; 100 rows 390 and 351; 256 rows 740 and
// 392).  A dW in fp32 takes two parts too, 17 bits together.  A dW in bf16
// takes bf16(value * scale) alone, a rounding of 2^-8 of the value at most, as
// rows have that were never quantised and as its own sums get at the end (off
// in the norm by 0.0023, and by 0.0017 without it): there the products cost,
// and two parts would double them.  Who wants them asks for fp32.
//
// Sums are fp32 in tensor memory, rounded once on the way out.  The tensor
// cores drop what lies below the accumulator's last bit, with each 16 of the
// reduction: about 2^-26 of a sum of one sign, which comes to 7e-6 for 7168
// inputs and to 1e-3, half the last rounding's size, for 2^20.
//
// What bounds it: the weights' bytes where experts have few rows (one token by
// 8 of 256 experts of 4096 x 7168: 75 us, 470 MB at 6.3 TB/s; 128 tokens 2070
// us, 7.1 TB/s), the tensor cores from about 300 rows an expert on (16384 rows
// by 4096 x 7168: 502 to 509 us alone, 1900 TFLOP/s, 565 to 585 under the power
// cap, where cuBLAS takes 481 to 517 and 553 to 560), the written
// bytes for dW of few rows (15 GB in 2.4 to 3.0 ms).  A single CTA's tile (128
// x 256, cta_group::1) took 733 us for the 16384 rows.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <atomic>
#include <type_traits>

#include "../../include/ep.h"
#include "ep_internal.h"
#include "segments.cuh"
#include "tcgen05.cuh"

namespace ep {
namespace {

enum Mode { kForward, kByRows, kByWeights };

constexpr int kLanes = 128;        // features of the M side a CTA
constexpr int kMaxCols = 256;      // columns of an accumulator
constexpr int kDepth = 64;         // reduction a stage: 128 bytes of bf16
constexpr int kMaxStages = 12;
constexpr int kABytes = kLanes * kDepth * 2;
constexpr int kBBytes = kMaxCols / 2 * kDepth * 2;      // a CTA's half, at most
constexpr int kPanel = 64 * kDepth * 2;         // 64 features by 64 rows
constexpr uint64_t kStepNs = 4000;              // far above what a stage takes
// Rows whose sum an fp32 gradient takes from one accumulator: the tensor cores
// drop what lies below the accumulator's last bit, about 2^-26 of the sum for
// each 16 rows (19,400 rows in one sum: off by 2.2e-5 in the norm).
constexpr int kMostRows = 2048;
constexpr int kMostParts = 4;                   // pairs that share a reduction: 8 CTAs
// Row tiles that share weight tiles in L2.  65536 rows by 4096 x 4096 in groups
// of 1, 8 and 64: 1095, 1120 and 1315 us; matrices beyond L2 need the sharing.
constexpr int kRowGroup = 8;

constexpr int kEpilogueWarps = 4, kCopyWarp = 4, kMmaWarp = 5, kClearWarp = 6;
constexpr int kFirstConvertWarp = 7, kConvertWarps = 12;
constexpr int kConvertGroups = 3;  // of warps, that take steps in turn
constexpr int kPieces = 4;         // of 16 values a converting thread has in a step
constexpr int kAhead = 2;          // steps of its own whose scales it loads ahead
static_assert(32 * kConvertWarps / kConvertGroups * kPieces * 16 == kMaxCols / 2 * kDepth);

__host__ __device__ constexpr int threads_of(bool fp8) {
  return 32 * (kFirstConvertWarp + (fp8 ? kConvertWarps : 0));
}
// Bytes that the epilogue's warps stage a tile's pieces in.
__host__ __device__ constexpr int staging_of(Mode m) {
  return kEpilogueWarps * (m == kByWeights ? 8192 : 2560);
}
// E4M3: scales that the converting warps share.
__host__ __device__ constexpr int scales_of(Mode m) {
  return kConvertGroups * 2 * (m == kByWeights ? kDepth : kMaxCols / 2);
}
// Whether E4M3 values enter as two bf16 parts, with a column each.
__host__ __device__ constexpr bool in_two_parts(Mode m, bool fp8, bool out32) {
  return fp8 && (m == kForward || out32);
}
// Rows of a tile (by weights: features of its N side).
__host__ __device__ constexpr int rows_of(bool two) { return two ? kMaxCols / 2 : kMaxCols; }

struct MmParams {
  int E, cap;
  int M;              // features of the M side an expert (outputs when gated)
  int depth;          // reduction (by weights: unused)
  int cols;           // by weights: features of the N side
  int m_tiles;
  int n_tiles;        // by weights
  int parts;          // of a tile's reduction
  const int32_t *start, *end;
  __nv_bfloat16* out;
  const float* xs;
  int x_width;        // features of an E4M3 row
  int ring_bytes;     // of the stages
  int32_t* err;
  bool add;           // by weights: to what is there
  bool leaves_l2;     // by weights: more is written than L2 holds
  bool stall;         // self-test: the first pair's copies never come
};

struct MmMaps {
  CUtensorMap a;
  CUtensorMap b[5];   // rows: boxes of 8, 16, 32, 64 and 128; by weights: b[0]
  CUtensorMap out;    // by weights
};

struct Smem {
  uint64_t full[kMaxStages];       // of the first CTA: both CTAs' operands are there
  uint64_t empty[kMaxStages];      // the products have read this CTA's
  uint64_t last[kMaxStages];       // a last step along the rows has landed here
  uint64_t raw[kMaxStages];        // E4M3 rows have landed here
  uint64_t acc_full[2];
  uint64_t acc_empty[2];           // of the first CTA: both have read it out
  uint64_t drained;
  // a reduction in parts: the other parts' sums are there (of the first pair);
  // this CTA's have been read (of the others)
  uint64_t sums_full, sums_read;
  uint32_t tmem;
  int most;                        // rows of a tile, at most
};

struct Item {
  int e, m0;          // expert, first feature of the M side
  int row0, rows;     // rows of the segment
  int c0;             // by weights: first feature of the N side
  int cols;           // columns of the product
  int blocks;         // steps of 64 along the reduction
  int first, steps;   // of them, this pair's
  int piece;          // of the segment's rows, by kMostRows
  bool more;          // pieces behind it
};

// The segment of expert e.
__device__ __forceinline__ void segment(const MmParams& p, int e, int& row0, int& rows) {
  clip_segment(p.start, p.end, p.cap, e, row0, rows);
}

// a / b for a >= 0, b > 0: 32-bit division where that does, a fifth of the
// 64-bit one's instructions.
__device__ __forceinline__ int64_t quotient(int64_t a, int b) {
  return a >> 32 == 0 ? int64_t(uint32_t(a) / uint32_t(b)) : a / b;
}

__device__ __forceinline__ int round16(int n) { return (n + 15) & ~15; }

// Place in the ring of stages.
struct Ring {
  int s = 0;
  uint32_t phase = 0;
  __device__ __forceinline__ void next(int stages) {
    if (++s == stages) {
      s = 0;
      phase ^= 1;
    }
  }
};

// A part of a reduction, `of` parts in all.
struct Part {
  int number, of;
};

__device__ __forceinline__ void share(Item& it, Part part) {
  it.first = int(int64_t(it.blocks) * part.number / part.of);
  it.steps = int(int64_t(it.blocks) * (part.number + 1) / part.of) - it.first;
}

template <Mode MODE, bool TWO, bool GATED, bool OUT32>
__device__ __forceinline__ Item item_at(const MmParams& p, const int* table, int64_t idx,
                                        int piece, Part part) {
  Item it;
  it.piece = piece;
  it.more = false;
  constexpr int kFeatures = GATED ? kLanes : 2 * kLanes;      // of a pair
  if (MODE == kByWeights) {
    const int tiles = p.m_tiles * p.n_tiles;
    it.e = int(quotient(idx, tiles));
    const int local = int(idx - int64_t(it.e) * tiles);
    it.m0 = local / p.n_tiles * kFeatures;
    it.c0 = local % p.n_tiles * rows_of(TWO);
    it.cols = p.cols - it.c0 > rows_of(TWO) / 2 ? kMaxCols : kMaxCols / 2;
    segment(p, it.e, it.row0, it.rows);
    if (OUT32) {
      const int64_t most = int64_t(kMostRows) * part.of, left = it.rows - piece * most;
      it.row0 += int(piece * most);
      it.more = left > most;
      it.rows = int(min(left, most));
    }
    it.blocks = int((int64_t(it.rows) + kDepth - 1) / kDepth);
    share(it, part);
    return it;
  }
  // the expert by its first row tile, then features outside, row tiles inside
  const int lo = expert_of(table, p.E, quotient(idx, p.m_tiles));
  it.e = lo;
  const int tiles = table[lo + 1] - table[lo];
  int64_t local = idx - int64_t(table[lo]) * p.m_tiles;
  const int group = int(quotient(local, kRowGroup * p.m_tiles));
  local -= int64_t(group) * kRowGroup * p.m_tiles;
  const int in_group = min(kRowGroup, tiles - group * kRowGroup);
  it.m0 = int(local) / in_group * kFeatures;
  const int tile = group * kRowGroup + int(local) % in_group;
  int row0, rows;
  segment(p, lo, row0, rows);
  const int per = round16(int((int64_t(rows) + tiles - 1) / tiles));
  it.row0 = row0 + tile * per;
  // (a table that came to its limit has fewer tiles than the rows need)
  it.rows = min(min(per, rows_of(TWO)), rows - tile * per);
  it.cols = round16(max(it.rows, 1)) * (TWO ? 2 : 1);
  it.c0 = 0;
  it.blocks = (p.depth + kDepth - 1) / kDepth;
  share(it, part);
  return it;
}

// A pair's way over the items, the pieces of one after another.
template <Mode MODE, bool TWO, bool GATED, bool OUT32>
struct Walk {
  const MmParams& p;
  const int* table;
  int64_t idx, items, pairs;
  Part part;
  Item it = {};

  __device__ __forceinline__ Walk(const MmParams& params, const int* t, int64_t first,
                                  int64_t pairs_, int64_t items_, Part part_)
      : p(params), table(t), idx(first), items(items_), pairs(pairs_), part(part_) {
    if (there()) it = item_at<MODE, TWO, GATED, OUT32>(p, table, idx, 0, part);
  }
  __device__ __forceinline__ bool there() const { return idx < items; }
  __device__ __forceinline__ bool last() const { return !it.more && idx + pairs >= items; }
  __device__ __forceinline__ void next() {
    const int piece = it.more ? it.piece + 1 : 0;
    if (!it.more) idx += pairs;
    if (there()) it = item_at<MODE, TWO, GATED, OUT32>(p, table, idx, piece, part);
  }
};

// Waits of a whole warp.  A lane polls, and may give up, on its own: all go on
// together and alike, as the warp-wide instructions behind a wait ask (elect,
// tcgen05.ld, barriers).
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity) {
  const bool ok = mbar_wait(bar, parity, kWaitTimeoutNs);
  return __all_sync(0xffffffffu, ok);
}

// For something that so many steps of a stage come before.
__device__ __forceinline__ bool wait_for_steps(uint64_t* bar, uint32_t parity, uint64_t steps) {
  bool ok = false;
  for (uint64_t i = 0; !ok && i <= steps * kStepNs / kWaitTimeoutNs; ++i)
    ok = mbar_wait(bar, parity, kWaitTimeoutNs);
  return __all_sync(0xffffffffu, ok);
}

// The same, for what other CTAs of the cluster wrote to their shared memory.
__device__ __forceinline__ bool wait_for_sums(uint64_t* bar, uint32_t parity, uint64_t steps) {
  bool ok = false;
  for (uint64_t i = 0; !ok && i <= steps * kStepNs / kWaitTimeoutNs; ++i)
    ok = mbar_wait_acquire(bar, parity, kWaitTimeoutNs);
  return __all_sync(0xffffffffu, ok);
}

__device__ __forceinline__ float silu(float g) { return g / (1.0f + expf(-g)); }

// How E4M3 values times their scale become bf16: the nearest, or what that
// leaves.
enum Bits { kNearest, kRest };

// 16 of them.
template <Bits PART>
__device__ __forceinline__ void widen16(uint4 q, float scale, uint32_t (&r)[8]) {
  const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint16_t two = uint16_t(w[i / 2] >> (16 * (i % 2)));
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(two));
    uint32_t a, b;
    asm("{\n\t.reg .f16 l, u;\n\t.reg .f32 x, y;\n\t.reg .b64 v, s;\n\t"
        "mov.b32 {l, u}, %2;\n\tcvt.f32.f16 x, l;\n\tcvt.f32.f16 y, u;\n\t"
        "mov.b64 v, {x, y};\n\tmov.b64 s, {%3, %3};\n\tmul.rn.f32x2 v, v, s;\n\t"
        "mov.b64 {%0, %1}, v;\n\t}"
        : "=r"(a), "=r"(b)
        : "r"(h), "f"(scale));
    const float x = __uint_as_float(a), y = __uint_as_float(b);
    r[i] = pack_bf16x2(x, y);
    if (PART == kRest) r[i] = pack_bf16x2(x - bf16_lo(r[i]), y - bf16_hi(r[i]));
  }
}

// Out of line: rare, and the loop around it is to stay small (the kernel is
// slowed by instruction fetch before anything else where it does not).
template <Bits PART>
__device__ __noinline__ void widen16_apart(uint4 q, float scale, uint32_t (&r)[8]) {
  widen16<PART>(q, scale, r);
}

// The two parts of 16 products without conversions.  Shifted four bits up, a
// magnitude of E4M3 is that of a bf16 2^-120 as large.  Of the scale, times
// 2^120, the first part takes its nearest number of four bits, by which any
// E4M3 value is exact in bf16, the second what is left, rounded twice to 8
// bits: together within 1.4 * 2^-12 of the product (1.31 over all mantissas).
// Scales of 128 and more (2^120 of which bf16 does not hold) and NaN go the way
// above; of scales below 2^-126 the first part is none.
template <Bits PART>
__device__ __forceinline__ void part16(uint4 q, float scale, uint32_t (&r)[8]) {
  const uint32_t w[4] = {q.x, q.y, q.z, q.w};
  uint32_t nan = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) nan |= (w[i] & 0x7f7f7f7fu) + 0x01010101u;
  if ((nan & 0x80808080u) != 0 || !(fabsf(scale) < 128.0f)) {
    uint32_t apart[8];
    widen16_apart<PART>(q, scale, apart);
#pragma unroll
    for (int i = 0; i < 8; ++i) r[i] = apart[i];
    return;
  }
  const float first = __uint_as_float((__float_as_uint(scale) + 0x00080000u) & 0xfff00000u);
  const float part = (PART == kNearest ? first : scale - first) * 0x1p120f;
  const uint32_t both = pack_bf16x2(part, part);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t up = (w[i] & 0x80808080u) | (w[i] >> 4 & 0x07070707u);
    const uint32_t low = w[i] << 4 & 0xf0f0f0f0u;
#pragma unroll
    for (int j = 0; j < 2; ++j)
      asm("mul.rn.bf16x2 %0, %1, %2;"
          : "=r"(r[2 * i + j])
          : "r"(__byte_perm(low, up, j ? 0x7362 : 0x5140)), "r"(both));
  }
}

// A barrier of `threads` threads (whole warps): whether all of them are `ok`.
// Each comes to it whether its own wait ran out or not, and all go on alike.
__device__ __forceinline__ bool group_agrees(int id, int threads, bool ok) {
  uint32_t all;
  __syncwarp();
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\t"
      "barrier.cta.red.and.aligned.pred q, %2, %3, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(all)
      : "r"(uint32_t(ok)), "r"(id), "r"(threads)
      : "memory");
  return all != 0;
}

template <Mode MODE, bool FP8, bool GATED, bool OUT32, bool SPLIT>
__global__ void __launch_bounds__(threads_of(FP8), 1)
    expert_mm_kernel(const __grid_constant__ MmMaps maps, const MmParams p) {
  extern __shared__ uint8_t shared_bytes[];
  // 1024-byte swizzle groups: what an operand's address is rounded up by is
  // the same in both CTAs
  uint8_t* ring = shared_bytes + (1023 & -smem_addr(shared_bytes));
  uint8_t* staging = ring + p.ring_bytes;
  Smem& sm = *reinterpret_cast<Smem*>(staging + staging_of(MODE));
  float* scale_at = reinterpret_cast<float*>(&sm + 1);
  int* table = reinterpret_cast<int*>(scale_at + (FP8 ? scales_of(MODE) : 0));
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x / 32, 0), lane = threadIdx.x % 32;
  const uint32_t lead = SPLIT ? cluster_rank() & ~1u : 0u, rank = cluster_rank() & 1;
  const int parts = SPLIT ? p.parts : 1;
  const Part part{int(lead / 2), parts};
  constexpr bool kAByFeature = MODE != kForward;      // inner dimension of A: features
  constexpr bool kBByFeature = MODE == kByWeights;
  constexpr bool kTwo = in_two_parts(MODE, FP8, OUT32);
  constexpr int kRows = rows_of(kTwo);
  constexpr int kRawWidth = kBByFeature ? 128 : kDepth;   // E4M3 values of a row in a step

  if (warp == kCopyWarp && lane == 0) {
    prefetch_map(&maps.a);
    prefetch_map(&maps.b[MODE == kByWeights ? 0 : 4]);
    for (int s = 0; s < kMaxStages; ++s) {
      mbar_init(&sm.full[s], FP8 ? 2 + 2 * kConvertWarps / kConvertGroups : 2);
      mbar_init(&sm.empty[s], 1);
      mbar_init(&sm.last[s], 1);
      mbar_init(&sm.raw[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&sm.acc_full[b], 1);
      mbar_init(&sm.acc_empty[b], 2 * kEpilogueWarps);
    }
    mbar_init(&sm.drained, 1);
    mbar_init(&sm.sums_full, kEpilogueWarps * (parts - 1 > 0 ? parts - 1 : 1));
    mbar_init(&sm.sums_read, kEpilogueWarps);
    sm.most = 0;
    fence_mbar_init();
  }
  pdl_wait();
  // not before: the kernel ahead may still want tensor memory of its own
  if (warp == kMmaWarp) tmem_alloc(&sm.tmem, 2 * kMaxCols);
  int64_t items;
  int stage_bytes = kABytes + kBBytes;
  if (MODE == kByWeights) {
    items = int64_t(p.E) * p.m_tiles * p.n_tiles;
  } else {
    // row tiles of the experts before each one, and the largest tile
    __syncthreads();
    int most = 0;
    count_experts(p.E, table, reinterpret_cast<int64_t*>(staging), [&](int e) {
      int row0, rows;
      segment(p, e, row0, rows);
      most = max(most, min(rows, kRows));
      return int((int64_t(rows) + kRows - 1) / kRows);
    });
    most = __reduce_max_sync(0xffffffffu, most);
    if (lane == 0) atomicMax(&sm.most, most);
    __syncthreads();
    items = int64_t(table[p.E]) * p.m_tiles;
    // E4M3: all rows in each CTA, else half of them; in groups of eight
    const int rows = round16(sm.most) / (FP8 ? 1 : 2);
    stage_bytes = kABytes + rows * (kDepth * 2);
  }
  // E4M3: a stage is always the same group's.  A group that skipped uses of a
  // stage could take the one before last for the last (their parities are
  // alike) where copies land out of order.
  int stages = min(kMaxStages, p.ring_bytes / stage_bytes);
  if (FP8) stages -= stages % kConvertGroups;
  tc_fence_before();
  cluster_sync();
  tc_fence_after();
  const uint32_t tmem = sm.tmem;
  // clusters, a pair each, or as many as share a tile's reduction
  const int64_t pair = blockIdx.x / (2 * parts), pairs = gridDim.x / (2 * parts);
  using Tiles = Walk<MODE, kTwo, GATED, OUT32>;
  Ring at;

  if (warp == kCopyWarp) {
    bool ok = !p.stall || pair != 0;
    uint64_t n = 0;      // stages filled so far
    [[maybe_unused]] uint32_t tile = 0;
    for (Tiles tiles(p, table, pair, pairs, items, part); ok && tiles.there(); tiles.next()) {
      const Item& it = tiles.it;
      const int half = it.cols / 2;
      // bytes of this CTA's copies into a stage
      const int bytes = kABytes + (FP8 ? 0 : half * kDepth * 2);
      const int m0 = it.m0 + int(rank) * (GATED ? kLanes / 2 : kLanes);
      const int col0 = kTwo ? 0 : int(rank) * half;
      for (int kb = 0; kb < it.steps; ++kb, ++n, at.next(stages)) {
        ok = warp_wait(&sm.empty[at.s], at.phase ^ 1);
        if (!ok) break;
        const uint32_t a = smem_addr(ring + at.s * stage_bytes), b = a + kABytes;
        const int k0 = (it.first + kb) * kDepth;
        // cleared past the segment's end before it counts as full
        const bool last = MODE == kByWeights && it.rows - k0 < kDepth;
        const uint32_t full = at_rank(smem_addr(&sm.full[at.s]), lead);
        const uint32_t bar = last ? smem_addr(&sm.last[at.s]) : full;
        if (elect_one()) {
          if (last)
            mbar_arrive_expect_tx(&sm.last[at.s], bytes);
          else if (rank == 0)
            mbar_arrive_expect_tx(&sm.full[at.s], 2 * bytes);
          else
            mbar_arrive_cluster(full);
          if (MODE == kForward) {
            if (GATED)
              tma_load_5d(a, &maps.a, bar, k0, 0, 0, m0 / 16, it.e);
            else
              tma_load_3d(a, &maps.a, bar, k0, m0, it.e);
          } else if (MODE == kByRows) {
            tma_load_3d(a, &maps.a, bar, m0, k0, it.e);
            tma_load_3d(a + kPanel, &maps.a, bar, m0 + 64, k0, it.e);
          } else {
            tma_load_2d(a, &maps.a, bar, m0, it.row0 + k0);
            tma_load_2d(a + kPanel, &maps.a, bar, m0 + 64, it.row0 + k0);
          }
          const uint32_t b_bar = FP8 ? smem_addr(&sm.raw[at.s]) : bar;
          if (FP8) mbar_arrive_expect_tx(&sm.raw[at.s], kRawWidth * (kBByFeature ? kDepth : half));
          if (kBByFeature) {
            for (int c = 0; c < half; c += FP8 ? 128 : 64)
              tma_load_2d(b + c / 64 * kPanel, &maps.b[0], b_bar, it.c0 + col0 + c,
                          it.row0 + k0);
          } else {
            // boxes of the binary digits of the CTA's rows; E4M3: all rows
            constexpr int kPitch = FP8 ? kRawWidth : kDepth * 2;
            int r = 0;
#pragma unroll
            for (int i = 4; i >= (FP8 ? 1 : 0); --i)
              if (half & (8 << i)) {
                tma_load_2d(b + r * kPitch, &maps.b[i], b_bar, k0,
                            it.row0 + (FP8 ? 0 : col0) + r);
                r += 8 << i;
              }
          }
        }
        __syncwarp();
      }
      // the sums of this part lie where the operands of its next tile come
      if (SPLIT && ok && part.number > 0 && !tiles.last()) {
        ok = wait_for_steps(&sm.sums_read, tile & 1, it.blocks);
        ++tile;
      }
    }
    if (!ok && lane == 0) {
      record_error(p.err, ERRBIT_TIMEOUT);
      // the first CTA's barriers count the copies of both, which land before
      // the pair may end (the second CTA waits for the first one's end)
      for (uint64_t i = n < uint64_t(stages) ? 0 : n - stages; i < n; ++i)
        if ((FP8 && !mbar_wait(&sm.raw[i % stages], i / stages & 1, kWaitTimeoutNs)) ||
            (rank == 0 && !mbar_wait(&sm.full[i % stages], i / stages & 1, kWaitTimeoutNs)))
          record_error(p.err, ERRBIT_TIMEOUT_PENDING);
    }
    __syncwarp();
  } else if (warp == kMmaWarp && rank == 0) {
    uint32_t tile = 0;
    bool ok = true;
    for (Tiles tiles(p, table, pair, pairs, items, part); ok && tiles.there(); tiles.next()) {
      const Item& it = tiles.it;
      if (it.steps == 0) continue;
      const uint32_t idesc = instr_desc(2 * kLanes, it.cols, kAByFeature, kBByFeature);
      const uint32_t buf = tile & 1, acc = tmem + buf * kMaxCols;
      ok = warp_wait(&sm.acc_empty[buf], (tile / 2 & 1) ^ 1);
      if (!ok) break;
      tc_fence_after();
      for (int kb = 0; kb < it.steps; ++kb, at.next(stages)) {
        ok = warp_wait(&sm.full[at.s], at.phase);
        if (!ok) break;
        tc_fence_after();
        const uint32_t a = smem_addr(ring + at.s * stage_bytes), b = a + kABytes;
        const uint64_t da = smem_desc(a, kAByFeature ? kPanel : 16, 1024);
        const uint64_t db = smem_desc(b, kBByFeature ? kPanel : 16, 1024);
        // 16 of the reduction further: 32 bytes of a row, or 16 rows
        constexpr uint32_t as = (kAByFeature ? 2048 : 32) >> 4, bs = (kBByFeature ? 2048 : 32) >> 4;
        const int steps =
            MODE == kByWeights
                ? min(kDepth / 16, (it.rows - (it.first + kb) * kDepth + 15) / 16)
                : kDepth / 16;
        if (elect_one()) {
#pragma unroll
          for (int i = 0; i < kDepth / 16; ++i)
            if (i < steps) mma_bf16(acc, da + i * as, db + i * bs, idesc, kb > 0 || i > 0);
          mma_commit(smem_addr(&sm.empty[at.s]), lead);
          if (kb == it.steps - 1) mma_commit(smem_addr(&sm.acc_full[buf]), lead);
        }
        __syncwarp();
      }
      ++tile;
    }
    if (!ok) {
      // products in flight end before the tensor memory is given back
      if (elect_one()) {
        record_error(p.err, ERRBIT_TIMEOUT);
        mma_commit(smem_addr(&sm.drained), lead);
      }
      __syncwarp();
      mbar_wait(&sm.drained, 0, kWaitTimeoutNs);
    }
    __syncwarp();
  } else if (MODE == kByWeights && warp == kClearWarp) {
    // Rows past the segment's end are another expert's, or nobody's: products
    // take steps of 16 rows, and this CTA's operands are zero up to a step's end.
    bool ok = true;
    uint32_t phases = 0;
    uint64_t passed = 0;      // steps since the last wait
    for (Tiles tiles(p, table, pair, pairs, items, part); ok && tiles.there(); tiles.next()) {
      const Item& it = tiles.it;
      for (int kb = 0; kb < it.steps; ++kb, ++passed, at.next(stages)) {
        const int left = it.rows - (it.first + kb) * kDepth;
        if (left >= kDepth) continue;
        // all steps before pass meanwhile
        ok = wait_for_steps(&sm.last[at.s], phases >> at.s & 1, passed);
        if (!ok) break;
        passed = 0;
        phases ^= 1u << at.s;
        uint8_t* a = ring + at.s * stage_bytes;
        const int panels = kLanes / 64 + (FP8 ? 0 : it.cols / 128);
        const int pieces = (round16(left) - left) * 8;
        for (int i = lane; i < panels * pieces; i += 32)
          *reinterpret_cast<uint4*>(a + i / pieces * kPanel + left * 128 + i % pieces * 16) =
              make_uint4(0, 0, 0, 0);
        fence_async_shared();
        __syncwarp();
        if (lane == 0) mbar_arrive_cluster(at_rank(smem_addr(&sm.full[at.s]), lead));
      }
    }
    if (!ok && lane == 0) record_error(p.err, ERRBIT_TIMEOUT);
    __syncwarp();
  } else if (FP8 && warp >= kFirstConvertWarp) {
    // Three groups of four warps take steps in turn; the rows' bytes come by
    // tensor copies, their scales are loaded kAhead turns ahead, past the ends
    // of tiles.
    constexpr int kThreads = 32 * kConvertWarps / kConvertGroups;
    const int group = (warp - kFirstConvertWarp) / (kConvertWarps / kConvertGroups);
    const int t = (threadIdx.x - kFirstConvertWarp * 32) % kThreads;
    // pieces of 16 values: forward, 4 of each of the rows for a step's 64
    // inputs; by weights, 8 of each of its 64 rows
    constexpr int kOfRow = kRawWidth / 16;
    const int row_t = t / kOfRow, c_t = t % kOfRow * 16;
    const int scales = p.x_width / 128;
    // one scale a thread, of its row, shared through two buffers a group
    constexpr int kScaled = kBByFeature ? kDepth : kThreads;
    float* const shared = scale_at + group * 2 * kScaled;
    int turn = 0;
    float sc[kAhead];
    int halves[kAhead];         // columns of the step's tile a CTA, 0 past the last one
    int lefts[kAhead];          // rows of the segment from the step's first on
    Tiles tiles(p, table, pair, pairs, items, part);
    const Item& it = tiles.it;
    int kb = -1;
    bool more = tiles.there();
    const auto step = [&] {
      if (!more || ++kb < it.steps) return;
      kb = 0;
      do {
        tiles.next();
        more = tiles.there();
      } while (more && it.steps == 0);
    };
    const auto load = [&](float& scale, int& half, int& left) {
      half = more ? it.cols / 2 : 0;
      const int at_k = (it.first + kb) * kDepth;
      left = it.rows - (kBByFeature ? at_k : 0);
      const int x = kBByFeature ? it.c0 + (kTwo ? 0 : int(rank) * half) : at_k;
      scale = 0.0f;
      if (more && t < kScaled && t < left && x < p.x_width)
        scale = __ldg(p.xs + (int64_t(it.row0) + it.rows - left + t) * scales + x / 128);
      // (unrolled, the loop outgrows the instruction cache: 65536 rows forward
      // 3694 us, and 3130 like this)
#pragma unroll 1
      for (int g = 0; g < kConvertGroups; ++g) step();
    };
#pragma unroll 1
    for (int g = 0; g <= group; ++g) step();      // to this group's first
    for (int g = 0; g < group; ++g) at.next(stages);
#pragma unroll
    for (int d = 0; d < kAhead; ++d) load(sc[d], halves[d], lefts[d]);
    bool ok = true, some = true;
    const auto convert = [&](auto which) {
      constexpr Bits PART = decltype(which)::value;
      while (ok && some) {
#pragma unroll
        for (int d = 0; d < kAhead; ++d) {
          const int half = halves[d];
          [[maybe_unused]] const int left = lefts[d];
          some = half > 0;
          if (!some) break;
          ok = warp_wait(&sm.raw[at.s], at.phase);
          uint8_t* to = ring + at.s * stage_bytes + kABytes;
          uint4 q[kPieces];
#pragma unroll
          for (int i = 0; i < kPieces; ++i)
            if (kBByFeature || row_t + kThreads / kOfRow * i < half)
              q[i] = *reinterpret_cast<const uint4*>(to + (t + i * kThreads) * 16);
          float* const mine = shared + turn * kScaled;
          turn ^= 1;
          if (t < kScaled) mine[t] = sc[d];
          ok = group_agrees(group + 1, kThreads, ok);
          if (!ok) break;
          if (kBByFeature) to += c_t / 64 * kPanel;
          const int c = c_t % 64 / 8;
#pragma unroll
          for (int i = 0; i < kPieces; ++i) {
            const int row = row_t + kThreads / kOfRow * i;
            if (kBByFeature ? c_t >= half : row >= half) break;
            const float scale = mine[row];
            uint32_t r[8];
            if constexpr (kBByFeature) {
              // a row of another segment, or of none, may hold anything
              if (row >= left) q[i] = make_uint4(0, 0, 0, 0);
              widen16<PART>(q[i], scale, r);
            } else {
              part16<PART>(q[i], scale, r);
            }
            *reinterpret_cast<uint4*>(to + row * 128 + ((c ^ (row & 7)) * 16)) =
                make_uint4(r[0], r[1], r[2], r[3]);
            *reinterpret_cast<uint4*>(to + row * 128 + (((c + 1) ^ (row & 7)) * 16)) =
                make_uint4(r[4], r[5], r[6], r[7]);
          }
          fence_async_shared();
          __syncwarp();
          if (lane == 0) mbar_arrive_cluster(at_rank(smem_addr(&sm.full[at.s]), lead));
          for (int g = 0; g < kConvertGroups; ++g) at.next(stages);
          load(sc[d], halves[d], lefts[d]);
        }
      }
    };
    if (!kTwo || rank == 0)
      convert(std::integral_constant<Bits, kNearest>());
    else
      convert(std::integral_constant<Bits, kRest>());
    if (!ok && lane == 0) record_error(p.err, ERRBIT_TIMEOUT);
    __syncwarp();
  } else if (warp < kEpilogueWarps) {
    uint8_t* mine = staging + warp * (staging_of(MODE) / kEpilogueWarps);
    uint32_t tile = 0;
    [[maybe_unused]] uint32_t joined = 0;
    int turn = 0;
    bool ok = true;
    for (Tiles tiles(p, table, pair, pairs, items, part); ok && tiles.there(); tiles.next()) {
      const Item& it = tiles.it;
      const uint32_t buf = tile & 1;
      const uint32_t acc = tmem + buf * kMaxCols + (uint32_t(warp * 32) << 16);
      if (it.steps > 0) {
        // the tile's whole reduction may pass before
        ok = wait_for_steps(&sm.acc_full[buf], tile / 2 & 1, it.steps);
        if (!ok) break;
        tc_fence_after();
      }
      if (SPLIT && part.number == 0) {
        ok = wait_for_sums(&sm.sums_full, joined & 1, it.blocks);
        if (!ok) break;
      } else if (SPLIT && joined > 0) {
        // (a part without steps has waited for nothing yet)
        ok = wait_for_steps(&sm.sums_read, (joined - 1) & 1, it.blocks);
        if (!ok) break;
      }
      // Sums of 32 columns: a part that is not the first leaves them where its
      // operands were (the products have read all of them, and the copying
      // warp waits), the first adds the others' to its own, in their order.
      const auto join = [&](int chunk, uint32_t (&v)[32]) {
        const uint32_t at = (chunk * kEpilogueWarps + warp) * 4096 + lane * 16;
        if (part.number > 0) {
#pragma unroll
          for (int i = 0; i < 8; ++i)
            *reinterpret_cast<uint4*>(ring + at + i * 512) =
                make_uint4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
          return;
        }
#pragma unroll 1
        for (int other = 1; other < parts; ++other) {
          const uint32_t from = at_rank(smem_addr(ring) + at, rank + 2 * other);
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const uint4 w = load_cluster(from + i * 512);
            const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
            for (int j = 0; j < 4; ++j)
              v[4 * i + j] =
                  __float_as_uint(__uint_as_float(v[4 * i + j]) + __uint_as_float(u[j]));
          }
        }
      };
      if (MODE == kByWeights) {
        constexpr int kWide = OUT32 ? 32 : 64;      // columns of 128 bytes
        const int m = it.m0 + int(rank) * kLanes + warp * 32;
        const int cols = kTwo ? it.cols / 2 : it.cols;
        // (adding nothing would still turn -0 and subnormal values into 0)
        const bool nothing = OUT32 && p.add && it.blocks == 0;
        // what more is added to stays
        const uint64_t policy = l2_policy(p.leaves_l2 && !it.more);
        // the pieces before have to be there
        if (OUT32 && it.piece > 0) {
          if (lane == 0) tma_store_wait<0>();
          __syncwarp();
        }
#pragma unroll 1
        for (int c = 0; c < cols && !nothing; c += kWide) {
          if (it.c0 + c >= p.cols || m >= p.M) break;
          uint32_t r[kWide / 32][32];
#pragma unroll
          for (int h = 0; h < kWide / 32; ++h) {
            if (it.steps > 0) {
              tmem_load_32x32(acc + c + h * 32, r[h]);
            } else {
#pragma unroll
              for (int i = 0; i < 32; ++i) r[h][i] = 0;
            }
          }
          tmem_wait_load();
          if (kTwo && it.steps > 0) {
            // the sums of the rests
            uint32_t rest[32];
            tmem_load_32x32(acc + cols + c, rest);
            tmem_wait_load();
#pragma unroll
            for (int i = 0; i < 32; ++i)
              r[0][i] = __float_as_uint(__uint_as_float(r[0][i]) + __uint_as_float(rest[i]));
          }
          if (SPLIT) {
#pragma unroll
            for (int h = 0; h < kWide / 32; ++h) join(c / 32 + h, r[h]);
            if (part.number > 0) continue;
          }
          // two pieces in turn: the one before the last has left this one
          uint8_t* piece = mine + turn * 4096;
          turn ^= 1;
          if (lane == 0) tma_store_wait_read<1>();
          __syncwarp();
#pragma unroll
          for (int v = 0; v < 8; ++v) {
            uint4 w;
            if (OUT32) {
              w = make_uint4(r[0][4 * v], r[0][4 * v + 1], r[0][4 * v + 2], r[0][4 * v + 3]);
            } else {
              const uint32_t* u = &r[(8 * v / 32) % (kWide / 32)][8 * v % 32];
              w = make_uint4(pack_bf16x2(__uint_as_float(u[0]), __uint_as_float(u[1])),
                             pack_bf16x2(__uint_as_float(u[2]), __uint_as_float(u[3])),
                             pack_bf16x2(__uint_as_float(u[4]), __uint_as_float(u[5])),
                             pack_bf16x2(__uint_as_float(u[6]), __uint_as_float(u[7])));
            }
            *reinterpret_cast<uint4*>(piece + lane * 128 + ((v ^ (lane & 7)) * 16)) = w;
          }
          fence_async_shared();
          __syncwarp();
          if (lane == 0) {
            if (OUT32 && (p.add || it.piece > 0))
              tma_add_3d(&maps.out, smem_addr(piece), it.c0 + c, m, it.e);
            else
              tma_store_3d(&maps.out, smem_addr(piece), it.c0 + c, m, it.e, policy);
            tma_store_commit();
          }
        }
      } else {
        constexpr int kWidth = GATED ? 16 : 32;             // features of this warp
        constexpr int kPitch = GATED ? 48 : 80;             // bytes of a staged row
        const int m = it.m0 + int(rank) * (kEpilogueWarps * kWidth) + warp * kWidth;
        const int rows = FP8 ? it.cols / 2 : it.cols;
#pragma unroll 1
        for (int c = 0; c < rows; c += 32) {
          if (m >= p.M) break;
          uint32_t r[32];      // of 16 lanes, and of the 16 behind them
          uint32_t(&r0)[16] = *reinterpret_cast<uint32_t(*)[16]>(r);
          uint32_t(&r1)[16] = *reinterpret_cast<uint32_t(*)[16]>(r + 16);
          if (it.steps > 0) {
            tmem_load_16x32(acc + c, r0);
            tmem_load_16x32(acc + c + (16u << 16), r1);
            if (FP8) {
              // the sums of the rests
              uint32_t s0[16], s1[16];
              tmem_load_16x32(acc + rows + c, s0);
              tmem_load_16x32(acc + rows + c + (16u << 16), s1);
              tmem_wait_load();
#pragma unroll
              for (int i = 0; i < 16; ++i) {
                r0[i] = __float_as_uint(__uint_as_float(r0[i]) + __uint_as_float(s0[i]));
                r1[i] = __float_as_uint(__uint_as_float(r1[i]) + __uint_as_float(s1[i]));
              }
            } else {
              tmem_wait_load();
            }
          } else {
#pragma unroll
            for (int i = 0; i < 32; ++i) r[i] = 0;
          }
          if (SPLIT) {
            join(c / 32, r);
            if (part.number > 0) continue;
          }
          // matrices of 8 features by 8 rows, transposed on the way
          const uint32_t to =
              smem_addr(mine) + (lane % 8 + lane / 16 * 8) * kPitch + (lane / 8 % 2) * 16;
          if (GATED) {
            float y[16];
#pragma unroll
            for (int i = 0; i < 16; ++i)
              y[i] = silu(__uint_as_float(r0[i])) * __uint_as_float(r1[i]);
#pragma unroll
            for (int j = 0; j < 4; j += 2)
              stmatrix_t4(to + j * 8 * kPitch, pack_bf16x2(y[4 * j], y[4 * j + 1]),
                          pack_bf16x2(y[4 * j + 2], y[4 * j + 3]),
                          pack_bf16x2(y[4 * j + 4], y[4 * j + 5]),
                          pack_bf16x2(y[4 * j + 6], y[4 * j + 7]));
          } else {
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
              for (int j = 0; j < 4; j += 2) {
                uint32_t w[4];
#pragma unroll
                for (int i = 0; i < 4; ++i)
                  w[i] = pack_bf16x2(__uint_as_float(h ? r1[4 * j + 2 * i] : r0[4 * j + 2 * i]),
                                     __uint_as_float(h ? r1[4 * j + 2 * i + 1]
                                                       : r0[4 * j + 2 * i + 1]));
                stmatrix_t4(to + j * 8 * kPitch + h * 32, w[0], w[1], w[2], w[3]);
              }
          }
          __syncwarp();
          constexpr int kVecs = kWidth / 8;                 // 16-byte pieces of a row
#pragma unroll
          for (int i = 0; i < kVecs; ++i) {
            const int row = lane / kVecs + i * (32 / kVecs), v = lane % kVecs;
            if (c + row < it.rows && m + v * 8 < p.M) {
              const uint4 w = *reinterpret_cast<const uint4*>(mine + row * kPitch + v * 16);
              *reinterpret_cast<uint4*>(p.out + (int64_t(it.row0) + c + row) * p.M + m + v * 8) = w;
            }
          }
          __syncwarp();
        }
      }
      if (it.steps > 0) {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_cluster(at_rank(smem_addr(&sm.acc_empty[buf]), lead));
        ++tile;
      }
      if (SPLIT) {
        ++joined;
        fence_async_shared();
        __syncwarp();
        if (lane == 0 && part.number > 0)
          mbar_arrive_release(at_rank(smem_addr(&sm.sums_full), rank));
        for (int other = 1; lane == 0 && part.number == 0 && other < parts; ++other)
          mbar_arrive_release(at_rank(smem_addr(&sm.sums_read), rank + 2 * other));
      }
    }
    if (MODE == kByWeights && lane == 0) tma_store_wait<0>();
    if (!ok && lane == 0) record_error(p.err, ERRBIT_TIMEOUT);
    __syncwarp();
  }
  tc_fence_before();
  cluster_sync();
  tc_fence_after();
  if (warp == kMmaWarp) tmem_free(tmem, 2 * kMaxCols);
}

// ---- host ---------------------------------------------------------------------

bool aligned(const void* p) { return p != nullptr && reinterpret_cast<uintptr_t>(p) % 16 == 0; }

bool config_ok(const ep_expert_config* c) {
  if (c == nullptr || c->num_experts < 1 || c->num_experts > 2048) return false;
  if (c->in_features < 8 || c->in_features > (1 << 20) || c->in_features % 8 != 0) return false;
  if (c->out_features < 8 || c->out_features > (1 << 20) || c->out_features % 8 != 0) return false;
  if (c->x_fp8 != 0 && c->x_fp8 != 1) return false;
  if (c->gated != 0 && c->gated != 1) return false;
  if (c->x_fp8 && c->in_features % 128 != 0) return false;
  if (c->gated && c->out_features % 32 != 0) return false;
  // strides of the tensor copies
  return int64_t(c->in_features) * c->out_features < (int64_t(1) << 38);
}

int32_t status(cudaError_t e) { return note_cuda(e) == cudaSuccess ? EP_OK : EP_ERR_CUDA; }

using EncodeFn = decltype(&cuTensorMapEncodeTiled);

cudaError_t encoder(EncodeFn* fn) {
  static std::atomic<EncodeFn> found{nullptr};
  *fn = found.load(std::memory_order_acquire);
  if (*fn != nullptr) return cudaSuccess;
  void* at = nullptr;
  cudaDriverEntryPointQueryResult how;
  const cudaError_t e = cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &at, 12000,
                                                         cudaEnableDefault, &how);
  if (e != cudaSuccess) return e;
  if (how != cudaDriverEntryPointSuccess || at == nullptr) return cudaErrorNotSupported;
  *fn = reinterpret_cast<EncodeFn>(at);
  found.store(*fn, std::memory_order_release);
  return cudaSuccess;
}

// A map of bf16 (or fp32) values, innermost dimension first, boxes of 128
// bytes by `box`; strides in elements, of all dimensions but the first.
template <int D>
cudaError_t encode(CUtensorMap* m, bool f32, const void* base, const uint64_t (&dims)[D],
                   const uint64_t (&strides)[D - 1], const uint32_t (&box)[D]) {
  EncodeFn fn;
  cudaError_t e = encoder(&fn);
  if (e != cudaSuccess) return e;
  cuuint64_t n[D], s[D - 1];
  cuuint32_t b[D], step[D];
  for (int i = 0; i < D; ++i) {
    n[i] = dims[i];
    b[i] = box[i];
    step[i] = 1;
    if (i > 0) s[i - 1] = strides[i - 1] * (f32 ? 4 : 2);
  }
  const CUresult r = fn(m, f32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16,
                        D, const_cast<void*>(base), n, s, b, step, CU_TENSOR_MAP_INTERLEAVE_NONE,
                        CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                        CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

// E4M3 [rows, width] in boxes of `wide` columns by `high` rows.
cudaError_t encode_bytes(CUtensorMap* m, const void* base, int rows, int width, int wide,
                         int high) {
  EncodeFn fn;
  cudaError_t e = encoder(&fn);
  if (e != cudaSuccess) return e;
  const cuuint64_t n[2] = {cuuint64_t(width), cuuint64_t(rows)}, s[1] = {cuuint64_t(width)};
  const cuuint32_t b[2] = {cuuint32_t(wide), cuuint32_t(high)}, step[2] = {1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(base), n, s, b, step,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS
             ? cudaSuccess
             : cudaErrorInvalidValue;
}

// [rows, width] in boxes of 64 columns by `high` rows.
cudaError_t encode_rows(CUtensorMap* m, const void* base, int rows, int width, int high) {
  return encode<2>(m, false, base, {uint64_t(width), uint64_t(rows)}, {uint64_t(width)},
                   {64, uint32_t(high)});
}

// [E, N, H] in boxes of 128 bytes by `high` rows.
cudaError_t encode_weights(CUtensorMap* m, bool f32, const void* base, int E, int N, int H,
                           int high) {
  return encode<3>(m, f32, base, {uint64_t(H), uint64_t(N), uint64_t(E)},
                   {uint64_t(H), uint64_t(N) * H}, {f32 ? 32u : 64u, uint32_t(high), 1});
}

// Dynamic shared memory: the ring takes what the staging pieces, the barriers
// and the table of the most experts leave of 227 KiB.
constexpr int kSmemLimit = 227 * 1024;
constexpr int64_t kL2Bytes = 129 << 20;

constexpr int rest_bytes(Mode m, bool fp8, int table) {
  return 1024 + staging_of(m) + int(sizeof(Smem)) + 4 * ((fp8 ? scales_of(m) : 0) + table);
}
static_assert(kSmemLimit - rest_bytes(kByWeights, true, 0) >= 6 * (kABytes + kBBytes));

template <Mode MODE, bool FP8, bool GATED, bool OUT32, bool SPLIT>
cudaError_t launch_parts(const MmMaps& maps, MmParams p, int clusters, cudaStream_t s) {
  auto* kernel = expert_mm_kernel<MODE, FP8, GATED, OUT32, SPLIT>;
  // once per kernel and device
  static std::atomic<uint64_t> raised{0};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev >= 64 || !(raised.load(std::memory_order_acquire) >> dev & 1)) {
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemLimit);
    if (e != cudaSuccess) return e;
    if (dev < 64) raised.fetch_or(uint64_t(1) << dev, std::memory_order_release);
  }
  const int rest = rest_bytes(MODE, FP8, MODE == kByWeights ? 0 : p.E + 1);
  p.ring_bytes = (kSmemLimit - rest) / 1024 * 1024;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(2 * p.parts * clusters);
  cfg.blockDim = dim3(threads_of(FP8));
  cfg.dynamicSmemBytes = size_t(p.ring_bytes + rest);
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2 * p.parts;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kernel, maps, p);
}

// most_items: tiles at most; steps: of a tile's reduction (about).
template <Mode MODE, bool FP8, bool GATED, bool OUT32>
cudaError_t launch(const MmMaps& maps, MmParams p, int64_t most_items, int64_t steps,
                   cudaStream_t s) {
  const int64_t pairs = device_info().sm_count / 2;
  // Where tiles leave most pairs without work, two or four of them share a
  // tile's reduction, down to 16 steps each: 8 rows by 1024 x 7168, in 1, 2 and
  // 4 parts, 19.7, 13.8 and 11.5 us; dW of 8192 rows, 512 x 512, 38.8, 27.6 and
  // 23.5; but 8 steps a part 7.5 us alone, 8.4 shared.  Clusters fill three
  // quarters of the SMs at most: what does not fit into the groups of SMs that
  // clusters are placed in would come in a second round (16 clusters of 8:
  // 39.8 us, 32 of 4 23.5).
  p.parts = 1;
  while (p.parts < kMostParts && most_items * p.parts * 2 <= pairs * 3 / 4 &&
         steps >= 32 * p.parts)
    p.parts *= 2;
  const int clusters = int(most_items < pairs / p.parts ? most_items : pairs / p.parts);
  return p.parts > 1 ? launch_parts<MODE, FP8, GATED, OUT32, true>(maps, p, clusters, s)
                     : launch_parts<MODE, FP8, GATED, OUT32, false>(maps, p, clusters, s);
}

// Tiles that `rows` rows of E experts can make, at most, by feature tiles.
int64_t most_row_tiles(int rows, int E, bool fp8) {
  return int64_t(rows) / rows_of(fp8) + (rows < E ? rows : E);
}

MmParams params(const ep_expert_config* cfg, int cap, const int32_t* start, const int32_t* end,
                int32_t* err) {
  MmParams p = {};
  p.E = cfg->num_experts;
  p.cap = cap;
  p.start = start;
  p.end = end;
  p.err = err;
  return p;
}

cudaError_t forward(const ep_expert_config* c, int cap, int num_rows, const void* x,
                    const float* x_scale, const void* w, const int32_t* start, const int32_t* end,
                    void* out, int32_t* err, cudaStream_t s, bool stall = false) {
  MmParams p = params(c, cap, start, end, err);
  p.stall = stall;
  const int H = c->in_features, N = c->out_features, I = N / 2;
  const int features = c->gated ? kLanes : 2 * kLanes;
  p.M = c->gated ? I : N;
  p.depth = H;
  p.m_tiles = (p.M + features - 1) / features;
  p.out = static_cast<__nv_bfloat16*>(out);
  MmMaps maps;
  cudaError_t e;
  if (c->gated) {
    // 16 gate rows, the 16 up rows that belong to them, and so on: an epilogue
    // warp finds both in its lanes
    e = encode<5>(&maps.a, false, w,
                  {uint64_t(H), 16, 2, uint64_t(I / 16), uint64_t(c->num_experts)},
                  {uint64_t(H), uint64_t(I) * H, uint64_t(16) * H, uint64_t(N) * H},
                  {64, 16, 2, 4, 1});
  } else {
    e = encode_weights(&maps.a, false, w, c->num_experts, N, H, kLanes);
  }
  if (c->x_fp8) {
    p.xs = x_scale;
    p.x_width = H;
    for (int i = 1; i < 5 && e == cudaSuccess; ++i)
      e = encode_bytes(&maps.b[i], x, cap, H, kDepth, 8 << i);
  } else {
    for (int i = 0; i < 5 && e == cudaSuccess; ++i)
      e = encode_rows(&maps.b[i], x, cap, H, 8 << i);
  }
  if (e != cudaSuccess) return e;
  const int64_t items = most_row_tiles(num_rows, p.E, c->x_fp8) * p.m_tiles;
  const int64_t steps = (p.depth + kDepth - 1) / kDepth;
  if (c->gated)
    return c->x_fp8 ? launch<kForward, true, true, false>(maps, p, items, steps, s)
                    : launch<kForward, false, true, false>(maps, p, items, steps, s);
  return c->x_fp8 ? launch<kForward, true, false, false>(maps, p, items, steps, s)
                  : launch<kForward, false, false, false>(maps, p, items, steps, s);
}

cudaError_t by_rows(const ep_expert_config* c, int cap, int num_rows, const void* dy,
                    const void* w, const int32_t* start, const int32_t* end, void* dx,
                    int32_t* err, cudaStream_t s) {
  MmParams p = params(c, cap, start, end, err);
  p.M = c->in_features;
  p.depth = c->out_features;
  p.m_tiles = (p.M + 2 * kLanes - 1) / (2 * kLanes);
  p.out = static_cast<__nv_bfloat16*>(dx);
  MmMaps maps;
  cudaError_t e = encode_weights(&maps.a, false, w, c->num_experts, c->out_features,
                                 c->in_features, kDepth);
  for (int i = 0; i < 5 && e == cudaSuccess; ++i)
    e = encode_rows(&maps.b[i], dy, cap, c->out_features, 8 << i);
  if (e != cudaSuccess) return e;
  const int64_t items = most_row_tiles(num_rows, p.E, false) * p.m_tiles;
  const int64_t steps = (p.depth + kDepth - 1) / kDepth;
  return launch<kByRows, false, false, false>(maps, p, items, steps, s);
}

cudaError_t by_weights(const ep_expert_config* c, int cap, int num_rows, const void* dy, const void* x,
                       const float* x_scale, const int32_t* start, const int32_t* end, void* dw,
                       int type, int32_t* err, cudaStream_t s) {
  MmParams p = params(c, cap, start, end, err);
  const bool f32 = type != EP_GRAD_BF16;
  p.M = c->out_features;
  p.cols = c->in_features;
  p.m_tiles = (p.M + 2 * kLanes - 1) / (2 * kLanes);
  const int wide = rows_of(in_two_parts(kByWeights, c->x_fp8 != 0, f32));
  p.n_tiles = (p.cols + wide - 1) / wide;
  p.add = type == EP_GRAD_FP32_ADD;
  const int64_t size = int64_t(p.E) * p.M * p.cols * (f32 ? 4 : 2);
  // What does not stay in L2 until it is read goes first (256 matrices of 4096
  // x 7168: 3000 us, 2700 like this; kept instead 3360).
  p.leaves_l2 = size > kL2Bytes;
  if (cap == 0) return p.add ? cudaSuccess : cudaMemsetAsync(dw, 0, size, s);
  MmMaps maps;
  cudaError_t e = encode_rows(&maps.a, dy, cap, p.M, kDepth);
  if (e == cudaSuccess) e = encode_weights(&maps.out, f32, dw, p.E, p.M, p.cols, 32);
  if (c->x_fp8) {
    p.xs = x_scale;
    p.x_width = p.cols;
    if (e == cudaSuccess) e = encode_bytes(&maps.b[0], x, cap, p.cols, 128, kDepth);
  } else if (e == cudaSuccess) {
    e = encode_rows(&maps.b[0], x, cap, p.cols, kDepth);
  }
  if (e != cudaSuccess) return e;
  const int64_t items = int64_t(p.E) * p.m_tiles * p.n_tiles;
  const int64_t steps = int64_t(num_rows) / p.E / kDepth;
  if (f32)
    return c->x_fp8 ? launch<kByWeights, true, false, true>(maps, p, items, steps, s)
                    : launch<kByWeights, false, false, true>(maps, p, items, steps, s);
  return c->x_fp8 ? launch<kByWeights, true, false, false>(maps, p, items, steps, s)
                  : launch<kByWeights, false, false, false>(maps, p, items, steps, s);
}

}  // namespace
}  // namespace ep

using namespace ep;

extern "C" {

int32_t ep_expert_mm(const ep_expert_config* cfg, int32_t cap, int32_t num_rows, const void* d_x,
                     const float* d_x_scale, const void* d_w, const int32_t* d_expert_start,
                     const int32_t* d_expert_end, void* d_out, int32_t* d_err, void* stream) {
  if (!config_ok(cfg) || cap < 0 || num_rows < 0) return EP_ERR_INVALID_ARG;
  if (!aligned(d_w) || !aligned(d_expert_start) || !aligned(d_expert_end))
    return EP_ERR_INVALID_ARG;
  if (d_err != nullptr && !aligned(d_err)) return EP_ERR_INVALID_ARG;
  if (cap > 0 && (!aligned(d_x) || !aligned(d_out))) return EP_ERR_INVALID_ARG;
  if (cfg->x_fp8 ? cap > 0 && !aligned(d_x_scale) : d_x_scale != nullptr)
    return EP_ERR_INVALID_ARG;
  if (cap == 0 || num_rows == 0) return EP_OK;
  return status(forward(cfg, cap, num_rows, d_x, d_x_scale, d_w, d_expert_start, d_expert_end,
                        d_out, d_err, static_cast<cudaStream_t>(stream)));
}

int32_t ep_selftest_expert_timeout(const ep_expert_config* cfg, int32_t cap, int32_t num_rows,
                                   const void* d_x, const float* d_x_scale, const void* d_w,
                                   const int32_t* d_expert_start, const int32_t* d_expert_end,
                                   void* d_out, int32_t* d_err, void* stream) {
  if (!config_ok(cfg) || cap < 1 || num_rows < 1) return EP_ERR_INVALID_ARG;
  if (!aligned(d_w) || !aligned(d_expert_start) || !aligned(d_expert_end) || !aligned(d_x) ||
      !aligned(d_out) || !aligned(d_err))
    return EP_ERR_INVALID_ARG;
  if (cfg->x_fp8 ? !aligned(d_x_scale) : d_x_scale != nullptr) return EP_ERR_INVALID_ARG;
  return status(forward(cfg, cap, num_rows, d_x, d_x_scale, d_w, d_expert_start, d_expert_end,
                        d_out, d_err, static_cast<cudaStream_t>(stream), true));
}

int32_t ep_expert_mm_backward(const ep_expert_config* cfg, int32_t cap, int32_t num_rows,
                              const void* d_grad_out, const void* d_w, const void* d_x,
                              const float* d_x_scale, const int32_t* d_expert_start,
                              const int32_t* d_expert_end, void* d_grad_x, void* d_grad_w,
                              int32_t grad_w_type, int32_t* d_err, void* stream) {
  if (!config_ok(cfg) || cfg->gated || cap < 0 || num_rows < 0) return EP_ERR_INVALID_ARG;
  if (!aligned(d_expert_start) || !aligned(d_expert_end)) return EP_ERR_INVALID_ARG;
  if (d_err != nullptr && !aligned(d_err)) return EP_ERR_INVALID_ARG;
  if (cap > 0 && !aligned(d_grad_out)) return EP_ERR_INVALID_ARG;
  if (d_grad_x == nullptr && d_grad_w == nullptr) return EP_ERR_INVALID_ARG;
  if (d_grad_x != nullptr && (!aligned(d_grad_x) || !aligned(d_w))) return EP_ERR_INVALID_ARG;
  if (grad_w_type < EP_GRAD_BF16 || grad_w_type > EP_GRAD_FP32_ADD) return EP_ERR_INVALID_ARG;
  if (d_grad_w != nullptr) {
    if (!aligned(d_grad_w) || (cap > 0 && !aligned(d_x))) return EP_ERR_INVALID_ARG;
    if (cfg->x_fp8 ? cap > 0 && !aligned(d_x_scale) : d_x_scale != nullptr)
      return EP_ERR_INVALID_ARG;
  }
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  cudaError_t e = cudaSuccess;
  if (d_grad_x != nullptr && cap > 0 && num_rows > 0)
    e = by_rows(cfg, cap, num_rows, d_grad_out, d_w, d_expert_start, d_expert_end, d_grad_x, d_err,
                s);
  if (e == cudaSuccess && d_grad_w != nullptr)
    e = by_weights(cfg, cap, num_rows, d_grad_out, d_x, d_x_scale, d_expert_start, d_expert_end, d_grad_w,
                   grad_w_type, d_err, s);
  return status(e);
}

}  // extern "C"

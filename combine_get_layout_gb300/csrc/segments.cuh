// Experts' segments of a layout, as the kernels over all experts' rows use
// them: clipped to the rows that there are, and counted.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace ep {

// Rows [first, first + rows) of what [start, end) holds of [0, cap).  (Ends are
// compared, not subtracted, before they are clipped: an end far below its
// start would leave 32 bits, and come back as a large number of rows.)
__host__ __device__ __forceinline__ void clip_rows(int32_t start, int32_t end, int cap, int& first,
                                                   int& rows) {
  first = start < 0 ? 0 : start < cap ? start : cap;
  const int past = end < cap ? end : cap;
  rows = past > first ? past - first : 0;
}

// Rows [first, first + rows) of expert e among `cap`.
__device__ __forceinline__ void clip_segment(const int32_t* start, const int32_t* end, int cap,
                                             int e, int& first, int& rows) {
  clip_rows(__ldg(start + e), __ldg(end + e), cap, first, rows);
}

// table[e] = the sum of count(0..e-1), for e = 0..E, at most INT32_MAX (where
// it stops, segments overlap).  All threads of the CTA (whole warps, up to
// 1024) call; count(e) is called once for each e.  partial: 32 values of shared
// memory.  Ends with a barrier.
template <class F>
__device__ __forceinline__ void count_experts(int E, int* table, int64_t* partial, F&& count) {
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32, warps = blockDim.x / 32;
  int64_t before = 0;
  if (threadIdx.x == 0) table[0] = 0;
  for (int e0 = 0; e0 < E; e0 += blockDim.x) {
    const int e = e0 + threadIdx.x;
    int64_t v = e < E ? count(e) : 0;
#pragma unroll
    for (int o = 1; o < 32; o *= 2) {
      const int64_t u = __shfl_up_sync(0xffffffffu, v, o);
      if (lane >= o) v += u;
    }
    if (lane == 31) partial[warp] = v;
    __syncthreads();
    int64_t all = 0;
    for (int w = 0; w < warps; ++w) {
      const int64_t u = partial[w];
      if (w < warp) v += u;
      all += u;
    }
    if (e < E) table[e + 1] = int(min(before + v, int64_t(INT32_MAX)));
    before += all;
    __syncthreads();
  }
}

// The expert whose part of the table holds i: table[e] <= i < table[e + 1].
__device__ __forceinline__ int expert_of(const int* table, int E, int64_t i) {
  int lo = 0, hi = E;
  while (hi - lo > 1) {
    const int mid = (lo + hi) / 2;
    if (table[mid] <= i)
      lo = mid;
    else
      hi = mid;
  }
  return lo;
}

}  // namespace ep

// Tensor copies (TMA) and 5th-generation tensor core wrappers in inline PTX.
#pragma once

#include <cuda.h>

#include "ep_device.cuh"

namespace ep {

// True in one lane of a converged warp, always the same.  Around copies and
// products in a loop that the whole warp runs, it leaves their operands
// uniform; a loop that lane 0 runs alone took about 430 ns a stage.
__device__ __forceinline__ bool elect_one() {
  uint32_t one;
  asm volatile(
      "{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(one));
  return one != 0;
}

// ---- pairs of CTAs (in clusters of one or more pairs) ------------------------------------------

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}

// The address, in the cluster's shared memory, of what lies at `addr` in the
// CTA of this rank.
__device__ __forceinline__ uint32_t at_rank(uint32_t addr, uint32_t rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
  return r;
}

// All threads of both CTAs.
__device__ __forceinline__ void cluster_sync() {
  __syncwarp();
  asm volatile(
      "barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::
          : "memory");
}

// Arrives on a barrier of either CTA (address from at_rank).  What the
// arrival hands over is ordered by fences of its own: tc_fence_before for
// tensor memory, fence_async_shared for operands in shared memory.  Those lie
// in the arriving CTA's shared memory, which is the one place they are at and
// where that CTA's tensor cores read them: the fence ends when they are there,
// and the arrival, which comes after it, is all that leaves for the other CTA.
// No cache lies between, for which a scope wider than the CTA would matter;
// PTX's own text promises it at cluster scope alone.  (With a release of
// cluster scope on every arrival each waited for the thread's memory
// operations, about 1 us: every case ran at half its speed.
// On operands' arrivals alone, with an acquire of cluster scope behind them:
// 128 tokens by 256 experts of 4096 x 7168, E4M3 rows, 2060 -> 3240 us,
// 64 experts of 768 rows 1460 -> 2320, gradients of 4096 tokens 4840 -> 5550.)
__device__ __forceinline__ void mbar_arrive_cluster(uint32_t bar) {
  asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}

// The same, handing over what the warp wrote before to a CTA of the cluster
// that waits by mbar_wait_acquire.
__device__ __forceinline__ void mbar_arrive_release(uint32_t bar) {
  asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar)
               : "memory");
}

__device__ __forceinline__ bool mbar_wait_acquire(uint64_t* bar, uint32_t parity,
                                                  uint64_t timeout_ns) {
  const bool ok = mbar_wait(bar, parity, timeout_ns);
  asm volatile("fence.acq_rel.cluster;" ::: "memory");
  return ok;
}

// 16 bytes of a CTA's shared memory (address from at_rank).
__device__ __forceinline__ uint4 load_cluster(uint32_t at) {
  uint4 v;
  asm volatile("ld.shared::cluster.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(at)
               : "memory");
  return v;
}

// ---- tensor copies ----------------------------------------------------------
// Global -> this CTA's shared memory of one box at the given coordinates,
// innermost first; completion counted on `bar`, which may be the other CTA's
// of the pair (address from at_rank).  Parts outside the tensor read as zeros
// and count.  The innermost coordinate times the element size is a multiple
// of 16.

__device__ __forceinline__ void prefetch_map(const CUtensorMap* m) {
  asm volatile("prefetch.tensormap [%0];" ::"l"(m) : "memory");
}

__device__ __forceinline__ void tma_load_2d(uint32_t dst, const CUtensorMap* m, uint32_t bar,
                                            int c0, int c1) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      ".cta_group::2 [%0], [%1, {%3, %4}], [%2];" ::"r"(dst),
      "l"(m), "r"(bar), "r"(c0), "r"(c1)
      : "memory");
}

__device__ __forceinline__ void tma_load_3d(uint32_t dst, const CUtensorMap* m, uint32_t bar,
                                            int c0, int c1, int c2) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      ".cta_group::2 [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(dst),
      "l"(m), "r"(bar), "r"(c0), "r"(c1), "r"(c2)
      : "memory");
}

__device__ __forceinline__ void tma_load_5d(uint32_t dst, const CUtensorMap* m, uint32_t bar,
                                            int c0, int c1, int c2, int c3, int c4) {
  asm volatile(
      "cp.async.bulk.tensor.5d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      ".cta_group::2 [%0], [%1, {%3, %4, %5, %6, %7}], [%2];" ::"r"(dst),
      "l"(m), "r"(bar), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(c4)
      : "memory");
}

// How long L2 keeps what a store writes.
__device__ __forceinline__ uint64_t l2_policy(bool leaves_first) {
  uint64_t first, normal;
  asm("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(first));
  asm("createpolicy.fractional.L2::evict_normal.b64 %0, 1.0;" : "=l"(normal));
  return leaves_first ? first : normal;
}

// Shared -> global; what lies outside the tensor is not written.
__device__ __forceinline__ void tma_store_3d(const CUtensorMap* m, uint32_t src, int c0, int c1,
                                             int c2, uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.3d.global.shared::cta.tile.bulk_group.L2::cache_hint "
      "[%0, {%2, %3, %4}], [%1], %5;" ::"l"(m),
      "r"(src), "r"(c0), "r"(c1), "r"(c2), "l"(policy)
      : "memory");
}

// Added to what is there.
__device__ __forceinline__ void tma_add_3d(const CUtensorMap* m, uint32_t src, int c0, int c1,
                                           int c2) {
  asm volatile(
      "cp.reduce.async.bulk.tensor.3d.global.shared::cta.add.tile.bulk_group "
      "[%0, {%2, %3, %4}], [%1];" ::"l"(m),
      "r"(src), "r"(c0), "r"(c1), "r"(c2)
      : "memory");
}

__device__ __forceinline__ void tma_store_commit() {
  asm volatile("cp.async.bulk.commit_group;" ::: "memory");
}
// All but the newest N groups of the calling thread have read their source.
template <int N>
__device__ __forceinline__ void tma_store_wait_read() {
  asm volatile("cp.async.bulk.wait_group.read %0;" ::"n"(N) : "memory");
}
template <int N>
__device__ __forceinline__ void tma_store_wait() {
  asm volatile("cp.async.bulk.wait_group %0;" ::"n"(N) : "memory");
}

// Orders this thread's shared-memory writes before later reads by copies and
// tensor cores.
__device__ __forceinline__ void fence_async_shared() {
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}

// ---- tensor cores, used by pairs ------------------------------------------------

// All 32 lanes of a warp in each CTA of the pair; the address of `cols` (a
// power of two, 32 to 512) columns of tensor memory goes to *at (shared).
// Waits until they are free.
__device__ __forceinline__ void tmem_alloc(uint32_t* at, uint32_t cols) {
  asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                   smem_addr(at)),
               "r"(cols)
               : "memory");
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;");
}
__device__ __forceinline__ void tmem_free(uint32_t addr, uint32_t cols) {
  asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(addr), "r"(cols));
}

__device__ __forceinline__ void tc_fence_before() {
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void tc_fence_after() {
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
}

// Descriptor of a shared operand in 128-byte swizzle (1024-byte aligned rows
// of 128 bytes): `lead` and `stride` are the byte offsets of the layout.
//   inner dimension = reduction: 8-row groups every `stride` bytes, lead unused
//   inner dimension = rows of the product: 64-wide panels every `lead` bytes,
//   groups of 8 along the reduction every `stride` bytes
__device__ __forceinline__ uint64_t smem_desc(uint32_t addr, uint32_t lead, uint32_t stride) {
  return uint64_t((addr & 0x3ffff) >> 4) | uint64_t(lead >> 4) << 16 |
         uint64_t(stride >> 4) << 32 | uint64_t(1) << 46 | uint64_t(2) << 61;
}

// Instruction descriptor: bf16 operands, fp32 accumulation, M x N; ta, tb:
// operand's inner dimension is not the reduction.
__host__ __device__ constexpr uint32_t instr_desc(int m, int n, bool ta, bool tb) {
  return 1u << 4 | 1u << 7 | 1u << 10 | uint32_t(ta) << 15 | uint32_t(tb) << 16 |
         uint32_t(n / 8) << 17 | uint32_t(m / 16) << 24;
}

// D (tensor memory) = A B (+ D), 16 of the reduction, by one thread of the
// first CTA: each CTA holds half of A's and half of B's rows at the
// descriptors' addresses, and its half of D's rows for all columns.
__device__ __forceinline__ void mma_bf16(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                         bool add) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(uint32_t(add))
      : "memory");
}

// Arrives on the barriers at this place in both CTAs, the first of which has
// this rank in the cluster, when this thread's products so far are done.
__device__ __forceinline__ void mma_commit(uint32_t bar, uint32_t lead) {
  asm volatile(
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 "
      "[%0], %1;" ::"r"(bar),
      "h"(uint16_t(3u << lead))
      : "memory");
}

__device__ __forceinline__ void tmem_wait_load() {
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
}

// 16 lanes by 32 columns: register 4 j + i holds lane l / 4 + 8 (i / 2), column
// 8 j + 2 (l % 4) + i % 2 in thread l.
__device__ __forceinline__ void tmem_load_16x32(uint32_t at, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x4.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15])
      : "r"(at));
}

// 32 lanes by 32 columns: thread l holds lane l.
__device__ __forceinline__ void tmem_load_32x32(uint32_t at, uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]),
        "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]),
        "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(at));
}

// Four 8x8 matrices of 16-bit values, transposed: thread l's register m holds
// (l / 4, 2 (l % 4)) and its neighbour of matrix m; column i of matrix m goes
// to the 16 bytes that thread 8 m + i addresses.
__device__ __forceinline__ void stmatrix_t4(uint32_t at, uint32_t a, uint32_t b, uint32_t c,
                                            uint32_t d) {
  asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(at),
               "r"(a), "r"(b), "r"(c), "r"(d)
               : "memory");
}

}  // namespace ep

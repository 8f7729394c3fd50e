// gs_tcgen05.cuh -- the PTX of the tensor-core kernels for one CTA or a pair of
// CTAs (cta_group 1 or 2): barriers with bounded waits, TMA loads and stores,
// tensor memory, and the descriptors of shared-memory operands.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "gs_device.cuh"
#include "gs_elem.cuh"

namespace gs {

constexpr uint64_t kTcWaitNs = 2000000000ull;

__device__ __forceinline__ uint32_t tc_smem(const void* p) {
  return (uint32_t)__cvta_generic_to_shared(p);
}
// True in one lane of a whole warp.  Roles run as whole warps up to the
// instructions of one lane: loop counters, addresses and descriptors then stay
// in uniform registers, where a role of a single lane makes the compiler move
// every operand there for each instruction (50 to 70 cycles each).
__device__ __forceinline__ bool tc_elect() {
  uint32_t p;
  asm volatile(
      "{\n\t.reg .pred p;\n\telect.sync _|p, 0xFFFFFFFF;\n\tselp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(p));
  return p != 0;
}
__device__ __forceinline__ uint64_t tc_now() {
  uint64_t t;
  asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t));
  return t;
}
__device__ __forceinline__ bool tc_try_wait(uint64_t* bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(tc_smem(bar)), "r"(parity)
      : "memory");
  return ok != 0;
}
// Bounded wait; gives up on timeout (setting the abort flag and the status) or
// when another role of this CTA has given up.
__device__ __forceinline__ bool tc_wait(uint64_t* bar, uint32_t parity, volatile int* abort_flag,
                                        int32_t* status) {
  if (tc_try_wait(bar, parity)) return true;
  const uint64_t t0 = tc_now();
  while (!tc_try_wait(bar, parity)) {
    if (*abort_flag) return false;
    if (tc_now() - t0 > kTcWaitNs) {
      *abort_flag = 1;
      atomicExch(status, (int32_t)GS_ERR_TIMEOUT);
      return false;
    }
  }
  return true;
}
// The same where other CTAs of the cluster wrote what the barrier tells of.
__device__ __forceinline__ bool tc_try_wait_cluster(uint64_t* bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(tc_smem(bar)), "r"(parity)
      : "memory");
  return ok != 0;
}
__device__ __forceinline__ bool tc_wait_cluster(uint64_t* bar, uint32_t parity, volatile int* abort_flag,
                                                int32_t* status) {
  return tc_wait(bar, parity, abort_flag, status) && tc_try_wait_cluster(bar, parity);
}
// The same for a whole warp, which goes on or gives up together.
__device__ __forceinline__ bool tc_wait_warp(uint64_t* bar, uint32_t parity, volatile int* abort_flag,
                                             int32_t* status) {
  return __all_sync(0xFFFFFFFFu, tc_wait(bar, parity, abort_flag, status));
}
// Bounded wait for work in flight that does not look at the abort flag.
__device__ __forceinline__ void tc_drain(uint64_t* bar, uint32_t parity) {
  const uint64_t t0 = tc_now();
  while (!tc_try_wait(bar, parity))
    if (tc_now() - t0 > kTcWaitNs) return;
}
__device__ __forceinline__ void tc_bar_init(uint64_t* bar, uint32_t count) {
  asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(tc_smem(bar)), "r"(count) : "memory");
}
__device__ __forceinline__ void tc_expect(uint64_t* bar, uint32_t bytes) {
  asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(tc_smem(bar)), "r"(bytes)
               : "memory");
}
__device__ __forceinline__ void tc_arrive(uint64_t* bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(tc_smem(bar)) : "memory");
}
// Arrives at the barrier at bar's place in CTA `rank` of the cluster.
__device__ __forceinline__ void tc_arrive_at(uint64_t* bar, uint32_t rank) {
  asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(remote(bar, rank))
               : "memory");
}

// The shared::cluster address of p's place in the pair's leading CTA (for one CTA,
// of its own).
template <int CG>
__device__ __forceinline__ uint32_t tc_leader(const void* p) {
  return CG == 2 ? remote(p, cluster_rank() & ~1u) : tc_smem(p);
}
// Tile loads into this CTA whose bytes are counted by `bar`, a shared::cluster
// address (the leading CTA's barrier for a pair).
template <int CG>
__device__ __forceinline__ void tc_load2(const CUtensorMap* map, uint32_t bar, void* dst, int32_t x,
                                         int32_t y) {
  if constexpr (CG == 2)
    asm volatile(
        "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3}], [%4];" ::"r"(tc_smem(dst)),
        "l"(map), "r"(x), "r"(y), "r"(bar)
        : "memory");
  else
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3}], [%4];" ::"r"(tc_smem(dst)),
        "l"(map), "r"(x), "r"(y), "r"(bar)
        : "memory");
}
template <int CG>
__device__ __forceinline__ void tc_load3(const CUtensorMap* map, uint32_t bar, void* dst, int32_t x,
                                         int32_t y, int32_t z) {
  if constexpr (CG == 2)
    asm volatile(
        "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(tc_smem(dst)),
        "l"(map), "r"(x), "r"(y), "r"(z), "r"(bar)
        : "memory");
  else
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(tc_smem(dst)),
        "l"(map), "r"(x), "r"(y), "r"(z), "r"(bar)
        : "memory");
}
__device__ __forceinline__ void tc_store2(const CUtensorMap* map, const void* src, int32_t x, int32_t y) {
  asm volatile(
      "cp.async.bulk.tensor.2d.global.shared::cta.tile.bulk_group [%0, {%1, %2}], [%3];" ::"l"(map),
      "r"(x), "r"(y), "r"(tc_smem(src))
      : "memory");
}

// ---- tensor memory --------------------------------------------------------------
__device__ __forceinline__ void tc_before() {
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void tc_after() {
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
}
// By one whole warp (of each CTA of a pair).
template <int CG>
__device__ __forceinline__ void tc_alloc(uint32_t* slot, uint32_t cols) {
  if constexpr (CG == 2) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(tc_smem(slot)),
                 "r"(cols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  } else {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(tc_smem(slot)),
                 "r"(cols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
}
template <int CG>
__device__ __forceinline__ void tc_dealloc(uint32_t tmem, uint32_t cols) {
  if constexpr (CG == 2)
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(cols) : "memory");
  else
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(cols) : "memory");
}
// Arrives at bar (of both CTAs of a pair) when every MMA and copy issued before
// by this thread is done.
template <int CG>
__device__ __forceinline__ void tc_commit(uint64_t* bar) {
  if constexpr (CG == 2)
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::
            "r"(tc_smem(bar)),
        "h"((uint16_t)(3u << (cluster_rank() & ~1u)))
        : "memory");
  else
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(
                     tc_smem(bar))
                 : "memory");
}

// 32 lanes x 32 consecutive columns of 32 bits -> 32 registers per thread,
// readable after tc_wait_ld.
__device__ __forceinline__ void tc_ld32(uint32_t taddr, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]),
        "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]),
        "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr));
}
// Waits for this thread's tcgen05.ld; n registers (a multiple of 32) are passed
// through, so that nothing reads them before.
template <int N>
__device__ __forceinline__ void tc_wait_ld(uint32_t* r) {
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
  for (int i = 0; i < N; i += 8)
    asm volatile(""
                 : "+r"(r[i]), "+r"(r[i + 1]), "+r"(r[i + 2]), "+r"(r[i + 3]), "+r"(r[i + 4]),
                   "+r"(r[i + 5]), "+r"(r[i + 6]), "+r"(r[i + 7])
                 :
                 : "memory");
}

// ---- shared-memory operands ---------------------------------------------------------
// Rows of 128 bytes in the 128-byte swizzle that TMA writes, sum dimension along
// the row: 8-row groups 1024 bytes apart, descriptor version 1.
__device__ __forceinline__ uint64_t tc_desc_k(uint32_t saddr) {
  return (uint64_t)((saddr >> 4) & 0x3FFFu) | (1ull << 16) | ((uint64_t)(1024 >> 4) << 32) |
         (1ull << 46) | (2ull << 61);
}
// Scales of 32 rows of 16 bytes, unswizzled: 8-row groups 128 bytes apart.
__device__ __forceinline__ uint64_t tc_desc_scales(uint32_t saddr) {
  return (uint64_t)((saddr >> 4) & 0x3FFFu) | (1ull << 16) | ((uint64_t)(128 >> 4) << 32) | (1ull << 46);
}

// Tile t of a raster that takes `group` tile rows at a time, so that consecutive
// tiles share panels of both operands.
__device__ __forceinline__ void tc_tile(int t, int group, int tiles_m, int tiles_n, int& mt, int& nt) {
  const int per_group = group * tiles_n;
  const int first = (t / per_group) * group;
  const int rows = min(group, tiles_m - first);
  const int r = t % per_group;
  mt = first + r % rows;
  nt = r / rows;
}

}  // namespace gs

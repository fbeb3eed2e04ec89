// tensor.cuh -- tensor-core and tensor-copy helpers (sm_100a): shared-memory
// and instruction descriptors, tcgen05 issue and read-back, tiled bulk copies, and the bounded waits of a warp-specialised kernel.
#pragma once
#include <cuda.h>

#include "common.cuh"

namespace moe {

// ------------------------------------------------------------- descriptors
// Operand tile in shared memory, 128-byte swizzle.  K-major: rows of 64 bf16
// (128 bytes), 8-row groups 1024 bytes apart (the stride offset); a K step of
// 16 is 32 bytes further.  MN-major: for each k a row of 64 channels (128
// bytes), groups of 8 k 1024 bytes apart (the stride offset), blocks of 64
// channels `lead` bytes apart (the leading offset); a K step of 16 is 2048
// bytes further.
__device__ __forceinline__ uint64_t tile_desc(uint32_t addr, uint32_t lead) {
  return (uint64_t)((addr & 0x3ffffu) >> 4) | ((uint64_t)(lead >> 4) << 16) | ((uint64_t)(1024u >> 4) << 32) |
         (1ull << 46) | (2ull << 61);
}
// bf16 x bf16 -> fp32, A of m rows (mn_major_a: stored MN-major), B of n rows, K-major.
__device__ __forceinline__ uint32_t mma_desc(int m, int n, bool mn_major_a) {
  return (1u << 4) | (1u << 7) | (1u << 10) | (mn_major_a ? 1u << 15 : 0u) | ((uint32_t)(n >> 3) << 17) |
         ((uint32_t)(m >> 4) << 24);
}

// ----------------------------------------------------------------- tcgen05
// All of these act on a pair of CTAs (a cluster of two): each holds half of
// A's rows, half of B's and the accumulator of its own rows of A; one thread
// of the pair's first CTA issues.  What one thread issues is called by its
// whole warp and issued by the lane that elect.sync names (always the same):
// under `if (lane == 0)` the operands are not known to be the warp's, and an
// issue took 78 cycles, so that a stage of four products took 800.
__device__ __forceinline__ void mma_bf16(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool add) {
  asm volatile(
      "{\n .reg .pred p, e;\n setp.ne.b32 p, %4, 0;\n elect.sync _|e, 0xffffffff;\n @e "
      "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"((uint32_t)add)
      : "memory");
}
// Arrives on `bar` of both CTAs when the MMAs this warp issued so far have completed.
__device__ __forceinline__ void mma_commit(uint64_t* bar) {
  asm volatile(
      "{\n .reg .pred e;\n elect.sync _|e, 0xffffffff;\n @e "
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;\n}" ::"r"(
          smem_u32(bar)),
      "h"((uint16_t)3)
      : "memory");
}
__device__ __forceinline__ void tmem_alloc(uint32_t* slot, uint32_t cols) {
  asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(slot)), "r"(cols)
               : "memory");
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_free(uint32_t addr, uint32_t cols) {
  asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(addr), "r"(cols) : "memory");
}
__device__ __forceinline__ void tc_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
// 32 columns of this warp's 32 lanes: v[j] = column j of this thread's lane.
__device__ __forceinline__ void tmem_ld32(uint32_t addr, float (&v)[32]) {
  uint32_t* r = reinterpret_cast<uint32_t*>(v);
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
        "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
        "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(addr));
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
}

// -------------------------------------------------------------- bulk copies
__device__ __forceinline__ void tma_prefetch(const CUtensorMap* m) {
  asm volatile("prefetch.tensormap [%0];" ::"l"(m) : "memory");
}
// Tiled copies into this CTA's shared memory that complete on `bar`, a
// shared::cluster address in either CTA of the pair (called by a whole warp).
__device__ __forceinline__ void tma_2d(void* dst, const CUtensorMap* m, int x, int y, uint32_t bar) {
  asm volatile(
      "{\n .reg .pred e;\n elect.sync _|e, 0xffffffff;\n @e "
      "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, "
      "%3}], [%4];\n}" ::"r"(smem_u32(dst)),
      "l"(m), "r"(x), "r"(y), "r"(bar)
      : "memory");
}
__device__ __forceinline__ void tma_3d(void* dst, const CUtensorMap* m, int x, int y, int z, uint32_t bar) {
  asm volatile(
      "{\n .reg .pred e;\n elect.sync _|e, 0xffffffff;\n @e "
      "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, "
      "%3, %4}], [%5];\n}" ::"r"(smem_u32(dst)),
      "l"(m), "r"(x), "r"(y), "r"(z), "r"(bar)
      : "memory");
}
// Arrives once and raises the phase's transaction count (called by a whole warp).
__device__ __forceinline__ void mbar_expect(uint64_t* bar, uint32_t bytes) {
  asm volatile(
      "{\n .reg .pred e;\n elect.sync _|e, 0xffffffff;\n @e mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;\n}" ::"r"(
          smem_u32(bar)),
      "r"(bytes)
      : "memory");
}
// 16 bytes global -> shared, or zeros (`in` false: nothing is read), where `on`.
__device__ __forceinline__ void cp_async16_if(uint32_t dst, const void* src, bool in, bool on) {
  asm volatile("{\n .reg .pred p;\n setp.ne.b32 p, %3, 0;\n @p cp.async.cg.shared.global [%0], [%1], 16, %2;\n}" ::"r"(dst),
               "l"(src), "r"(in ? 16 : 0), "r"((uint32_t)on)
               : "memory");
}
// Arrives on `bar` (one of its expected arrivals) when this thread's copies so far have completed.
__device__ __forceinline__ void cp_async_arrive(uint64_t* bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
}
__device__ __forceinline__ void cp_async_wait_all() { asm volatile("cp.async.wait_all;" ::: "memory"); }

// Stores and loads under a predicate: unrolled runs of them stay free of branches.
__device__ __forceinline__ void st32_if(void* p, uint32_t v, bool on) {
  asm volatile("{\n .reg .pred p;\n setp.ne.b32 p, %2, 0;\n @p st.global.b32 [%0], %1;\n}" ::"l"(p), "r"(v),
               "r"((uint32_t)on)
               : "memory");
}
__device__ __forceinline__ void st16_if(void* p, uint16_t v, bool on) {
  asm volatile("{\n .reg .pred p;\n setp.ne.b32 p, %2, 0;\n @p st.global.b16 [%0], %1;\n}" ::"l"(p), "h"(v),
               "r"((uint32_t)on)
               : "memory");
}
__device__ __forceinline__ uint32_t ld32_if(const void* p, bool on) {
  uint32_t v;
  asm volatile("{\n .reg .pred p;\n setp.ne.b32 p, %2, 0;\n mov.b32 %0, 0;\n @p ld.global.cg.b32 %0, [%1];\n}"
               : "=r"(v)
               : "l"(p), "r"((uint32_t)on)
               : "memory");
  return v;
}

// ------------------------------------------------------------ bounded waits
// Arrives on `bar`, a shared::cluster address of this CTA or its pair, with
// the default release at CTA scope.  Nothing that the other CTA's threads read
// or write is published by it: what it announces stays in this CTA's shared
// memory or TMEM and is read there by this SM's tensor cores (behind a proxy
// or tcgen05 fence of the arriving thread).  A release at cluster scope would
// also wait for every global access in flight, 1.1 us each time.
__device__ __forceinline__ void mbar_arrive_at(uint32_t bar) {
  asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}
// The address of this CTA's `p` in CTA `rank` of the cluster.
__device__ __forceinline__ uint32_t peer_u32(const void* p, int rank) {
  uint32_t r;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(smem_u32(p)), "r"(rank));
  return r;
}
__device__ __forceinline__ bool mbar_try_wait_cluster(uint64_t* bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n .reg .pred p;\n mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2, %3;\n selp.u32 %0, 1, 0, "
      "p;\n}"
      : "=r"(ok)
      : "r"(smem_u32(bar)), "r"(parity), "r"(100000u)
      : "memory");
  return ok != 0;
}
// The same for a whole warp: true for all lanes or for none.
__device__ __forceinline__ bool wait_or_stop(uint64_t* bar, uint32_t parity, volatile int* stop, uint32_t* err);
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, volatile int* stop, uint32_t* err) {
  return __all_sync(0xffffffffu, wait_or_stop(bar, parity, stop, err));
}
// Waits for a phase; gives up (false) after kWaitLimitNs, recording the
// timeout, or as soon as another role of the CTA has given up.
__device__ __forceinline__ bool wait_or_stop(uint64_t* bar, uint32_t parity, volatile int* stop, uint32_t* err) {
  if (mbar_try_wait_cluster(bar, parity)) return true;
  const unsigned long long t0 = global_ns();
  while (!mbar_try_wait_cluster(bar, parity)) {
    if (*stop) return false;
    if (global_ns() - t0 > kWaitLimitNs) {
      *stop = 1;
      atomicOr(err, kErrCopyTimeout);
      return false;
    }
  }
  return true;
}
// A barrier of `threads` threads that tells each whether any of them says so.
__device__ __forceinline__ bool bar_any(int id, int threads, bool say) {
  uint32_t r;
  asm volatile(
      "{\n .reg .pred p, q;\n setp.ne.b32 p, %1, 0;\n barrier.cta.red.or.pred q, %2, %3, p;\n selp.u32 %0, 1, 0, q;\n}"
      : "=r"(r)
      : "r"((uint32_t)say), "r"(id), "r"(threads)
      : "memory");
  return r != 0;
}

// ------------------------------------------------------------ host: tensor maps
// bf16 matrices [z][y][x] with row and matrix strides in bytes (multiples of
// 16), 128-byte swizzle, zeros outside.  Returns false on failure.
bool tensor_map(CUtensorMap* m, const void* base, uint64_t x, uint64_t y, uint64_t z, uint64_t row_bytes,
                uint64_t mat_bytes, uint32_t box_x, uint32_t box_y, uint32_t box_z = 1);

}  // namespace moe

// device.cuh -- sm_100a building blocks shared by the kernels of this library:
// mbarriers with bounded waits, TMA tile loads, tcgen05 (TMEM alloc, MMA,
// commit, loads) and the fp8 cast/decode instructions.  Hand-written inline
// PTX; nothing here is taken from a vendor library.
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

namespace fp8lin {

// Status codes written to the device status word (mirror fp8_status).
constexpr int kDevTimeout = -5;

// A wait gives up after this many nanoseconds of %globaltimer.
#ifndef FP8LIN_WAIT_LIMIT_NS
#define FP8LIN_WAIT_LIMIT_NS 2000000000ull
#endif

__device__ __forceinline__ uint32_t smem_u32(const void* p) {
  return static_cast<uint32_t>(__cvta_generic_to_shared(p));
}

__device__ __forceinline__ uint64_t globaltimer_ns() {
  uint64_t t;
  asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t));
  return t;
}

// ---------------------------------------------------------------- dependent launch
// Programmatic dependent launch: kernels are launched with programmatic stream
// serialization, start their prologue while the previous kernel drains, and
// wait for it (its completion and memory flush) before touching global data.
__device__ __forceinline__ void pdl_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void pdl_trigger() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

// ---------------------------------------------------------------- mbarrier

__device__ __forceinline__ void mbar_init(uint64_t* bar, uint32_t count) {
  asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(smem_u32(bar)), "r"(count) : "memory");
}

__device__ __forceinline__ void fence_mbar_init() {
  asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
}

__device__ __forceinline__ void mbar_arrive(uint64_t* bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_u32(bar)) : "memory");
}

__device__ __forceinline__ void mbar_arrive_expect_tx(uint64_t* bar, uint32_t bytes) {
  asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(smem_u32(bar)), "r"(bytes)
               : "memory");
}

// try_wait with acquire at cluster scope: for barriers that other CTAs of the
// cluster arrive on (release.cluster) after writing shared memory this CTA
// then reads through distributed shared memory.
__device__ __forceinline__ bool mbar_try_wait_acq_cluster(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok != 0;
}

__device__ __forceinline__ bool mbar_try_wait(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok != 0;
}

// Wait until the phase with the given parity has completed.  Bounded: returns
// false (and records a timeout in *status) after FP8LIN_WAIT_LIMIT_NS, or as
// soon as *abort becomes nonzero (another role of the CTA gave up).  status and
// abort may be NULL.  kCluster: acquire at cluster scope (see above).
template <bool kCluster = false>
__device__ __forceinline__ bool mbar_wait(uint64_t* bar, uint32_t parity, int* status,
                                          volatile int* abort, uint64_t limit_ns = FP8LIN_WAIT_LIMIT_NS) {
  const uint32_t a = smem_u32(bar);
  auto probe = [&]() { return kCluster ? mbar_try_wait_acq_cluster(a, parity) : mbar_try_wait(a, parity); };
  #pragma unroll 1
  for (int i = 0; i < 64; ++i)
    if (probe()) return true;
  const uint64_t t0 = globaltimer_ns();
  #pragma unroll 1
  while (true) {
    #pragma unroll 1
    for (int i = 0; i < 256; ++i)
      if (probe()) return true;
    if (abort && *abort) return false;
    if (globaltimer_ns() - t0 > limit_ns) {
      if (status) atomicExch(status, kDevTimeout);
      if (abort) *abort = 1;
      return false;
    }
  }
}

// mbar_wait whose probes let the hardware suspend the warp for up
// to a millisecond until the phase completes.  Without the hint a waiting warp
// probes again and again; eight epilogue warps doing so through a mainloop
// cost issue slots and, at the power limit, clock.
__device__ __forceinline__ bool mbar_await(uint64_t* bar, uint32_t parity, int* status, volatile int* abort,
                                           uint64_t limit_ns = FP8LIN_WAIT_LIMIT_NS) {
  const uint32_t a = smem_u32(bar);
  auto probe = [&]() {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(a), "r"(parity), "r"(1000000u)
        : "memory");
    return ok != 0;
  };
  if (probe()) return true;
  const uint64_t t0 = globaltimer_ns();
  #pragma unroll 1
  while (true) {
    #pragma unroll 1
    for (int i = 0; i < 64; ++i)
      if (probe()) return true;
    if (abort && *abort) return false;
    if (globaltimer_ns() - t0 > limit_ns) {
      if (status) atomicExch(status, kDevTimeout);
      if (abort) *abort = 1;
      return false;
    }
  }
}

// Barriers of two warps (64 threads), the second with a vote.
__device__ __forceinline__ void duo_sync(int id) { asm volatile("barrier.sync %0, 64;" ::"r"(id) : "memory"); }
__device__ __forceinline__ bool duo_all(int id, bool v) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.u32 p, %1, 0;\n\t"
      "barrier.red.and.pred q, %2, 64, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"(static_cast<uint32_t>(v)), "r"(id)
      : "memory");
  return r != 0;
}

// mbar_await by two warps that barriers of 64 threads join: true for all of
// their threads or for none, so that neither is left at such a barrier alone.
__device__ __forceinline__ bool duo_await(int id, uint64_t* bar, uint32_t parity, int* status, volatile int* abort,
                                          uint64_t limit_ns = FP8LIN_WAIT_LIMIT_NS) {
  return duo_all(id, mbar_await(bar, parity, status, abort, limit_ns));
}

// Called by one thread behind a block's last barrier.  If a wait of the block
// gave up, copies it started (or another block of its cluster started for it)
// may still be on their way to its shared memory: they take microseconds, and
// get kSettleNs, before the memory is another block's.  A block that did not
// give up has seen all of its copies land.
constexpr uint64_t kSettleNs = 10000000;
__device__ __forceinline__ void settle_copies(const volatile int* abort) {
  if (!*abort) return;
  const uint64_t t0 = globaltimer_ns();
  while (globaltimer_ns() - t0 < kSettleNs) __nanosleep(1000);
}

// ---------------------------------------------------------------- TMA

__device__ __forceinline__ void prefetch_tmap(const CUtensorMap* m) {
  asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(m)) : "memory");
}

// 3-D (inner, outer, batch) tiled bulk tensor load global -> shared (this CTA), completion counted
// in bytes on `bar`.  Each load fills only the issuing CTA's shared memory.
__device__ __forceinline__ void tma_load_3d(void* dst, const CUtensorMap* m, uint64_t* bar, int32_t x,
                                            int32_t y, int32_t z) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(m)), "r"(smem_u32(bar)), "r"(x), "r"(y), "r"(z)
      : "memory");
}

// 3-D (column, row, batch) tiled bulk tensor store shared (this CTA) ->
// global, tracked as a bulk group of the issuing thread.  Rows/columns outside
// the tensor are clipped.
__device__ __forceinline__ void tma_store_3d(const CUtensorMap* m, const void* src, int32_t x, int32_t y, int32_t z) {
  asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.bulk_group [%0, {%2, %3, %4}], [%1];" ::"l"(
                   reinterpret_cast<uint64_t>(m)),
               "r"(smem_u32(src)), "r"(x), "r"(y), "r"(z)
               : "memory");
}
// Asynchronous L2 prefetch of a global byte range (16-byte aligned address,
// size a multiple of 16).  Only a hint; L2 is the point of coherence, so a
// line fetched early is updated by any later write to it.
__device__ __forceinline__ void prefetch_l2_bulk(const void* src, uint32_t bytes) {
  asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(reinterpret_cast<uint64_t>(src)), "r"(bytes)
               : "memory");
}

// Bulk copy from this CTA's shared memory into another CTA's of the cluster
// (dst and bar from mapa_shared), completion counted in bytes on bar.  Both
// addresses 16-byte aligned, bytes a multiple of 16.  No multicast.
__device__ __forceinline__ void bulk_copy_to_cluster(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.shared::cta.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
      "r"(smem_u32(src)), "r"(bytes), "r"(bar)
      : "memory");
}

__device__ __forceinline__ void bulk_commit() { asm volatile("cp.async.bulk.commit_group;" ::: "memory"); }
// Wait until at most N committed bulk groups still read their shared source.
template <int N>
__device__ __forceinline__ void bulk_wait_read() {
  asm volatile("cp.async.bulk.wait_group.read %0;" ::"n"(N) : "memory");
}
// Order this thread's generic-proxy shared-memory writes before later
// async-proxy (TMA) reads of them.
__device__ __forceinline__ void fence_proxy_async_smem() {
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}

// ---------------------------------------------------------------- tcgen05

__device__ __forceinline__ void tmem_alloc(uint32_t* dst_smem, uint32_t ncols) {
  asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(dst_smem)),
               "r"(ncols)
               : "memory");
}
__device__ __forceinline__ void tmem_relinquish() {
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_dealloc(uint32_t taddr, uint32_t ncols) {
  asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(ncols) : "memory");
}
__device__ __forceinline__ void tc_fence_before() {
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void tc_fence_after() {
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
}

// D(tmem) (+)= A(smem desc) x B(smem desc), fp8/fp6/fp4 kind, fp32 accumulate.
__device__ __forceinline__ void umma_f8f6f4(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                            uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}

// Arrive once on `bar` when all tcgen05.mma issued so far by this thread are done.
__device__ __forceinline__ void umma_commit(uint64_t* bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(
                   smem_u32(bar))
               : "memory");
}

// 32 lanes x 32 bit, 32 consecutive columns per thread.
__device__ __forceinline__ void tmem_ld32(uint32_t taddr, uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
        "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
        "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void tmem_ld_wait() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }

// Shared-memory matrix descriptor (tcgen05 format): start address, leading
// and stride byte offsets (all >> 4), version 1, 128-byte swizzle.
__device__ __forceinline__ uint64_t smem_desc_sw128(uint32_t saddr, uint32_t lbo_bytes, uint32_t sbo_bytes) {
  uint64_t d = 0;
  d |= static_cast<uint64_t>((saddr >> 4) & 0x3FFF);
  d |= static_cast<uint64_t>((lbo_bytes >> 4) & 0x3FFF) << 16;
  d |= static_cast<uint64_t>((sbo_bytes >> 4) & 0x3FFF) << 32;
  d |= 1ull << 46;  // descriptor version (sm_100)
  d |= 2ull << 61;  // layout: 128-byte swizzle
  return d;
}

// Instruction descriptor for kind::f8f6f4, dense, fp32 accumulator.
// fmt: 0 = E4M3, 1 = E5M2; major: 0 = K-major, 1 = MN-major.
__host__ __device__ constexpr uint32_t idesc_f8(int fmt_a, int fmt_b, int major_a, int major_b, int M, int N) {
  return (1u << 4)                                   // D format: f32
         | (static_cast<uint32_t>(fmt_a) << 7)       // A format
         | (static_cast<uint32_t>(fmt_b) << 10)      // B format
         | (static_cast<uint32_t>(major_a) << 15)    // A major
         | (static_cast<uint32_t>(major_b) << 16)    // B major
         | (static_cast<uint32_t>(N >> 3) << 17)     // N / 8
         | (static_cast<uint32_t>(M >> 4) << 24);    // M / 16
}

// Instruction descriptor for kind::i8, dense: signed 8-bit operands, both
// K-major, int32 accumulator without saturation.
__host__ __device__ constexpr uint32_t idesc_i8(int M, int N) {
  return (2u << 4)                                   // D format: s32
         | (1u << 7) | (1u << 10)                    // A, B: signed 8-bit
         | (static_cast<uint32_t>(N >> 3) << 17)     // N / 8
         | (static_cast<uint32_t>(M >> 4) << 24);    // M / 16
}

// ---------------------------------------------------------------- CTA pairs
// A cluster of two CTAs runs one 2-SM MMA tile (tcgen05 cta_group::2).  Every
// CTA loads only its own operand halves into its own shared memory (no load is
// shared between CTAs), and the MMA issuer signals each CTA's barriers one by
// one.

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
// Shared::cluster address of the same shared-memory offset in CTA `rank`.
__device__ __forceinline__ uint32_t mapa_shared(uint32_t saddr, uint32_t rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(saddr), "r"(rank));
  return r;
}
// A word in the shared memory of a CTA of the cluster.
__device__ __forceinline__ void st_cluster_u32(uint32_t cluster_addr, uint32_t v) {
  asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(cluster_addr), "r"(v) : "memory");
}

// CTA and cluster barriers in their non-.aligned forms, which count threads
// one by one.  In the warp-specialized GEMM one lane of a warp runs the
// producer or MMA loop while its other lanes go ahead (timestamps on a B200
// show them reaching the teardown barrier ~0.7 us apart); the .aligned forms
// (what __syncthreads() emits) require the whole warp at the instruction
// together and leave that to the compiler's reconvergence, the non-.aligned
// forms are correct whatever the arrival order.
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
}
__device__ __forceinline__ void cta_sync() { asm volatile("barrier.sync 0;" ::: "memory"); }
// The two halves of cluster_sync, for work that can run between them (not
// .aligned: a warp may reach them diverged).
__device__ __forceinline__ void cluster_arrive() {
  asm volatile("barrier.cluster.arrive.release;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() {
  asm volatile("barrier.cluster.wait.acquire;" ::: "memory");
}

// Arrive on an mbarrier of any CTA of the cluster (release at cluster scope).
__device__ __forceinline__ void mbar_arrive_cluster(uint32_t cluster_addr) {
  asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(cluster_addr) : "memory");
}
__device__ __forceinline__ void tmem_alloc_pair(uint32_t* dst_smem, uint32_t ncols) {
  asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(dst_smem)),
               "r"(ncols)
               : "memory");
}
__device__ __forceinline__ void tmem_relinquish_pair() {
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_dealloc_pair(uint32_t taddr, uint32_t ncols) {
  asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(ncols) : "memory");
}
// 2-SM MMA: M = 256 over the pair (each CTA's shared memory holds its 128 rows
// of A and N/2 rows of B at the same offsets), accumulator rows in each CTA's
// TMEM.  Issued by the pair's even CTA only.
__device__ __forceinline__ void umma_f8f6f4_pair(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                                 uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}
// Arrive once on the mbarrier at `cluster_addr` (either CTA of the pair) when
// all 2-SM MMAs issued so far by this thread are done.
__device__ __forceinline__ void umma_commit_pair(uint32_t cluster_addr) {
  asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(cluster_addr)
               : "memory");
}
// Tiled load into this CTA's shared memory whose completion is counted on the
// pair's even CTA's mbarrier (`bar_cluster_addr`).
__device__ __forceinline__ void tma_load_3d_pair(void* dst, const CUtensorMap* m, uint32_t bar_cluster_addr, int32_t x,
                                                 int32_t y, int32_t z) {
  asm volatile(
      "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(m)), "r"(bar_cluster_addr), "r"(x), "r"(y), "r"(z)
      : "memory");
}

// ---------------------------------------------------------------- gpu-scope flags

__device__ __forceinline__ uint32_t ld_acquire_u32(const uint32_t* p) {
  uint32_t v;
  asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
  return v;
}

// Wait, with the whole warp, until the global flag *f is nonzero (another CTA
// raised it with a release store after writing the data it guards).  Lane 0
// polls; once it sees the flag every lane reads it again with acquire
// semantics, so each lane's later loads see the guarded data.  Bounded like
// mbar_wait: after FP8LIN_WAIT_LIMIT_NS a timeout is recorded in *status and
// false returned (also as soon as *abort is set).
__device__ __forceinline__ bool flag_wait_warp(const uint32_t* f, int* status, volatile int* abort,
                                               uint64_t limit_ns = FP8LIN_WAIT_LIMIT_NS) {
  int ok = 1;
  if ((threadIdx.x & 31) == 0 && !ld_acquire_u32(f)) {
    ok = 0;
    const uint64_t t0 = globaltimer_ns();
    #pragma unroll 1
    while (true) {
      #pragma unroll 1
      for (int i = 0; i < 64 && !ok; ++i) ok = ld_acquire_u32(f) != 0;
      if (ok) break;
      if (abort && *abort) break;
      if (globaltimer_ns() - t0 > limit_ns) {
        if (status) atomicExch(status, kDevTimeout);
        if (abort) *abort = 1;
        break;
      }
    }
  }
  ok = __shfl_sync(0xFFFFFFFFu, ok, 0);
  if (ok) (void)ld_acquire_u32(f);
  return ok != 0;
}

// Release a flag for the CTAs of another SM after every lane of the warp has
// written the data it guards: the warp barrier orders the lanes' stores
// before lane 0's fence (cumulative), the fence before the flag store.
__device__ __forceinline__ void warp_release_flag(uint32_t* f, uint32_t v) {
  __syncwarp();
  if ((threadIdx.x & 31) == 0) {
    asm volatile("fence.acq_rel.gpu;" ::: "memory");
    asm volatile("st.relaxed.gpu.global.u32 [%0], %1;" ::"l"(f), "r"(v) : "memory");
  }
}

// Order this thread's generic-proxy accesses of global memory (e.g. the
// acquire of a flag) before its later async-proxy (bulk copy) accesses.
__device__ __forceinline__ void fence_proxy_async_global() {
  asm volatile("fence.proxy.async.global;" ::: "memory");
}

// Bulk copy global -> this CTA's shared memory (no tensor map), completion
// counted in bytes on `bar`.  Both addresses 16-byte aligned, bytes a
// multiple of 16.  No multicast.
__device__ __forceinline__ void bulk_copy_g2s(void* dst, const void* src, uint32_t bytes, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
          smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(src)), "r"(bytes), "r"(smem_u32(bar))
      : "memory");
}

// ---------------------------------------------------------------- gpu-scope atomics

// Relaxed max on a global word, no return value.
// The delayed-scaling update rule: the next scale is fp8_max / m for the
// window maximum m, and the current scale s is kept when m is 0 or infinite
// or the quotient overflows.
__device__ __forceinline__ float next_scale(float s, float m, float fp8_max) {
  if (m > 0.0f && !isinf(m)) {
    const float q = __fdiv_rn(fp8_max, m);
    if (!isinf(q)) return q;
  }
  return s;
}

__device__ __forceinline__ void red_max_u32(uint32_t* p, uint32_t v) {
  asm volatile("red.relaxed.gpu.global.max.u32 [%0], %1;" ::"l"(p), "r"(v) : "memory");
}
// 64-bit relaxed fetch-add at gpu scope.
__device__ __forceinline__ uint64_t atom_add_relaxed_u64(void* p, uint64_t v) {
  uint64_t old;
  asm volatile("atom.relaxed.gpu.global.add.u64 %0, [%1], %2;" : "=l"(old) : "l"(p), "l"(v) : "memory");
  return old;
}
// fetch-add with acquire-release semantics at gpu scope: everything this thread
// did before is visible to whoever acquires a later value of the counter, and
// everything released by earlier incrementers is visible to this thread.
__device__ __forceinline__ uint32_t atom_add_acq_rel(uint32_t* p, uint32_t v) {
  uint32_t old;
  asm volatile("atom.acq_rel.gpu.global.add.u32 %0, [%1], %2;" : "=r"(old) : "l"(p), "r"(v) : "memory");
  return old;
}

// ---------------------------------------------------------------- fp8 casts

// Two fp32 -> packed fp8x2, round to nearest even, saturating to the largest
// finite value.  `lo` lands in the low byte (lower address).
__device__ __forceinline__ uint16_t cvt_e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ uint16_t cvt_e5m2x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e5m2x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}

// Packed fp8x2 -> two fp32 (exact: every fp8 value is an fp16 value).
__device__ __forceinline__ float2 dec_e4m3x2(uint16_t v) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(v));
  __half2 hh = *reinterpret_cast<__half2*>(&h);
  return __half22float2(hh);
}
__device__ __forceinline__ float2 dec_e5m2x2(uint16_t v) {
  uint32_t h;
  asm("cvt.rn.f16x2.e5m2x2 %0, %1;" : "=r"(h) : "h"(v));
  __half2 hh = *reinterpret_cast<__half2*>(&h);
  return __half22float2(hh);
}

}  // namespace fp8lin

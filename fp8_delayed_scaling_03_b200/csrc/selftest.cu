// selftest.cu -- the bounded waits every kernel relies on, exercised on
// purpose (fp8_wait_selftest).  One CTA: warp 0 waits on a global flag with
// the flag protocol of the stream-K fixup, warp 1 on an mbarrier of its own
// shared memory with the protocol of the GEMM pipelines, warps 2 and 3 together
// on mbarriers with the protocol of the grouped product's epilogue, each with
// the caller's time limit.  A flag that nothing sets and the mbarriers (which
// nothing ever arrives on) make the waits run out: each records
// FP8_ERR_DEVICE_TIMEOUT in the device status word and returns, and the kernel
// ends normally, so the context stays usable.  No wait here can outlast its
// limit.
//
// Warps 2 and 3 go through tiles whose barriers have completed, up to one whose
// barrier never does; warp 3 gets there late and finds the abort flag set by
// warp 2's wait, or by its own.  Both have to leave at that tile.
#include "device.cuh"
#include "internal.h"
#include "launch.h"

namespace fp8lin {
namespace {

constexpr int kDuoTiles = 5;      // the last one's barrier never completes

__global__ void __launch_bounds__(128) wait_selftest_kernel(const uint32_t* flag, int* status, int* results,
                                                            uint64_t limit_ns) {
  __shared__ __align__(8) uint64_t bar[2];
  __shared__ int gave_up, left[2], alone;
  pdl_wait();
  pdl_trigger();
  if (threadIdx.x == 0) {
    mbar_init(&bar[0], 1);
    mbar_init(&bar[1], 1);
    fence_mbar_init();
    gave_up = 0;
  }
  __syncthreads();
  const int warp = threadIdx.x >> 5;
  const bool lead = (threadIdx.x & 31) == 0;
  if (warp == 0) {
    const bool ok = flag_wait_warp(flag, status, nullptr, limit_ns);
    if (lead) results[0] = ok ? 1 : 0;
  } else if (warp == 1) {
    if (lead) alone = mbar_wait(&bar[0], 0, status, nullptr, limit_ns) ? 1 : 0;
  } else {
    int tile = 0;
    for (; tile < kDuoTiles; ++tile) {
      if (warp == 3) __nanosleep(2000);
      // (on a barrier's first phase the preceding one, of parity 1, counts as complete)
      if (!duo_await(1, &bar[1], tile + 1 < kDuoTiles ? 1u : 0u, status, &gave_up, limit_ns)) break;
      duo_sync(1);
    }
    if (lead) left[warp - 2] = tile;
  }
  __syncthreads();
  if (threadIdx.x == 32) results[1] = left[0] == left[1] && left[0] == kDuoTiles - 1 ? alone : -1;
  if (threadIdx.x == 0) settle_copies(&gave_up);   // (no copies here: the pause that a block takes which gave up)
}

}  // namespace

cudaError_t launch_wait_selftest(const uint32_t* flag, int* status, int* results, uint64_t limit_ns,
                                 cudaStream_t s) {
  return launch_pdl(wait_selftest_kernel, dim3(1), dim3(128), 0, s, flag, status, results, limit_ns);
}

}  // namespace fp8lin

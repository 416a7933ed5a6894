// wait.cuh -- bounded mbarrier waits and the tile raster of the fused
// products: the same protocol as the GEMM kernel's (../gemm_kernel.cuh), kept
// apart so that the operators build without its kernels.  A wait that outlives
// the timeout records its site in the device watchdog record and raises the
// CTA's abort flag; every role then leaves its loop.
#pragma once
#include <cstdint>

#include "../ptx.cuh"

namespace gb300 {
namespace ops {

// Where a wait gave up (the watchdog record's second word; the numbers are
// the GEMM kernel's).
enum WaitSite : uint32_t {
  kSiteEmpty = 1,      // producer waiting for a free stage
  kSiteFull = 2,       // MMA issuer waiting for a filled stage
  kSiteTmemEmpty = 3,  // MMA issuer waiting for a drained accumulator buffer
  kSiteTmemFull = 4,   // epilogue waiting for a finished accumulator
  kSiteMmaDone = 5,    // teardown: waiting for the last MMAs
  kSiteDrain = 6,      // teardown: producer waiting for its last stages
};

constexpr uint32_t kStatusTimeout = 5;  // == GEMM_ERR_TIMEOUT

struct Watch {
  volatile uint32_t* abort;
  uint32_t* err;  // device record, 4 words
  uint64_t timeout_ns;
};

// Slow path: false when the wait gave up, because the CTA is aborting (and
// honor_abort) or after timeout_ns.
template <bool kClusterScope>
__device__ __noinline__ bool wait_slow(uint32_t bar, uint32_t parity, Watch w, uint32_t site,
                                       int32_t item, bool honor_abort) {
  const uint64_t t0 = ptx::globaltimer_ns();
  while (true) {
    const bool done = kClusterScope ? ptx::mbar_try_wait_cluster(bar, parity)
                                    : ptx::mbar_try_wait(bar, parity);
    if (done) return true;
    if (honor_abort && *w.abort) return false;
    if (ptx::globaltimer_ns() - t0 > w.timeout_ns) {
      if (atomicCAS(w.err, 0u, kStatusTimeout) == 0u) {
        w.err[1] = site;
        w.err[2] = blockIdx.x;
        w.err[3] = static_cast<uint32_t>(item);
      }
      *w.abort = 1u;
      return false;
    }
  }
}

template <bool kClusterScope>
__device__ __forceinline__ bool wait_bar(uint32_t bar, uint32_t parity, const Watch& w,
                                         uint32_t site, int32_t item, bool honor_abort = true) {
  const bool done =
      kClusterScope ? ptx::mbar_try_wait_cluster(bar, parity) : ptx::mbar_try_wait(bar, parity);
  return done || wait_slow<kClusterScope>(bar, parity, w, site, item, honor_abort);
}

// The whole warp waits and agrees on the outcome, so the code after it stays
// converged.
template <bool kClusterScope>
__device__ __forceinline__ bool wait_bar_warp(uint32_t bar, uint32_t parity, const Watch& w,
                                              uint32_t site, int32_t item,
                                              bool honor_abort = true) {
  return __all_sync(0xffffffffu, wait_bar<kClusterScope>(bar, parity, w, site, item, honor_abort));
}

// Grouped raster: down a group of `group` tile-rows before moving one
// tile-column right, so tiles in flight share A and B rows in L2.
__device__ __forceinline__ void raster(int32_t t, int32_t tiles_m, int32_t tiles_n, int32_t group,
                                       int32_t& mb, int32_t& nb) {
  const int32_t per = group * tiles_n;
  const int32_t g = t / per;
  const int32_t m0 = g * group;
  const int32_t gs = min(group, tiles_m - m0);
  const int32_t r = t - g * per;
  mb = m0 + r % gs;
  nb = r / gs;
}

}  // namespace ops
}  // namespace gb300

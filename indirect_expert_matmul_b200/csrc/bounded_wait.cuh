// Bounded mbarrier waits of the tensor-core kernels: a wait that runs out sets
// the CTA's abort flag and MOE_ERR_TIMEOUT in the status word, and every role
// leaves its loop.
#pragma once

#include "common.cuh"
#include "ptx.cuh"

namespace moe {

// ~2 s.  The waits for a CTA's own copies and MMAs before it leaves keep this limit
// where a test shortens the others: what is in flight lands.
constexpr long long kWaitLimitCycles = 1ll << 32;
constexpr uint32_t kSleepNs = 20000; // upper bound of one hardware wait

__device__ __forceinline__ void expired(uint64_t* bar, volatile int* abort_flag, int* status) {
    *abort_flag = 1;
    const int site = (1 << 30) | ((int)(threadIdx.x >> 5) << 20) | (int)(ptx::smem_u32(bar) & 0xfffffu);
    atomicCAS(status + (kHdrWaitSite - kHdrStatus), 0, site);
    set_status(status, MOE_ERR_TIMEOUT);
}

// Bounded wait of one thread that runs a role by itself (CLUSTER: for arrivals by
// another CTA too); false when it has expired or the kernel is aborting.  The
// thread sleeps in hardware between polls (suspend-time hint), so waiting roles do
// not take issue slots from the dequantisation warps.
template <bool CLUSTER = false>
__device__ __forceinline__ bool wait_bar(uint64_t* bar, uint32_t parity, volatile int* abort_flag, int* status,
                                         long long limit) {
    if (!CLUSTER && ptx::mbar_try_wait(bar, parity)) return true;
    const long long t0 = clock64();
    while (true) {
        if (CLUSTER ? ptx::mbar_try_wait_cluster(bar, parity) : ptx::mbar_try_wait_sleep(bar, parity, kSleepNs))
            return true;
        if (*abort_flag) return false;
        if (clock64() - t0 > limit) {
            expired(bar, abort_flag, status);
            return false;
        }
    }
}

// The same by a whole warp, every lane polling (no lane-0 branch).  The lanes vote on
// each poll, so that they leave together with one outcome: a lane that left alone
// on its limit or the abort flag, where another has just seen the phase complete,
// would be missed for ever where the warp next meets.
template <bool CLUSTER = false>
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, volatile int* abort_flag, int* status,
                                          long long limit) {
    if (!CLUSTER && ptx::mbar_try_wait_all(bar, parity)) return true;
    const long long t0 = clock64();
    while (true) {
        const bool done = CLUSTER ? ptx::mbar_try_wait_cluster(bar, parity) : ptx::mbar_try_wait_sleep(bar, parity, kSleepNs);
        if (__all_sync(0xffffffffu, done)) return true;
        const bool late = clock64() - t0 > limit;
        if (__any_sync(0xffffffffu, late || *abort_flag)) {
            if (late) expired(bar, abort_flag, status);
            return false;
        }
    }
}

}  // namespace moe

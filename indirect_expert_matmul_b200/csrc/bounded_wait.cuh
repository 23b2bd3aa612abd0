// Bounded mbarrier waits of the tensor-core kernels: a wait that runs out sets
// the CTA's abort flag and MOE_ERR_TIMEOUT in the status word, and every role
// leaves its loop.
#pragma once

#include "common.cuh"
#include "ptx.cuh"

namespace moe {

constexpr long long kWaitLimitCycles = 1ll << 32; // ~2 s
constexpr uint32_t kSleepNs = 20000; // upper bound of one hardware wait

// Bounded wait by one lane (CLUSTER: of arrivals by another CTA too); false when the kernel is aborting.  The lane
// sleeps in hardware between polls (suspend-time hint), so waiting roles do
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
            *abort_flag = 1;
            const int site = (1 << 30) | ((int)(threadIdx.x >> 5) << 20) | (int)(ptx::smem_u32(bar) & 0xfffffu);
            atomicCAS(status + (kHdrWaitSite - kHdrStatus), 0, site);
            set_status(status, MOE_ERR_TIMEOUT);
            return false;
        }
    }
}

// lane 0 waits, the warp learns the outcome (CLUSTER: of arrivals by another CTA too)
template <bool CLUSTER = false>
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, volatile int* abort_flag, int* status,
                                          long long limit) {
    // every lane polls (no lane-0 branch); lanes that see different phases simply poll again
    if (!CLUSTER && ptx::mbar_try_wait(bar, parity)) return true;
    const long long t0 = clock64();
    while (true) {
        if (CLUSTER ? ptx::mbar_try_wait_cluster(bar, parity) : ptx::mbar_try_wait_sleep(bar, parity, kSleepNs))
            return true;
        if (*abort_flag) return false;
        if (clock64() - t0 > limit) {
            if ((threadIdx.x & 31) == 0) {
                *abort_flag = 1;
                const int site = (1 << 30) | ((int)(threadIdx.x >> 5) << 20) | (int)(ptx::smem_u32(bar) & 0xfffffu);
                atomicCAS(status + (kHdrWaitSite - kHdrStatus), 0, site);
                set_status(status, MOE_ERR_TIMEOUT);
            }
            return false;
        }
    }
}

}  // namespace moe

// fa_wait.cuh -- bounded mbarrier waits of kernels whose roles share one abort flag.
//
// A wait that runs out records kStatusTimeout in the translation unit's status word
// and raises the flag; every other wait of the CTA then gives up too, so that the CTA
// drains what is in flight, frees its tensor memory and exits.
#pragma once

#include "fa_internal.h"
#include "fa_ptx.cuh"

namespace fa {

struct WaitCtl {
    volatile int* abort;            // of the CTA, in shared memory
    int* status;                    // of the translation unit
    unsigned long long timeout_ns;
};

// The slow path: kSleep suspends the thread between checks (off the critical path, where
// polling would take issue slots from busy warps of its sub-partition).
template <bool kSleep>
__device__ __noinline__ bool wait_bounded(uint32_t bar, uint32_t parity, WaitCtl c) {
    const uint64_t t0 = globaltimer_ns();
    while (true) {
        if (kSleep ? mbar_try_wait_sleep(bar, parity, 20000u) : mbar_try_wait(bar, parity)) return true;
        if (*c.abort) return false;
        if (globaltimer_ns() - t0 > c.timeout_ns) {
            *c.abort = 1;
            atomicCAS(c.status, 0, kStatusTimeout);
            return false;
        }
    }
}
// One thread: true when the phase completed, false when the CTA gave up.
template <bool kSleep = true>
__device__ __forceinline__ bool wait_one(uint32_t bar, uint32_t parity, const WaitCtl& c) {
    return mbar_try_wait(bar, parity) || wait_bounded<kSleep>(bar, parity, c);
}
// Every lane of a converged warp, with one result (an issue loop stays warp-uniform).
template <bool kSleep = false>
__device__ __forceinline__ bool wait_warp(uint32_t bar, uint32_t parity, const WaitCtl& c) {
    return __all_sync(0xffffffffu, mbar_try_wait(bar, parity) || wait_bounded<kSleep>(bar, parity, c));
}
// What must land before the CTA may exit, whatever has happened: a tenth of a second at most.
__device__ __forceinline__ void drain(uint32_t bar, uint32_t parity, const WaitCtl& c) {
    volatile int never = 0;
    wait_one(bar, parity, WaitCtl{&never, c.status, 100000000ull});
}

}  // namespace fa

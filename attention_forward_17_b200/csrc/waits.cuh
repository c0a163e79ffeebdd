// Bounded waits on mbarriers, shared by the attention kernels and the self-test that lets
// one run out of time.
#pragma once

#include "ptx.cuh"

namespace fa {

constexpr int kStatusTimeout = -7;  // FA_ERR_TIMEOUT
constexpr uint64_t kWaitLimitNs = 2000000000ull;      // 2 s
constexpr uint64_t kWaitLimitAbortNs = 1000000ull;    // 1 ms once the CTA has aborted

// Polls the mbarrier phase until it completes or `limit_ns` (globaltimer)
// passes; on time-out marks the CTA aborted and records FA_ERR_TIMEOUT.  Once
// aborted, further waits give up after `limit_abort_ns`.
__device__ __forceinline__ void wait_slow(uint32_t bar, uint32_t parity, volatile uint32_t* abort,
                                          int* status, uint64_t limit_ns, uint64_t limit_abort_ns) {
    const uint64_t t0 = global_timer_ns();
    for (uint32_t it = 1;; ++it) {
        if (mbar_try_wait(bar, parity)) return;
        if ((it & 31u) == 0) {
            const uint64_t limit = *abort ? limit_abort_ns : limit_ns;
            if (global_timer_ns() - t0 > limit) {
                if (!*abort) {
                    *abort = 1u;
                    if (status) atomicExch(status, kStatusTimeout);
                }
                return;
            }
        }
    }
}

}  // namespace fa

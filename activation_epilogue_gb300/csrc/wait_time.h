// How long a kernel's wait has lasted, as the kernel's own time: between two looks at the clock at most
// a millisecond counts, ten times what a look's suspension takes, so that a context that another one
// displaces from the GPU for seconds does not come back to a wait that has run out.  Plain arithmetic,
// for the kernels and for a test on the host.
#pragma once

#include <cstdint>

#ifdef __CUDACC__
#define WAIT_HOST_DEVICE __host__ __device__
#else
#define WAIT_HOST_DEVICE
#endif

namespace gemm_epi {

constexpr uint64_t kWaitLookNs = 1000 * 1000;

struct WaitTime {
    uint64_t last, total;
    // now: the clock in nanoseconds at the wait's start
    explicit WAIT_HOST_DEVICE WaitTime(uint64_t now) : last(now), total(0) {}
    // the time waited by `now`
    WAIT_HOST_DEVICE uint64_t at(uint64_t now)
    {
        const uint64_t step = now - last;
        total += step < kWaitLookNs ? step : kWaitLookNs;
        last = now;
        return total;
    }
};

}  // namespace gemm_epi

// The waits of a kernel's roles for one another: how long, and when they give up.  Apart
// from the barriers, so that it also runs on the host.
#pragma once

#include <cstdint>

#ifdef __CUDACC__
#define VF_WAIT_FN __host__ __device__ __forceinline__
#else
#define VF_WAIT_FN inline
#endif

namespace vfp {

constexpr uint64_t kWaitNs = 2000000000ull;
// The most that one turn of a wait counts for.  A turn takes some 4 us; where the clock has
// run on for longer the kernel was not running (another context was, or a debugger held
// it), and neither were the copies and products that it waits for.
constexpr uint64_t kTurnNs = 100000;

// Waits until done(), for kWaitNs of the kernel's own time at most; false when it gave up
// (done() is asked once more then), or failed() says that another role did.
template <class Done, class Failed, class Clock>
VF_WAIT_FN bool wait_until(const Done &done, const Failed &failed, const Clock &now) {
    uint64_t last = now(), waited = 0;
    while (!done()) {
        if (failed()) return false;
        const uint64_t t = now();
        waited += t - last < kTurnNs ? t - last : kTurnNs;
        last = t;
        if (waited > kWaitNs) return done();
    }
    return true;
}

}  // namespace vfp

// mk_wait.cuh -- bounded waits of the kernels outside mk_kernels.cu: each
// gives up after a limit, records the site in the device error word and
// raises the call's abort word, so that every other wait of the call ends too.
#pragma once

#include "mk_common.h"
#include "mk_host.h"
#include "mk_ptx.cuh"

namespace mk {

struct Waiter {
    DevError* err;     // the device error word
    uint32_t* abort;   // this call's abort word
    long long limit_ns;
};

__device__ __forceinline__ void report(DevError* e, uint32_t code, uint32_t site, uint32_t info) {
    if (atomicCAS(&e->code, 0u, code) == 0u) {
        e->site = site;
        e->cta = blockIdx.x;
        e->info = info;
        __threadfence();
    }
}

__device__ __noinline__ bool wait_gave_up(const Waiter& w, uint64_t t0, uint32_t site, uint32_t info) {
    if (ld_relaxed_u32(w.abort) != 0u) return true;
    if ((long long)(globaltimer() - t0) <= w.limit_ns) return false;
    report(w.err, ERR_TIMEOUT, site, info);
    st_relaxed_u32(w.abort, 1u);
    return true;
}

// An mbarrier phase.  False: timed out, or the call was aborted elsewhere.
__device__ __forceinline__ bool await_mbar(uint64_t* bar, uint32_t parity, const Waiter& w, uint32_t site) {
    if (mbar_try_wait(bar, parity)) return true;
    const uint64_t t0 = globaltimer();
    for (uint32_t n = 1; !mbar_try_wait(bar, parity); ++n)
        if ((n & 63u) == 0u && wait_gave_up(w, t0, site, parity)) return false;
    return true;
}

// *p >= target (acquire).
__device__ __forceinline__ bool await_geq(const uint32_t* p, uint32_t target, const Waiter& w, uint32_t site) {
    if (ld_acquire_u32(p) >= target) return true;
    const uint64_t t0 = globaltimer();
    for (uint32_t n = 1; ld_acquire_u32(p) < target; ++n) {
        __nanosleep(32);
        if ((n & 15u) == 0u && wait_gave_up(w, t0, site, target)) return false;
    }
    return true;
}

// Taken by every lane of a warp; all lanes get the same answer.
__device__ __forceinline__ bool warp_await_mbar(uint64_t* bar, uint32_t parity, const Waiter& w, uint32_t site) {
    return __all_sync(0xffffffffu, await_mbar(bar, parity, w, site));
}

}  // namespace mk

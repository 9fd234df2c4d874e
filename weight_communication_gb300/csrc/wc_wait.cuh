// wc_wait.cuh -- waits on shared-memory barriers that end in any case.
//
// A wait that is not answered within about two seconds is given up, so that a
// kernel whose copies or products never come ends and leaves the GPU usable.
// The limit is time in which the waiting warp ran: the process may be suspended
// on the GPU for any time, and a clock alone would then count a wait as lost
// that is answered as soon as the process runs again.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "wc_device.cuh"

namespace wc {

// Nanoseconds of the GPU's clock, modulo 2^32 (4.3 s).
struct WaitLimit {
    static constexpr uint32_t kLimit = 2000000000u;
    // Two looks at the clock are 64 tries apart, far less than this; whatever is
    // longer the process did not run, and counts as this much.
    static constexpr uint32_t kGap = 10000000u;

    uint32_t last, waited;
    __host__ __device__ explicit WaitLimit(uint32_t now) : last(now), waited(0u) {}
    __host__ __device__ bool spent(uint32_t now) {
        const uint32_t gap = now - last;
        last = now;
        waited += gap < kGap ? gap : kGap;
        return waited >= kLimit;
    }
};

__device__ __forceinline__ uint32_t timer_ns() {
    uint32_t t;
    asm volatile("mov.u32 %0, %globaltimer_lo;" : "=r"(t));
    return t;
}

__device__ __forceinline__ uint32_t smem_of(const void *p) {
    return uint32_t(__cvta_generic_to_shared(p));
}

// One lane of a converged warp.
__device__ __forceinline__ bool elected() {
    uint32_t r;
    asm volatile(
        "{\n.reg .pred p;\n"
        "elect.sync _|p, 0xFFFFFFFF;\n"
        "selp.u32 %0, 1, 0, p;\n}\n"
        : "=r"(r));
    return r != 0;
}

__device__ __forceinline__ void mbar_init(uint32_t bar, uint32_t count) {
    asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(count) : "memory");
}

__device__ __forceinline__ void mbar_arrive(uint32_t bar) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}

__device__ __forceinline__ bool mbar_try(uint32_t bar, uint32_t parity) {
    uint32_t done;
    asm volatile(
        "{\n.reg .pred p;\n"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n"
        "selp.u32 %0, 1, 0, p;\n}\n"
        : "=r"(done)
        : "r"(bar), "r"(parity)
        : "memory");
    return done != 0;
}

// A converged warp waits for the phase of that parity to end; false if it gave
// up, which is counted in *given_up.  (The vote makes the answer, and the branch
// on it, uniform.)
__device__ __forceinline__ bool mbar_wait(uint32_t bar, uint32_t parity, unsigned int *given_up) {
    if (__all_sync(kFull, mbar_try(bar, parity))) return true;
    WaitLimit limit(timer_ns());
    for (uint32_t i = 0; i < (1u << 28); ++i) {
        if (__all_sync(kFull, mbar_try(bar, parity))) return true;
        if ((i & 63u) == 63u && __any_sync(kFull, limit.spent(timer_ns()))) break;
    }
    if (elected()) atomicAdd(given_up, 1u);
    __syncwarp();
    return false;
}

}  // namespace wc

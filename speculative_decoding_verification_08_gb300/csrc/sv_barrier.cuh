// sv_barrier.cuh -- shared-memory barriers with bounded waits, bulk copies into
// shared memory, and the waits of dependent launches: what every kernel family
// of the library uses.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace sv {

// ---------------------------------------------------------------------------
// mbarrier, bulk-copy and timing primitives (inline PTX)

constexpr uint32_t kStatusTimeout = 16u;
constexpr uint64_t kWaitLimitNs = 250000000ull;  // any single wait gives up after 250 ms

__device__ __forceinline__ uint32_t smem_u32(const void *p) {
    return (uint32_t)__cvta_generic_to_shared(p);
}

__device__ __forceinline__ void mbar_init(unsigned long long *bar, uint32_t count) {
    asm volatile("mbarrier.init.shared.b64 [%0], %1;" ::"r"(smem_u32(bar)), "r"(count) : "memory");
}

__device__ __forceinline__ void mbar_arrive_expect_tx(unsigned long long *bar, uint32_t bytes) {
    asm volatile("mbarrier.arrive.expect_tx.shared.b64 _, [%0], %1;" ::"r"(smem_u32(bar)),
                 "r"(bytes)
                 : "memory");
}

__device__ __forceinline__ void mbar_arrive(unsigned long long *bar) {
    asm volatile("mbarrier.arrive.shared.b64 _, [%0];" ::"r"(smem_u32(bar)) : "memory");
}

__device__ __forceinline__ uint64_t global_ns() {
    uint64_t t;
    asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t));
    return t;
}

// One try: the thread may sleep in it for up to kTrySuspendNs and is woken
// as soon as the phase completes, so a waiting warp issues a few instructions
// per wait instead of spinning.
constexpr uint32_t kTrySuspendNs = 1000000u;

__device__ __forceinline__ bool mbar_try(unsigned long long *bar, uint32_t parity) {
    uint32_t done;
    asm volatile(
        "{ .reg .pred p; mbarrier.try_wait.parity.shared.b64 p, [%1], %2, %3; selp.u32 %0, 1, 0, p; }"
        : "=r"(done)
        : "r"(smem_u32(bar)), "r"(parity), "r"(kTrySuspendNs)
        : "memory");
    return done != 0;
}

// Wait for the phase with the given parity to complete, for at most
// kWaitLimitNs of wall-clock time.  The clock is read only once a first try
// has failed: a phase that is already complete costs one try_wait.
__device__ __forceinline__ bool mbar_wait(unsigned long long *bar, uint32_t parity) {
    if (mbar_try(bar, parity)) return true;
    const uint64_t t0 = global_ns();
    while (true) {
        if (mbar_try(bar, parity)) return true;
        if (global_ns() - t0 > kWaitLimitNs) return false;
    }
}

__device__ __forceinline__ void bulk_copy_g2s(void *dst, const void *src, uint32_t bytes,
                                              unsigned long long *bar) {
    asm volatile(
        "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
            smem_u32(dst)),
        "l"(src), "r"(bytes), "r"(smem_u32(bar))
        : "memory");
}

__device__ __forceinline__ void grid_dependents_may_launch() {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

__device__ __forceinline__ void wait_for_primary_grid() {
    asm volatile("griddepcontrol.wait;" ::: "memory");
}

}  // namespace sv

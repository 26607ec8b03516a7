// fsdp_wait.cuh -- mbarriers in shared memory and bounded waits on them, for
// the operators' kernels. Every wait is given up after kWaitNs; the block
// counts itself and ends (fsdp_ops_wait_timeouts). One counter per source
// file that includes this.
#pragma once

#include <cuda_runtime.h>

#include <cstdint>

namespace fsdp {
namespace wait {
namespace {

constexpr uint64_t kWaitNs = 2000000000ull;

__device__ unsigned long long g_wait_timeouts;

__device__ __forceinline__ uint32_t saddr(const void *p)
{
    return (uint32_t)__cvta_generic_to_shared(p);
}
__device__ __forceinline__ void bar_init(uint64_t *bar, uint32_t count)
{
    asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(saddr(bar)), "r"(count) : "memory");
}
__device__ __forceinline__ bool bar_try(uint64_t *bar, uint32_t parity)
{
    uint32_t done;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(done)
        : "r"(saddr(bar)), "r"(parity)
        : "memory");
    return done != 0;
}
__device__ __forceinline__ uint64_t now_ns()
{
    uint64_t t;
    asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t));
    return t;
}
// Waits for the phase of `parity` at most kWaitNs (and 2^27 polls, should the
// timer stand still); false if it gave up.
__device__ __forceinline__ bool bar_wait(uint64_t *bar, uint32_t parity)
{
    if (bar_try(bar, parity))
        return true;
    const uint64_t t0 = now_ns();
    for (uint32_t round = 0; round < (1u << 22); round++) {
        for (int k = 0; k < 32; k++)
            if (bar_try(bar, parity))
                return true;
        if (now_ns() - t0 > kWaitNs)
            return false;
    }
    return false;
}
// The same by a whole warp: one answer for all lanes.
__device__ __forceinline__ bool warp_wait(uint64_t *bar, uint32_t parity)
{
    return __all_sync(0xffffffffu, bar_wait(bar, parity));
}
__device__ __forceinline__ void bar_expect(uint64_t *bar, uint32_t bytes)
{
    asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(saddr(bar)), "r"(bytes)
                 : "memory");
}
// After a wait was given up: bulk copies into the block's shared memory may
// still be under way; 10 ms for them before the block ends.
__device__ __forceinline__ void let_copies_land()
{
    const uint64_t t0 = now_ns();
    for (int i = 0; i < (1 << 20) && now_ns() - t0 < 10000000ull; i++)
        __nanosleep(1000);
}

inline cudaError_t wait_timeouts(unsigned long long *n)
{
    return cudaMemcpyFromSymbol(n, g_wait_timeouts, sizeof *n);
}

}  // namespace
}  // namespace wait
}  // namespace fsdp

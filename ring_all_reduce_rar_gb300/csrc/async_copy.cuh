// async_copy.cuh -- mbarriers, bulk copies into shared memory and bounded
// waits for them, as the model operators' kernels use them.
//
// Every wait has a limit.  A wait that runs out raises a flag of the CTA, which
// the CTA's other waits poll, and records it for rar_status.
#pragma once

#include "op_elem.cuh"

namespace rar {

__device__ __forceinline__ uint32_t smem_u32(const void *p) { return (uint32_t)__cvta_generic_to_shared(p); }
__device__ __forceinline__ void mbar_init(uint64_t *bar, uint32_t count) {
    asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(smem_u32(bar)), "r"(count) : "memory");
}
__device__ __forceinline__ void mbar_fence_init() { asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory"); }
__device__ __forceinline__ void mbar_expect_tx(uint64_t *bar, uint32_t bytes) {
    asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(smem_u32(bar)), "r"(bytes) : "memory");
}
__device__ __forceinline__ void mbar_arrive(uint64_t *bar) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_u32(bar)) : "memory");
}
__device__ __forceinline__ bool mbar_try_wait(uint64_t *bar, uint32_t parity) {
    uint32_t done;
    asm volatile(
        "{\n\t.reg .pred P;\n\t"
        "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 P, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, P;\n\t}"
        : "=r"(done)
        : "r"(smem_u32(bar)), "r"(parity)
        : "memory");
    return done != 0;
}
// `bytes` (a multiple of 16) to shared memory; arrives on `bar`.
__device__ __forceinline__ void bulk_load(void *dst, const void *src, uint32_t bytes, uint64_t *bar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(smem_u32(dst)), "l"(src),
                 "r"(bytes), "r"(smem_u32(bar))
                 : "memory");
}
__device__ __forceinline__ unsigned long long now_ns() {
    unsigned long long t;
    asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t));
    return t;
}

struct WaitLimits {
    RingStatus *status;
    unsigned long long timeout_ns;
    int mute;  // RAR_FAULT_MUTE: the rank (matrix, piece) whose copies never complete, or -1
};
// RingStatus::rank of a wait that ran out here; `step` then says what was
// waited for, `slice` which CTA waited.
enum { WAIT_OF_XENT = -2, WAIT_OF_NORM = -3 };

// Waits for the phase of `bar` with this parity; false once the limit has
// passed or another wait of the CTA has given up.
__device__ __forceinline__ bool mbar_wait(int *failed, const WaitLimits &lim, uint64_t *bar, uint32_t parity, int of, int what) {
    if (mbar_try_wait(bar, parity)) return true;
    if (*(volatile int *)failed) return false;
    const unsigned long long t0 = now_ns();
    const unsigned long long most = lim.timeout_ns / 16ull + (1ull << 20);
    for (unsigned long long it = 0; it < most; it++) {
        if (mbar_try_wait(bar, parity)) return true;
        if ((it & 63) == 63) {
            if (*(volatile int *)failed) return false;
            if (now_ns() - t0 > lim.timeout_ns) break;
        }
    }
    *(volatile int *)failed = 1;
    lim.status->code = RAR_ETIMEOUT;
    lim.status->rank = of;
    lim.status->step = what;
    lim.status->slice = (int)blockIdx.x;
    __threadfence();
    atomicAdd(&lim.status->seq, 1u);
    return false;
}

// Waits for loads that were issued: they land by themselves, so the limit
// (1 s) is only reached on a broken device, or where some of a stage's were never
// issued (by the other CTA of a failed pair, or a muted rank).  False then: whatever the
// CTA did issue has landed meanwhile.
__device__ __forceinline__ bool mbar_drain(uint64_t *bar, uint32_t parity) {
    const unsigned long long t0 = now_ns();
    for (unsigned long long it = 0; it < (1ull << 32); it++) {
        if (mbar_try_wait(bar, parity)) return true;
        if ((it & 63) == 63 && now_ns() - t0 > 1000000000ull) break;
    }
    return false;
}

}  // namespace rar

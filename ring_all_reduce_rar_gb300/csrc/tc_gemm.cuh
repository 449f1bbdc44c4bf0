// tc_gemm.cuh -- building blocks of a matrix product on the tensor cores by
// pairs of CTAs (a cluster of two): TMA loads into
// 128-byte-swizzled shared memory, tcgen05.mma of 256 x 256 x 16 steps issued by
// one thread of the pair, accumulators in tensor memory.
//
// Operands come in boxes of 64 16-bit elements (128 bytes) of 64 or 128 rows,
// whatever the operand's role:
//   rows = M or N, columns = K   "K-major": the rows of 8 x 128 bytes that the
//       swizzle works on follow each other every 1024 bytes; a step of 16 along
//       K is 32 bytes further in the row;
//   rows = K, columns = M or N   "MN-major": groups of 8 K rows are 1024 bytes
//       apart, the next 64 columns are the next box; a step of 16 along K is 2048
//       bytes further.
// So no operand is transposed in memory.
#pragma once

#include <cuda.h>

#include "async_copy.cuh"

namespace rar {

constexpr int kTcStages = 7;
constexpr int kTcStageBytes = 32768;       // a CTA's share of A (128 x 64) and of B (128 x 64)
constexpr int kTcEpilogueWarps = 8;        // two per quarter of the accumulator's lanes
constexpr int kTcThreads = 32 * (kTcEpilogueWarps + 2);

constexpr int kTcSmem = kTcStages * kTcStageBytes + 1024;  // + alignment to the swizzle's 1024 bytes

struct TcShared {
    uint64_t full[kTcStages];   // leader: both CTAs' loads of a stage have landed
    uint64_t empty[kTcStages];  // each CTA: the products that read a stage are done
    uint64_t acc_full[2];       // each CTA: an accumulator is complete
    uint64_t acc_empty[2];      // leader: both CTAs' epilogues have read it
    uint32_t tmem;
    int failed;
};

__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
// The same shared-memory place in CTA `rank` of the cluster.
__device__ __forceinline__ uint32_t peer_addr(uint32_t addr, uint32_t rank) {
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
    return r;
}
__device__ __forceinline__ void cluster_sync_all() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ void tc_arrive_cluster(uint32_t cluster_addr) {
    asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(cluster_addr) : "memory");
}
// Waits for a barrier of the pair (see mbar_wait); role: what was waited for.
__device__ __forceinline__ bool tc_wait(TcShared *sh, const WaitLimits &lim, uint64_t *bar, uint32_t parity, int role) {
    return mbar_wait(&sh->failed, lim, bar, parity, WAIT_OF_XENT, role);
}

__device__ __forceinline__ void tc_prefetch_map(const CUtensorMap *map) {
    asm volatile("prefetch.tensormap [%0];" ::"l"(map) : "memory");
}
__device__ __forceinline__ void tc_load_box(const CUtensorMap *map, uint32_t dst, uint32_t cluster_bar, int x, int y) {
    asm volatile(
        "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
        "l"(map), "r"(x), "r"(y), "r"(cluster_bar)
        : "memory");
}

// Shared-memory operand descriptor: 128-byte swizzle, version 1; strides in
// bytes (see the top of this file).
__device__ __forceinline__ uint64_t tc_operand(uint32_t addr, uint32_t leading, uint32_t stride) {
    return (uint64_t)((addr & 0x3FFFFu) >> 4) | ((uint64_t)(leading >> 4) << 16) | ((uint64_t)(stride >> 4) << 32) |
           (1ull << 46) | (2ull << 61);
}
// Instruction descriptor of kind::f16 with 32-bit accumulators, M = 256 over
// the pair.
__device__ __forceinline__ uint32_t tc_instruction(bool bf16, bool a_mn, bool b_mn, uint32_t n) {
    const uint32_t type = bf16 ? 1u : 0u;
    return (1u << 4) | (type << 7) | (type << 10) | ((a_mn ? 1u : 0u) << 15) | ((b_mn ? 1u : 0u) << 16) | ((n >> 3) << 17) |
           ((256u >> 4) << 24);
}
__device__ __forceinline__ void tc_mma(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool accumulate) {
    asm volatile(
        "{\n\t.reg .pred P;\n\tsetp.ne.u32 P, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, P;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(accumulate ? 1u : 0u)
        : "memory");
}
// Arrives on `bar` in both CTAs once the products issued so far are done.
__device__ __forceinline__ void tc_commit(uint64_t *bar) {
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(smem_u32(bar)),
        "h"((uint16_t)3)
        : "memory");
}
__device__ __forceinline__ void tc_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }

// 32 columns of this warp's 32 accumulator lanes, one lane a thread.
__device__ __forceinline__ void tc_read32(uint32_t addr, float *v) {
    uint32_t *r = reinterpret_cast<uint32_t *>(v);
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
        "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
          "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
          "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(addr));
}
__device__ __forceinline__ void tc_read8(uint32_t addr, float *v) {
    uint32_t *r = reinterpret_cast<uint32_t *>(v);
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
                 : "r"(addr));
}
__device__ __forceinline__ void tc_write8(uint32_t addr, const float *v) {
    const uint32_t *r = reinterpret_cast<const uint32_t *>(v);
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(addr), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
                 : "memory");
}
__device__ __forceinline__ void tc_write_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tc_read_wait() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }

// 32-byte accesses: a whole sector a thread.
__device__ __forceinline__ void store_32b(void *p, const uint32_t *r) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]),
                 "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
                 : "memory");
}
__device__ __forceinline__ void load_32b(const void *p, uint32_t *r) {
    asm volatile("ld.global.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
                 : "l"(p)
                 : "memory");
}

// Barriers and tensor memory of the pair; every thread of both CTAs calls
// these two, first and last.
__device__ __forceinline__ void tc_begin(TcShared *sh) {
    if (threadIdx.x == 0) {
        sh->failed = 0;
        for (int s = 0; s < kTcStages; s++) {
            mbar_init(&sh->full[s], 1);
            mbar_init(&sh->empty[s], 1);
        }
        for (int s = 0; s < 2; s++) {
            mbar_init(&sh->acc_full[s], 1);
            mbar_init(&sh->acc_empty[s], 2 * kTcEpilogueWarps);
        }
        mbar_fence_init();
    }
    if (threadIdx.x / 32 == kTcEpilogueWarps) {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_u32(&sh->tmem)) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    }
    tc_fence_before();
    __syncthreads();
    cluster_sync_all();
    tc_fence_after();
}
__device__ __forceinline__ void tc_end(TcShared *sh) {
    tc_fence_before();
    __syncthreads();
    cluster_sync_all();
    tc_fence_after();
    if (threadIdx.x / 32 == kTcEpilogueWarps)
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, 512;" ::"r"(sh->tmem) : "memory");
}

}  // namespace rar

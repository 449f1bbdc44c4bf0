// rmsnorm.cuh -- what the residual norm (rmsnorm.cu) and its gradient
// (rmsnorm_grad.cu) share: rows over threads, and the shapes of their launches.
#pragma once

#include <algorithm>

#include "async_copy.cuh"
#include "op_host.h"

namespace rar {

template <int DT>
__device__ __forceinline__ const char *row_of(const void *base, long long t, long long stride) {
    return static_cast<const char *>(base) + t * stride * ElemInfo<DT>::bytes;
}
template <int DT>
__device__ __forceinline__ char *row_of(void *base, long long t, long long stride) {
    return static_cast<char *>(base) + t * stride * ElemInfo<DT>::bytes;
}

// Sum over the `warps` warps of a row (red: a float a warp of the CTA).
// Everyone gets the same bits.  All threads of the CTA come here.
__device__ __forceinline__ float row_sum(float v, float *red, int warps) {
    v = warp_sum(v);
    if (warps == 1) return v;
    const int warp = threadIdx.x / 32;
    if (threadIdx.x % 32 == 0) red[warp] = v;
    __syncthreads();
    const int w0 = warp / warps * warps;
    // up to 16 warps: a lane each, added by the same tree in every warp
    float t = threadIdx.x % 32 < warps ? red[w0 + threadIdx.x % 32] : 0.0f;
    return warp_sum(t);
}

constexpr int kNormMaxThreads = 512;
constexpr int kNormMaxStages = 8;

// Barrier `bar`: the n threads of a row, without the loading warp.
__device__ __forceinline__ void row_threads_sync(int bar, int n) { asm volatile("bar.sync %0, %1;" ::"r"(bar), "r"(n) : "memory"); }

// A warp has read a stage of a ring; one lane comes here, after its warp's __syncwarp.
// After a wait of the CTA that ran out no stage is free any more: the row that a warp
// gave up may still be on its way, and its barrier must not be armed a second time.
__device__ __forceinline__ void free_stage(int *failed, uint64_t *empty) {
    if (!*(volatile int *)failed) mbar_arrive(empty);
}

// Warps a row and vectors a thread, both powers of two, for `vecs` vectors: up to
// `most` threads of one vector, then up to 4 vectors; v is 0 where that does not hold the row.
struct RowShape {
    int v, warps;
};
inline RowShape row_shape(size_t vecs, int most = kNormMaxThreads) {
    RowShape r{1, 1};
    while ((size_t)r.warps * 32 < vecs && r.warps * 32 < most) r.warps *= 2;
    while ((size_t)r.warps * 32 * r.v < vecs) r.v *= 2;
    return r.v <= 4 ? r : RowShape{0, r.warps};
}
// Calls f(IntC<V>{}) for v = 1, 2, 4.
template <typename F>
cudaError_t dispatch_v(int v, F &&f) {
    switch (v) {
    case 1: return f(IntC<1>{});
    case 2: return f(IntC<2>{});
    case 4: return f(IntC<4>{});
    }
    return cudaErrorInvalidValue;
}
// Shared memory that a launch may ask for: the 227 KB of a CTA without 1 KB, which is
// more than any of these kernels declares itself.
constexpr size_t kNormMaxSmem = 226 * 1024;

// A launch of a kernel whose shared memory may pass 48 KB.  The limit belongs to the
// kernel in the whole process: it is the same in every call, so that a call in another
// thread cannot lower it between this one's two steps.
template <typename Args>
cudaError_t launch_any(void (*kern)(Args), dim3 grid, int threads, size_t smem, cudaStream_t stream, const Args &k) {
    if (smem > 32 * 1024) {
        const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kNormMaxSmem);
        if (e != cudaSuccess) return e;
    }
    return launch_pdl(kern, grid, dim3((unsigned)threads), smem, stream, k);
}
// CTAs an SM and stages of a ring kernel of `threads` threads (of which registers
// allow sm_threads an SM) for rows of stage_bytes in all: at most 4 CTAs in 220 KB, at
// least 3 rows ahead if CTAs share an SM, 2 if one has it to itself.  ctas 0: the rows
// do not fit, or there are too few for the ring to turn.  Rows of under 4 warps
// stay with the other kernels, too.
// A stage is used by one group of row threads alone (stages is a multiple of
// `groups`).  With a stage shared by two groups, one could wait for the stage's second row
// while its first has not landed; the parity that it waits for is then that of the phase
// before the first, which counts as complete.
struct RingShape {
    int ctas, stages;
};
inline RingShape ring_shape(const rar_ctx *h, size_t rows, const RowShape &shape, int threads, int sm_threads, int groups, size_t stage_bytes) {
    constexpr size_t kSmem = 220 * 1024;  // of an SM, less what the kernels declare
    if (!shape.v || shape.warps < 4) return {0, 0};
    int ctas = std::max(1, std::min(4, sm_threads / threads));
    while (ctas > 1 && kSmem / ctas / stage_bytes < 3) ctas--;
    const int stages = (int)std::min<size_t>(kSmem / ctas / stage_bytes, kNormMaxStages) / groups * groups;
    if (stages < 2 || rows < (size_t)h->sm_count * ctas * 4) return {0, 0};
    return {ctas, stages};
}
// Threads of a CTA that takes a row of `dim` single elements: about 4 each.
inline int any_threads(size_t dim) { return (int)std::min<size_t>(std::max<size_t>((dim / 4 + 31) / 32 * 32, 32), kNormMaxThreads); }
}  // namespace rar

// rmsnorm.cu -- the residual stream's join with the ranks' partial results,
// its RMS norm with an optional 8-bit output, and the gradient
// (rar_add_rmsnorm, rar_add_rmsnorm_grad).
//
//   s = residual + x_c + x_(c+1) + ...   (c: the element's chunk, ring order)
//   rstd = 1 / sqrt(mean(s^2) + eps),  y = s rstd weight
//   dx = dsum + rstd (weight dout - s rstd^2 mean(weight dout s))
//   dweight = sum over the rows of dout s rstd
//
// Bound by memory: (p + 1) reads and 2 writes an element against p + 6
// operations.
#include <algorithm>

#include "async_copy.cuh"
#include "op_host.h"

namespace rar {

struct NormArgs {
    RankPtrs parts;
    int p;
    long long rows, dim;
    long long part_stride, residual_stride, sum_stride, out_stride, out8_stride;
    const void *residual, *weight;
    float eps;
    void *sum, *out;
    float *rstd;
    uint8_t *out8;
    float *scales;
    long long group, n_groups;
    int group_shift;  // log2 of a group's 16-byte vectors, where they are 1, 2, ... 32
    float inv_dim;
    int warps;       // warps a row
    int stages;      // the ring kernel: rows in flight
    WaitLimits limits;
};

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
constexpr int kRingRowThreads = 256;  // of a row in the ring kernel
constexpr int kNormRanks = 8;  // ranks whose loads are in flight together

// Element (t, j) of the sum over the ranks, in the order that starts at rank r.
template <int DT>
__device__ __forceinline__ float fold_element(const NormArgs &a, int r, long long j) {
    float f = 0.0f;
    for (int k0 = 0; k0 < a.p; k0 += kNormRanks) {
        float w[kNormRanks];
#pragma unroll
        for (int k = 0; k < kNormRanks; k++)
            if (k0 + k < a.p) {
                w[k] = load_f<DT>(rank_ptr(a.parts, a.p, r), j);
                r = r + 1 == a.p ? 0 : r + 1;
            }
#pragma unroll
        for (int k = 0; k < kNormRanks; k++)
            if (k0 + k < a.p) f = k0 + k ? f + w[k] : w[k];
    }
    return f;
}

// Barrier `bar`: the n threads of a row, without the loading warp.
__device__ __forceinline__ void row_threads_sync(int bar, int n) { asm volatile("bar.sync %0, %1;" ::"r"(bar), "r"(n) : "memory"); }

// What a row's threads do once they hold its s: the norm and every output.
// QUANT: 0 none; 1 a group is 2^group_shift aligned lanes of a warp, its maximum a
// shuffle; 2 any group, maxima in shared memory (a maximum does not depend on
// the order, so neither do the codes).  n threads a row; gmax: the row's maxima,
// clear (QUANT 2).  All threads that sync() joins come here.
template <int DT, int V, int QUANT, typename SYNC>
__device__ __forceinline__ void norm_outputs(const NormArgs &a, long long t, bool live, int tid, int n, float rstd, float (&s)[V][16 / ElemInfo<DT>::bytes],
                                             const RowBits<DT> (&w)[V], unsigned *gmax, SYNC &&sync) {
    constexpr int VE = RowBits<DT>::VE;
    const int vecs = live ? (int)(a.dim / VE) : 0;
    if (live && a.rstd && tid == 0) a.rstd[t] = rstd;
#pragma unroll
    for (int v = 0; v < V; v++) {
        const int vec = tid + v * n;
        const bool has = vec < vecs;
        if (a.sum && has) store_vec<DT>(row_of<DT>(a.sum, t, a.sum_stride), vec, s[v]);
        float amax = 0.0f;
#pragma unroll
        for (int e = 0; e < VE; e++) {
            s[v][e] *= rstd;
            if (a.weight) s[v][e] *= w[v].get(e);
            if (QUANT && has) amax = fmaxf(amax, fabsf(s[v][e]));
        }
        if (a.out && has) store_vec<DT>(row_of<DT>(a.out, t, a.out_stride), vec, s[v]);
        if (QUANT == 1) {
            for (int o = 1 << a.group_shift >> 1; o; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, o));
            const float scale = scale_of(amax);
            if (has) {
                if ((vec & ((1 << a.group_shift) - 1)) == 0) a.scales[t * a.n_groups + (vec >> a.group_shift)] = scale;
                store_codes(a.out8 + t * a.out8_stride + (long long)vec * VE, s[v], scale);
            }
        }
        // (a vector lies in one group: a multiple of 32 columns, or the row)
        if (QUANT == 2 && has) atomicMax(gmax + (unsigned)(vec * VE) / (unsigned)a.group, __float_as_uint(amax));
    }
    if (QUANT == 2) {
        sync();
        if (live)
            for (int k = tid; k < (int)a.n_groups; k += n) a.scales[t * a.n_groups + k] = scale_of(__uint_as_float(gmax[k]));
#pragma unroll
        for (int v = 0; v < V; v++) {
            const int vec = tid + v * n;
            if (vec < vecs)
                store_codes(a.out8 + t * a.out8_stride + (long long)vec * VE, s[v],
                            scale_of(__uint_as_float(gmax[(unsigned)(vec * VE) / (unsigned)a.group])));
        }
    }
}
// 1 / sqrt(mean + eps) of a row from the sum of its squares.
__device__ __forceinline__ float rstd_of(const NormArgs &a, float ss) {
    return __frsqrt_rn(fmaf(ss, a.inv_dim, a.eps));
}

// A vector's sum over the ranks, from rank c on and round to c - 1.
// load(r, bits): the vector as rank r holds it; RANKS of them in flight.
template <int DT, int RANKS, typename LOAD>
__device__ __forceinline__ void fold_from(const NormArgs &a, int c, float (&s)[RowBits<DT>::VE], LOAD &&load) {
    int r = c;
    for (int k0 = 0; k0 < a.p; k0 += RANKS) {
        RowBits<DT> w[RANKS];
#pragma unroll
        for (int k = 0; k < RANKS; k++)
            if (k0 + k < a.p) {
                load(r, w[k]);
                r = r + 1 == a.p ? 0 : r + 1;
            }
#pragma unroll
        for (int k = 0; k < RANKS; k++)
            if (k0 + k < a.p) {
                if (k == 0 && k0 == 0) {
#pragma unroll
                    for (int e = 0; e < RowBits<DT>::VE; e++) s[e] = w[0].get(e);
                } else {
                    add_vec<DT>(s, w[k]);
                }
            }
    }
}
// The vector at global index i of a row that lies in chunk `chunk` alone, or (-1)
// over a boundary: its elements in each chunk take that chunk's order.
template <int DT, int RANKS, typename LOAD>
__device__ __forceinline__ void fold_vector(const NormArgs &a, const Chunks &chunks, int chunk, long long i, float (&s)[RowBits<DT>::VE], LOAD &&load) {
    constexpr int VE = RowBits<DT>::VE;
    int c = chunk, last = chunk;
    if (chunk < 0) c = chunks.of(i), last = chunks.of(i + VE - 1);
    long long from = i;
#pragma unroll 1
    for (;;) {
        float f[VE];
        fold_from<DT, RANKS>(a, c, f, load);
#pragma unroll
        for (int e = 0; e < VE; e++) s[e] = i + e >= from ? f[e] : s[e];
        if (++c > last) break;
        from = chunk_start(c, chunks.base, chunks.extra);
    }
}

// Rows that 16-byte accesses reach: `warps` warps hold a row in registers, V
// vectors a thread (vector v of a thread: tid + v n), in 32 bits.  Every input is
// read once, and before anything is written (in-place outputs).
template <int DT, int V, int QUANT>
__global__ void __launch_bounds__(kNormMaxThreads, V == 1 ? 2 : 1) add_rmsnorm_kernel(const __grid_constant__ NormArgs a) {
    constexpr int VE = RowBits<DT>::VE;
    extern __shared__ unsigned group_max[];  // QUANT 2: [rows of the CTA][n_groups], bits of floats >= 0
    __shared__ float red[kNormMaxThreads / 32];
    pdl_wait();
    pdl_launch_dependents();
    const int n = a.warps * 32, in_cta = threadIdx.x / n, tid = threadIdx.x % n;
    const long long t = (long long)blockIdx.x * (blockDim.x / n) + in_cta;
    const bool live = t < a.rows;
    const int vecs = live ? (int)(a.dim / VE) : 0;
    if (QUANT == 2)
        for (int i = threadIdx.x; i < (int)(blockDim.x / n * a.n_groups); i += blockDim.x) group_max[i] = 0u;
    const Chunks chunks(a.rows * a.dim, a.p);
    int chunk = live ? chunks.of(t * a.dim) : 0;
    if ((t + 1) * a.dim > chunk_start(chunk + 1, chunks.base, chunks.extra)) chunk = -1;  // the row lies over a boundary

    float s[V][VE] = {};
    RowBits<DT> w[V];
    float ss = 0.0f;
#pragma unroll
    for (int v = 0; v < V; v++) {
        const int vec = tid + v * n;
        const bool has = vec < vecs;
        RowBits<DT> res;
        if (a.residual) res.load(row_of<DT>(a.residual, t, a.residual_stride), vec, has);
        fold_vector<DT, kNormRanks>(a, chunks, has ? chunk : 0, t * a.dim + (long long)vec * VE, s[v],
                                    [&](int r, RowBits<DT> &b) { b.load(row_of<DT>(rank_ptr(a.parts, a.p, r), t, a.part_stride), vec, has); });
        if (a.weight) w[v].load(a.weight, vec, has);
        if (a.residual) add_vec<DT>(s[v], res);
#pragma unroll
        for (int e = 0; e < VE; e++)
            if (has) ss = fmaf(s[v][e], s[v][e], ss);
    }
    ss = row_sum(ss, red, a.warps);
    if (QUANT == 2) __syncthreads();  // group_max is clear
    norm_outputs<DT, V, QUANT>(a, t, live, tid, n, rstd_of(a, ss), s, w, group_max + in_cta * a.n_groups, [] { __syncthreads(); });
}

// The same for many rows: persistent CTAs, to which a warp of its own brings the rows
// blockIdx, blockIdx + gridDim, ... of all ranks and the residual by bulk copies, `stages`
// rows ahead, a lane a matrix.  Two groups of `warps` warps take the rows in turn: one
// row's reduction is a chain of waits, and a second row in the works fills them
// (the ring alone holds too few rows for two CTAs an SM when p is 8).  Up to 256 threads a row:
// what a thread does once a row is then shared by two vectors or more.
template <int DT, int V, int QUANT>
__global__ void __launch_bounds__(2 * kRingRowThreads + 32, 1) add_rmsnorm_ring_kernel(const __grid_constant__ NormArgs a) {
    constexpr int VE = RowBits<DT>::VE;
    extern __shared__ __align__(128) unsigned char ring[];  // [stages][p + 1 matrices][dim], then QUANT 2: [2][2][n_groups]
    __shared__ float red[2][2][kRingRowThreads / 32];
    __shared__ uint64_t full[kNormMaxStages], empty[kNormMaxStages];
    __shared__ int failed, row_chunk[kNormMaxStages];
    const int n = a.warps * 32, matrices = a.p + (a.residual ? 1 : 0);
    const uint32_t row_bytes = (uint32_t)(a.dim * ElemInfo<DT>::bytes), stage_bytes = matrices * row_bytes;
    if (threadIdx.x == 0) {
        failed = 0;
        for (int s = 0; s < a.stages; s++) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], (uint32_t)a.warps);
        }
        mbar_fence_init();
    }
    if (QUANT == 2)
        for (int k = threadIdx.x; k < 4 * (int)a.n_groups; k += blockDim.x)
            reinterpret_cast<unsigned *>(ring + (size_t)a.stages * stage_bytes)[k] = 0u;
    __syncthreads();
    pdl_wait();
    pdl_launch_dependents();
    const Chunks chunks(a.rows * a.dim, a.p);
    const int group = threadIdx.x / n, tid = threadIdx.x - group * n;
    if (group == 2) {  // the loading warp
        unsigned k = 0;
        for (long long t = blockIdx.x; t < a.rows; t += gridDim.x, k++) {
            const int st = (int)(k % (unsigned)a.stages);
            const uint32_t turn = k / (unsigned)a.stages;
            const bool ok = turn == 0 || mbar_wait(&failed, a.limits, &empty[st], (turn - 1) & 1, WAIT_OF_NORM, 0);
            if (!__all_sync(0xFFFFFFFFu, ok)) break;
            if (tid == 0) {
                // the row's chunk, or -1 where it lies over a boundary
                const int c = chunks.of(t * a.dim);
                row_chunk[st] = (t + 1) * a.dim <= chunk_start(c + 1, chunks.base, chunks.extra) ? c : -1;
                mbar_expect_tx(&full[st], stage_bytes);
            }
            __syncwarp();
            for (int r = tid; r < matrices; r += 32)
                bulk_load(ring + (size_t)st * stage_bytes + (size_t)r * row_bytes,
                          r < a.p ? row_of<DT>((const void *)rank_ptr(a.parts, a.p, r), t, a.part_stride) : row_of<DT>(a.residual, t, a.residual_stride),
                          row_bytes, &full[st]);
        }
        // the CTA stays until its copies have landed
        for (unsigned q = k > (unsigned)a.stages ? k - (unsigned)a.stages : 0; q < k; q++)
            mbar_drain(&full[q % (unsigned)a.stages], (q / (unsigned)a.stages) & 1);
        return;
    }
    const int vecs = (int)(a.dim / VE), bar = 1 + group;
    unsigned *gmax = reinterpret_cast<unsigned *>(ring + (size_t)a.stages * stage_bytes) + 2 * group * (int)a.n_groups;
    RowBits<DT> w[V];
#pragma unroll
    for (int v = 0; v < V; v++)
        if (a.weight) w[v].load(a.weight, tid + v * n, tid + v * n < vecs);
    int parity = 0;
    unsigned st = (unsigned)group % (unsigned)a.stages, turn = (unsigned)group / (unsigned)a.stages;
    for (long long t = blockIdx.x + (long long)group * gridDim.x; t < a.rows; t += 2ll * gridDim.x, parity ^= 1) {
        // (a wait that ran out is recorded; the row's values are then whatever there is)
        mbar_wait(&failed, a.limits, &full[st], turn & 1, WAIT_OF_NORM, 1);
        const unsigned char *stage = ring + (size_t)st * stage_bytes;
        const int chunk = row_chunk[st];
        float s[V][VE];
        float ss = 0.0f;
#pragma unroll
        for (int v = 0; v < V; v++) {
            const int vec = tid + v * n;
            const bool has = vec < vecs;
            // (vectors past the row's end read its first one, and are not used)
            const unsigned char *at = stage + (has ? vec : 0) * 16;
            auto get = [&](int r, RowBits<DT> &b) {
                const uint4 q = *reinterpret_cast<const uint4 *>(at + (uint32_t)r * row_bytes);
                b.w[0] = q.x, b.w[1] = q.y, b.w[2] = q.z, b.w[3] = q.w;
            };
            if (chunk >= 0) {
                fold_from<DT, 4>(a, chunk, s[v], get);
            } else {
#pragma unroll
                for (int e = 0; e < VE; e++) s[v][e] = 0.0f;
                fold_vector<DT, 1>(a, chunks, has ? -1 : 0, t * a.dim + (long long)vec * VE, s[v], get);
            }
            if (a.residual) {
                RowBits<DT> res;
                get(a.p, res);
                add_vec<DT>(s[v], res);
            }
#pragma unroll
            for (int e = 0; e < VE; e++)
                if (has) ss = fmaf(s[v][e], s[v][e], ss);
        }
        __syncwarp();
        if (tid % 32 == 0) mbar_arrive(&empty[st]);
        // the row's sum over the warps (two buffers: one barrier a row)
        ss = warp_sum(ss);
        if (tid % 32 == 0) red[group][parity][tid / 32] = ss;
        row_threads_sync(bar, n);
        ss = warp_sum(tid % 32 < a.warps ? red[group][parity][tid % 32] : 0.0f);
        if (QUANT == 2)  // the last row's maxima have been used
            for (int g = tid; g < (int)a.n_groups; g += n) gmax[(parity ^ 1) * (int)a.n_groups + g] = 0u;
        norm_outputs<DT, V, QUANT>(a, t, true, tid, n, rstd_of(a, ss), s, w, gmax + parity * (int)a.n_groups, [&] { row_threads_sync(bar, n); });
        st += 2;
        if (st >= (unsigned)a.stages) st -= (unsigned)a.stages, turn++;
    }
}

// Any other row (odd widths and addresses, rows too long for the registers):
// s in shared memory in 32 bits, single elements, a CTA a row.
template <int DT>
__global__ void __launch_bounds__(kNormMaxThreads) add_rmsnorm_any_kernel(const __grid_constant__ NormArgs a) {
    extern __shared__ float row[];  // [dim], then [n_groups] maxima
    __shared__ float red[kNormMaxThreads / 32];
    unsigned *gmax = reinterpret_cast<unsigned *>(row + a.dim);
    pdl_wait();
    pdl_launch_dependents();
    const long long t = blockIdx.x, i0 = t * a.dim;
    const int dim = (int)a.dim, n = blockDim.x, groups = a.out8 ? (int)a.n_groups : 0;
    for (int k = threadIdx.x; k < groups; k += n) gmax[k] = 0u;
    const Chunks chunks(a.rows * a.dim, a.p);
    const int c_row = chunks.of(i0);
    const long long c_end = chunk_start(c_row + 1, chunks.base, chunks.extra);
    float ss = 0.0f;
    for (int j = threadIdx.x; j < dim; j += n) {
        float s = fold_element<DT>(a, i0 + j < c_end ? c_row : chunks.of(i0 + j), t * a.part_stride + j);
        if (a.residual) s += load_f<DT>(a.residual, t * a.residual_stride + j);
        row[j] = s;  // (read again by this thread alone)
        ss = fmaf(s, s, ss);
    }
    __syncthreads();  // gmax is clear, and the row's inputs are read
    ss = row_sum(ss, red, n / 32);
    const float rstd = rstd_of(a, ss);
    if (a.rstd && threadIdx.x == 0) a.rstd[t] = rstd;
    for (int j = threadIdx.x; j < dim; j += n) {
        const float s = row[j], y = s * rstd * (a.weight ? load_f<DT>(a.weight, j) : 1.0f);
        if (a.sum) store_f<DT>(a.sum, t * a.sum_stride + j, s);
        if (a.out) store_f<DT>(a.out, t * a.out_stride + j, y);
        row[j] = y;
        if (groups) atomicMax(gmax + (unsigned)j / (unsigned)a.group, __float_as_uint(fmaxf(fabsf(y), 0.0f)));
    }
    if (!groups) return;
    __syncthreads();
    for (int k = threadIdx.x; k < groups; k += n) a.scales[t * a.n_groups + k] = scale_of(__uint_as_float(gmax[k]));
    for (int j = threadIdx.x; j < dim; j += n)
        a.out8[t * a.out8_stride + j] = CodeOf(scale_of(__uint_as_float(gmax[(unsigned)j / (unsigned)a.group]))).one(row[j]);
}

struct NormGradArgs {
    long long rows, dim;
    long long dout_stride, dsum_stride, sum_stride, dx_stride;
    const void *dout, *dsum, *sum, *weight;
    const float *rstd;
    void *dx, *dweight;
    float *partial;  // [n_partial][dim]
    int n_partial;   // CTAs of the row kernel
    int stages;      // the ring kernel: rows in flight
    WaitLimits limits;
};

// Sums of a row over its threads' vectors: the dot product weight dout s, and
// this row's part of dweight.
template <int DT, int V>
__device__ __forceinline__ float grad_sums(const NormGradArgs &a, const RowBits<DT> (&dy)[V], const RowBits<DT> (&x)[V], const RowBits<DT> (&w)[V],
                                           float rstd, float (&dw)[V][16 / ElemInfo<DT>::bytes]) {
    float dot = 0.0f;
#pragma unroll
    for (int v = 0; v < V; v++)
#pragma unroll
        for (int e = 0; e < RowBits<DT>::VE; e++) {
            const float g = dy[v].get(e), f = x[v].get(e);
            dw[v][e] = fmaf(g, f * rstd, dw[v][e]);
            dot = fmaf(a.weight ? w[v].get(e) * g : g, f, dot);
        }
    return dot;
}
// dx of the row, from its dot product.
template <int DT, int V>
__device__ __forceinline__ void grad_outputs(const NormGradArgs &a, long long t, int tid, int n, const RowBits<DT> (&dy)[V], const RowBits<DT> (&x)[V],
                                             const RowBits<DT> (&ds)[V], const RowBits<DT> (&w)[V], float rstd, float dot) {
    constexpr int VE = RowBits<DT>::VE;
    const float c = __fdiv_rn(dot * rstd * rstd, (float)a.dim);
#pragma unroll
    for (int v = 0; v < V; v++) {
        const int vec = tid + v * n;
        float d[VE];
#pragma unroll
        for (int e = 0; e < VE; e++) {
            const float g = dy[v].get(e);
            d[e] = rstd * fmaf(-x[v].get(e), c, a.weight ? w[v].get(e) * g : g);
            if (a.dsum) d[e] += ds[v].get(e);
        }
        if (vec < (int)(a.dim / VE)) store_vec<DT>(row_of<DT>(a.dx, t, a.dx_stride), vec, d);
    }
}
template <int DT, int V>
__device__ __forceinline__ void grad_part(const NormGradArgs &a, int tid, int n, const float (&dw)[V][16 / ElemInfo<DT>::bytes]) {
    constexpr int VE = RowBits<DT>::VE;
    if (!a.dweight) return;
    float4 *part = reinterpret_cast<float4 *>(a.partial + (long long)blockIdx.x * a.dim);
#pragma unroll
    for (int v = 0; v < V; v++) {
        const int vec = tid + v * n;
        if (vec < (int)(a.dim / VE))
#pragma unroll
            for (int e = 0; e < VE; e += 4) part[vec * (VE / 4) + e / 4] = make_float4(dw[v][e], dw[v][e + 1], dw[v][e + 2], dw[v][e + 3]);
    }
}

// A CTA walks rows blockIdx, blockIdx + n_partial, ...; dout, sum and dsum of a
// row stay in registers as they were read (dx may be dout or dsum), and so does
// the CTA's part of dweight, a fixed set of columns a thread.
template <int DT, int V>
__global__ void __launch_bounds__(kNormMaxThreads, V == 1 ? 2 : 1) rmsnorm_grad_kernel(const __grid_constant__ NormGradArgs a) {
    constexpr int VE = RowBits<DT>::VE;
    __shared__ float red[2][kNormMaxThreads / 32];
    pdl_wait();
    pdl_launch_dependents();
    const int n = blockDim.x, vecs = (int)(a.dim / VE), tid = threadIdx.x;
    float dw[V][VE] = {};
    RowBits<DT> w[V];
#pragma unroll
    for (int v = 0; v < V; v++)
        if (a.weight) w[v].load(a.weight, tid + v * n, tid + v * n < vecs);
    int turn = 0;
    for (long long t = blockIdx.x; t < a.rows; t += gridDim.x, turn ^= 1) {
        RowBits<DT> dy[V], x[V], ds[V];
        const float rstd = a.rstd[t];
#pragma unroll
        for (int v = 0; v < V; v++) {
            const int vec = tid + v * n;
            dy[v].load(row_of<DT>(a.dout, t, a.dout_stride), vec, vec < vecs);
            x[v].load(row_of<DT>(a.sum, t, a.sum_stride), vec, vec < vecs);
            if (a.dsum) ds[v].load(row_of<DT>(a.dsum, t, a.dsum_stride), vec, vec < vecs);
        }
        float dot = grad_sums<DT, V>(a, dy, x, w, rstd, dw);
        if (!a.dx) continue;
        dot = row_sum(dot, red[turn], n / 32);  // two buffers: one barrier a row
        grad_outputs<DT, V>(a, t, tid, n, dy, x, ds, w, rstd, dot);
    }
    grad_part<DT, V>(a, tid, n, dw);
}

// The same for many rows, brought `stages` rows ahead by a warp of its own (see
// add_rmsnorm_ring_kernel).  needs dx.
template <int DT, int V>
__global__ void __launch_bounds__(kNormMaxThreads + 32, V == 1 ? 2 : 1) rmsnorm_grad_ring_kernel(const __grid_constant__ NormGradArgs a) {
    constexpr int VE = RowBits<DT>::VE;
    extern __shared__ __align__(128) unsigned char ring[];  // [stages][dout, sum, dsum][dim]
    __shared__ float red[2][kNormMaxThreads / 32], s_rstd[kNormMaxStages];
    __shared__ uint64_t full[kNormMaxStages], empty[kNormMaxStages];
    __shared__ int failed;
    const int n = blockDim.x - 32, tid = threadIdx.x, matrices = a.dsum ? 3 : 2;
    const uint32_t row_bytes = (uint32_t)(a.dim * ElemInfo<DT>::bytes), stage_bytes = matrices * row_bytes;
    if (tid == 0) {
        failed = 0;
        for (int s = 0; s < a.stages; s++) {
            mbar_init(&full[s], 2);  // the copies, and lane 3's store of rstd
            mbar_init(&empty[s], (uint32_t)n / 32);
        }
        mbar_fence_init();
    }
    __syncthreads();
    pdl_wait();
    pdl_launch_dependents();
    if (tid >= n) {  // the loading warp
        const int lane = tid - n;
        unsigned k = 0;
        for (long long t = blockIdx.x; t < a.rows; t += gridDim.x, k++) {
            const int st = (int)(k % (unsigned)a.stages);
            const uint32_t turn = k / (unsigned)a.stages;
            const bool ok = turn == 0 || mbar_wait(&failed, a.limits, &empty[st], (turn - 1) & 1, WAIT_OF_NORM, 0);
            if (!__all_sync(0xFFFFFFFFu, ok)) break;
            if (lane == 0) mbar_expect_tx(&full[st], stage_bytes);
            if (lane == 3) {
                s_rstd[st] = a.rstd[t];
                mbar_arrive(&full[st]);
            }
            __syncwarp();
            if (lane < matrices)
                bulk_load(ring + (size_t)st * stage_bytes + (size_t)lane * row_bytes,
                          lane == 0 ? row_of<DT>(a.dout, t, a.dout_stride) : lane == 1 ? row_of<DT>(a.sum, t, a.sum_stride) : row_of<DT>(a.dsum, t, a.dsum_stride),
                          row_bytes, &full[st]);
        }
        for (unsigned q = k > (unsigned)a.stages ? k - (unsigned)a.stages : 0; q < k; q++)
            mbar_drain(&full[q % (unsigned)a.stages], (q / (unsigned)a.stages) & 1);
        return;
    }
    const int vecs = (int)(a.dim / VE);
    float dw[V][VE] = {};
    RowBits<DT> w[V];
#pragma unroll
    for (int v = 0; v < V; v++)
        if (a.weight) w[v].load(a.weight, tid + v * n, tid + v * n < vecs);
    unsigned k = 0;
    for (long long t = blockIdx.x; t < a.rows; t += gridDim.x, k++) {
        const int st = (int)(k % (unsigned)a.stages), parity = (int)(k & 1);
        mbar_wait(&failed, a.limits, &full[st], (k / (unsigned)a.stages) & 1, WAIT_OF_NORM, 1);
        const unsigned char *stage = ring + (size_t)st * stage_bytes;
        RowBits<DT> dy[V], x[V], ds[V];
        auto get = [&](int r, int vec, RowBits<DT> &b) {
            const uint4 q = vec < vecs ? *(reinterpret_cast<const uint4 *>(stage + (size_t)r * row_bytes) + vec) : make_uint4(0, 0, 0, 0);
            b.w[0] = q.x, b.w[1] = q.y, b.w[2] = q.z, b.w[3] = q.w;
        };
#pragma unroll
        for (int v = 0; v < V; v++) {
            get(0, tid + v * n, dy[v]);
            get(1, tid + v * n, x[v]);
            if (a.dsum) get(2, tid + v * n, ds[v]);
        }
        const float rstd = s_rstd[st];
        __syncwarp();
        if (tid % 32 == 0) mbar_arrive(&empty[st]);
        float dot = warp_sum(grad_sums<DT, V>(a, dy, x, w, rstd, dw));
        if (tid % 32 == 0) red[parity][tid / 32] = dot;  // two buffers: one barrier a row
        row_threads_sync(1, n);
        dot = warp_sum(tid % 32 < n / 32 ? red[parity][tid % 32] : 0.0f);
        grad_outputs<DT, V>(a, t, tid, n, dy, x, ds, w, rstd, dot);
    }
    grad_part<DT, V>(a, tid, n, dw);
}

// Any other row: single elements, read once for the dot product and once more
// (from L1 or L2) for dx; the CTA's part of dweight in shared memory.
template <int DT>
__global__ void __launch_bounds__(kNormMaxThreads) rmsnorm_grad_any_kernel(const __grid_constant__ NormGradArgs a) {
    extern __shared__ float dw[];  // [dim], each column used by one thread
    __shared__ float red[2][kNormMaxThreads / 32];
    pdl_wait();
    pdl_launch_dependents();
    const int n = blockDim.x, dim = (int)a.dim;
    for (int j = threadIdx.x; j < dim; j += n) dw[j] = 0.0f;
    int turn = 0;
    for (long long t = blockIdx.x; t < a.rows; t += gridDim.x, turn ^= 1) {
        float dot = 0.0f;
        const float rstd = a.rstd[t];
#pragma unroll 4
        for (int j = threadIdx.x; j < dim; j += n) {
            const float g = load_f<DT>(a.dout, t * a.dout_stride + j), f = load_f<DT>(a.sum, t * a.sum_stride + j);
            dw[j] = fmaf(g, f * rstd, dw[j]);
            dot = fmaf(a.weight ? load_f<DT>(a.weight, j) * g : g, f, dot);
        }
        if (!a.dx) continue;
        dot = row_sum(dot, red[turn], n / 32);  // its barrier: the row is read before dx is written
        if (n == 32) __syncwarp();
        const float c = __fdiv_rn(dot * rstd * rstd, (float)a.dim);
#pragma unroll 4
        for (int j = threadIdx.x; j < dim; j += n) {
            const float g = load_f<DT>(a.dout, t * a.dout_stride + j), f = load_f<DT>(a.sum, t * a.sum_stride + j);
            float d = rstd * fmaf(-f, c, a.weight ? load_f<DT>(a.weight, j) * g : g);
            if (a.dsum) d += load_f<DT>(a.dsum, t * a.dsum_stride + j);
            store_f<DT>(a.dx, t * a.dx_stride + j, d);
        }
    }
    if (a.dweight)
        for (int j = threadIdx.x; j < dim; j += n) a.partial[(long long)blockIdx.x * a.dim + j] = dw[j];
}

// dweight from the CTAs' parts: 32 columns a CTA, 16 slices of the parts added
// side by side and then in order.
template <int DT>
__global__ void __launch_bounds__(512) rmsnorm_dweight_kernel(const __grid_constant__ NormGradArgs a) {
    __shared__ float part[16][33];
    pdl_wait();
    pdl_launch_dependents();
    const int c = threadIdx.x % 32, k = threadIdx.x / 32;
    const long long j = (long long)blockIdx.x * 32 + c;
    float d = 0.0f;
    if (j < a.dim) {
#pragma unroll 8
        for (int i = k; i < a.n_partial; i += 16) d += a.partial[(long long)i * a.dim + j];
    }
    part[k][c] = d;
    __syncthreads();
    if (k == 0 && j < a.dim) {
        for (int i = 1; i < 16; i++) d += part[i][c];
        store_f<DT>(a.dweight, j, d);
    }
}

namespace {

// CTAs of the gradient's row kernel, each with a part of dweight: two per SM
// of a GB300 (the workspace has to be sized without a handle).
constexpr size_t kNormGradCtas = 304;

size_t grad_plan(void *base, size_t rows, size_t dim, NormGradArgs *a) {
    WorkspacePlan w(base);
    const size_t k = std::min(rows, kNormGradCtas);
    float *partial = w.take<float>(k * dim);
    if (a) {
        a->partial = partial;
        a->n_partial = (int)k;
    }
    return w.used;
}

// Warps a row and vectors a thread, both powers of two, for `vecs` vectors: up to
// `most` threads of one vector, then up to 4 vectors; v is 0 where that does not hold the row.
struct RowShape {
    int v, warps;
};
RowShape row_shape(size_t vecs, int most = kNormMaxThreads) {
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
// A launch of a kernel whose dynamic shared memory may pass 48 KB.
template <typename Args>
cudaError_t launch_any(void (*kern)(Args), dim3 grid, int threads, size_t smem, cudaStream_t stream, const Args &k) {
    if (smem > 48 * 1024) {
        const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
        if (e != cudaSuccess) return e;
    }
    return launch_pdl(kern, grid, dim3((unsigned)threads), smem, stream, k);
}
// CTAs an SM and stages of a ring kernel of `threads` threads (of which registers
// allow sm_threads an SM) for rows of stage_bytes in all: at most 4 CTAs in 220 KB, at
// least 3 rows ahead if CTAs share an SM, 2 if one has it to itself.  ctas 0: the rows
// do not fit, or there are too few for the ring to turn.  Rows of under 4 warps
// stay with the other kernels, too.
struct RingShape {
    int ctas, stages;
};
RingShape ring_shape(const rar_ctx *h, size_t rows, const RowShape &shape, int threads, int sm_threads, size_t stage_bytes) {
    constexpr size_t kSmem = 220 * 1024;  // of an SM, less what the kernels declare
    if (!shape.v || shape.warps < 4) return {0, 0};
    int ctas = std::max(1, std::min(4, sm_threads / threads));
    while (ctas > 1 && kSmem / ctas / stage_bytes < 3) ctas--;
    const int stages = (int)std::min<size_t>(kSmem / ctas / stage_bytes, kNormMaxStages);
    if (stages < 2 || rows < (size_t)h->sm_count * ctas * 4) return {0, 0};
    return {ctas, stages};
}
// Threads of a CTA that takes a row of `dim` single elements: about 4 each.
int any_threads(size_t dim) { return (int)std::min<size_t>(std::max<size_t>((dim / 4 + 31) / 32 * 32, 32), kNormMaxThreads); }
int add_rmsnorm(rar_ctx *h, const rar_rmsnorm_args *a, cudaStream_t stream) {
    OpCheck c(h, "rar_add_rmsnorm");
    if (!a) return c.bad("args is NULL");
    int rc = c.dtype(a->dtype, true);
    if (rc != RAR_OK) return rc;
    if (a->p < 1 || a->p > RAR_MAX_P) return c.bad("p must be in [1, RAR_MAX_P]");
    if (a->dim < 1 || a->dim > RAR_NORM_MAX_DIM) return c.bad("dim must be in [1, RAR_NORM_MAX_DIM]");
    if (!(a->eps >= 0.0f)) return c.bad("eps must be at least 0");
    if (a->group % 32) return c.bad("group must be a multiple of 32");
    if (a->rows == 0) return RAR_OK;
    if (!a->parts) return c.bad("parts is NULL");
    if (a->out8 && !a->scales) return c.bad("scales is NULL");
    const size_t e = (size_t)elem_bytes(a->dtype);
    const size_t group = a->group ? a->group : a->dim, n_groups = (a->dim + group - 1) / group;
    MatrixSpan s;
    for (int r = 0; r < a->p; r++) {
        if ((rc = c.matrix("a part", a->parts[r], a->rows, a->dim, a->part_stride, e, e, &s)) != RAR_OK) return rc;
        c.input(s);
    }
    struct In { const char *name; const void *ptr; size_t rows, cols, stride; };
    const In ins[] = {{"residual", a->residual, a->rows, a->dim, a->residual_stride}, {"weight", a->weight, 1, a->dim, 0}};
    for (const In &i : ins)
        if (i.ptr) {
            if ((rc = c.matrix(i.name, i.ptr, i.rows, i.cols, i.stride, e, e, &s)) != RAR_OK) return rc;
            c.input(s);
        }
    struct Out { const char *name; void *ptr; size_t cols, stride, eb; };
    const Out outs[] = {{"sum", a->sum, a->dim, a->sum_stride, e}, {"out", a->out, a->dim, a->out_stride, e},
                        {"rstd", a->rstd, 1, 0, 4}, {"out8", a->out8, a->dim, a->out8_stride, 1},
                        {"scales", a->out8 ? a->scales : nullptr, n_groups, 0, 4}};
    for (const Out &o : outs)
        if (o.ptr) {
            if ((rc = c.matrix(o.name, o.ptr, a->rows, o.cols, o.stride, o.eb, o.eb, &s)) != RAR_OK) return rc;
            c.output(s);
        }
    // a row's inputs are all read before its outputs are written
    rc = c.overlaps([&](const MatrixSpan &out, const MatrixSpan &in) {
        return in.name != ins[1].name && (out.name == outs[0].name || out.name == outs[1].name);
    });
    if (rc != RAR_OK) return rc;

    DeviceGuard dg(h->device);
    if (dg.err != cudaSuccess) return cuda_fail(h, dg.err, "selecting the device");
    NormArgs k{};
    if ((rc = fill_ptrs(h, k.parts, const_cast<void *const *>(a->parts), a->p, stream)) != RAR_OK) return rc;
    auto stride = [&](size_t st, size_t cols) { return (long long)(st ? st : cols); };
    k.p = a->p;
    k.rows = (long long)a->rows;
    k.dim = (long long)a->dim;
    k.part_stride = stride(a->part_stride, a->dim);
    k.residual_stride = stride(a->residual_stride, a->dim);
    k.sum_stride = stride(a->sum_stride, a->dim);
    k.out_stride = stride(a->out_stride, a->dim);
    k.out8_stride = stride(a->out8_stride, a->dim);
    k.residual = a->residual;
    k.weight = a->weight;
    k.eps = a->eps;
    k.inv_dim = 1.0f / (float)a->dim;
    k.sum = a->sum;
    k.out = a->out;
    k.rstd = a->rstd;
    k.out8 = static_cast<uint8_t *>(a->out8);
    k.scales = a->scales;
    k.group = (long long)group;
    k.n_groups = (long long)n_groups;
    note_op_call(h, a->p, stream);
    const size_t ve = 16 / e;
    bool vec = a->dim % ve == 0;
    for (int r = 0; r < a->p && vec; r++) vec = vec16(a->parts[r], a->rows, k.part_stride, e);
    vec = vec && (!k.residual || vec16(k.residual, a->rows, k.residual_stride, e)) && (uintptr_t)k.weight % 16 == 0 &&
          (!k.sum || vec16(k.sum, a->rows, k.sum_stride, e)) && (!k.out || vec16(k.out, a->rows, k.out_stride, e)) &&
          (!k.out8 || ((uintptr_t)k.out8 % ve == 0 && (a->rows <= 1 || (size_t)k.out8_stride % ve == 0)));
    const RowShape shape = row_shape(a->dim / ve);
    if (a->rows > 0x7FFFFFFFu) return c.bad("too many rows");
    cudaError_t ce;
    if (vec && shape.v) {
        const size_t gv = group / ve;
        // a group's maximum by shuffles: its vectors are aligned lanes of one warp
        const bool lanes = group % ve == 0 && gv <= 32 && (gv & (gv - 1)) == 0;
        const int quant = !k.out8 ? 0 : lanes ? 1 : 2;
        k.group_shift = 0;
        while (lanes && ((size_t)1 << k.group_shift) < gv) k.group_shift++;
        k.warps = shape.warps;
        const size_t stage_bytes = (size_t)(a->p + (k.residual ? 1 : 0)) * a->dim * e;
        const RowShape ring_row = row_shape(a->dim / ve, kRingRowThreads);
        const int ring_threads = 2 * ring_row.warps * 32 + 32;
        const RingShape ring = ring_shape(h, a->rows, ring_row, ring_threads, 682, stage_bytes);
        if (ring.ctas) k.warps = ring_row.warps;
        k.stages = ring.stages;
        k.limits = {h->status, op_timeout_ns(h)};
        const size_t rows_cta = (size_t)std::max(1, 4 / shape.warps);
        const dim3 grid((unsigned)((a->rows + rows_cta - 1) / rows_cta)), block((unsigned)(rows_cta * shape.warps * 32));
        const size_t smem = quant == 2 ? sizeof(unsigned) * rows_cta * n_groups : 0;
        ce = dispatch_float(a->dtype, [&](auto dt) {
            return dispatch_v(ring.ctas ? ring_row.v : shape.v, [&](auto vv) {
                constexpr int DT = decltype(dt)::value, V = decltype(vv)::value;
                if (ring.ctas)
                    return launch_any(quant == 0   ? add_rmsnorm_ring_kernel<DT, V, 0>
                                      : quant == 1 ? add_rmsnorm_ring_kernel<DT, V, 1>
                                                   : add_rmsnorm_ring_kernel<DT, V, 2>,
                                      dim3((unsigned)(h->sm_count * ring.ctas)), ring_threads,
                                      ring.stages * stage_bytes + (quant == 2 ? 4 * sizeof(unsigned) * n_groups : 0), stream, k);
                return launch_pdl(quant == 0 ? add_rmsnorm_kernel<DT, V, 0> : quant == 1 ? add_rmsnorm_kernel<DT, V, 1> : add_rmsnorm_kernel<DT, V, 2>,
                                  grid, block, smem, stream, k);
            });
        });
    } else {
        const size_t smem = sizeof(float) * (a->dim + (k.out8 ? n_groups : 0));
        ce = dispatch_float(a->dtype, [&](auto dt) {
            return launch_any(add_rmsnorm_any_kernel<decltype(dt)::value>, dim3((unsigned)a->rows), any_threads(a->dim), smem, stream, k);
        });
    }
    return ce == cudaSuccess ? RAR_OK : cuda_fail(h, ce, "launching the residual norm");
}

int add_rmsnorm_grad(rar_ctx *h, const rar_rmsnorm_grad_args *a, cudaStream_t stream) {
    OpCheck c(h, "rar_add_rmsnorm_grad");
    if (!a) return c.bad("args is NULL");
    int rc = c.dtype(a->dtype, true);
    if (rc != RAR_OK) return rc;
    if (a->dim < 1 || a->dim > RAR_NORM_MAX_DIM) return c.bad("dim must be in [1, RAR_NORM_MAX_DIM]");
    const size_t e = (size_t)elem_bytes(a->dtype);
    struct In { const char *name; const void *ptr; size_t rows, cols, stride, eb; bool needed; };
    const In ins[] = {{"dout", a->dout, a->rows, a->dim, a->dout_stride, e, true},
                      {"dsum", a->dsum, a->rows, a->dim, a->dsum_stride, e, false},
                      {"sum", a->sum, a->rows, a->dim, a->sum_stride, e, true},
                      {"rstd", a->rstd, a->rows, 1, 0, 4, true},
                      {"weight", a->weight, 1, a->dim, 0, e, false}};
    MatrixSpan s;
    for (const In &i : ins)
        if (i.ptr || i.needed) {
            if ((rc = c.matrix(i.name, i.ptr, i.rows, i.cols, i.stride, i.eb, i.eb, &s)) != RAR_OK) return rc;
            c.input(s);
        }
    if (a->dx) {
        if ((rc = c.matrix("dx", a->dx, a->rows, a->dim, a->dx_stride, e, e, &s)) != RAR_OK) return rc;
        c.output(s);
    }
    if (a->dweight) {
        if ((rc = c.matrix("dweight", a->dweight, 1, a->dim, 0, e, e, &s)) != RAR_OK) return rc;
        c.output(s);
        if ((rc = c.workspace(a->workspace, a->workspace_bytes, grad_plan(nullptr, a->rows, a->dim, nullptr))) != RAR_OK)
            return rc;
    }
    const char *dx_name = "dx";
    rc = c.overlaps([&](const MatrixSpan &out, const MatrixSpan &in) {
        return std::string(out.name) == dx_name && (in.name == ins[0].name || in.name == ins[1].name);
    });
    if (rc != RAR_OK) return rc;

    DeviceGuard dg(h->device);
    if (dg.err != cudaSuccess) return cuda_fail(h, dg.err, "selecting the device");
    auto stride = [&](size_t st) { return (long long)(st ? st : a->dim); };
    NormGradArgs k{};
    k.rows = (long long)a->rows;
    k.dim = (long long)a->dim;
    k.dout_stride = stride(a->dout_stride);
    k.dsum_stride = stride(a->dsum_stride);
    k.sum_stride = stride(a->sum_stride);
    k.dx_stride = stride(a->dx_stride);
    k.dout = a->dout;
    k.dsum = a->dsum;
    k.sum = a->sum;
    k.weight = a->weight;
    k.rstd = a->rstd;
    k.dx = a->dx;
    k.dweight = a->dweight;
    grad_plan(a->workspace, a->rows, a->dim, &k);
    note_op_call(h, 1, stream);
    const size_t ve = 16 / e;
    const bool vec = a->dim % ve == 0 && vec16(k.dout, a->rows, k.dout_stride, e) && vec16(k.sum, a->rows, k.sum_stride, e) &&
                     (!k.dsum || vec16(k.dsum, a->rows, k.dsum_stride, e)) && (uintptr_t)k.weight % 16 == 0 &&
                     (!k.dx || vec16(k.dx, a->rows, k.dx_stride, e));
    const RowShape shape = row_shape(a->dim / ve);
    const size_t stage_bytes = (k.dsum ? 3 : 2) * a->dim * e;
    RingShape ring = vec && k.dx ? ring_shape(h, a->rows, shape, shape.warps * 32 + 32, shape.v == 1 ? 1088 : 544, stage_bytes) : RingShape{0, 0};
    ring.ctas = std::min(ring.ctas, (int)kNormGradCtas / h->sm_count);
    k.stages = ring.stages;
    k.limits = {h->status, op_timeout_ns(h)};
    if (ring.ctas) k.n_partial = std::min(k.n_partial, h->sm_count * ring.ctas);
    const dim3 grid((unsigned)k.n_partial);
    cudaError_t ce = dispatch_float(a->dtype, [&](auto dt) {
        constexpr int DT = decltype(dt)::value;
        cudaError_t e1 = cudaSuccess;
        if (a->rows && vec && shape.v)
            e1 = dispatch_v(shape.v, [&](auto vv) {
                if (ring.ctas)
                    return launch_any(rmsnorm_grad_ring_kernel<DT, decltype(vv)::value>, grid, shape.warps * 32 + 32, ring.stages * stage_bytes, stream, k);
                return launch_pdl(rmsnorm_grad_kernel<DT, decltype(vv)::value>, grid, dim3((unsigned)shape.warps * 32), 0, stream, k);
            });
        else if (a->rows)
            e1 = launch_any(rmsnorm_grad_any_kernel<DT>, grid, any_threads(a->dim), sizeof(float) * a->dim, stream, k);
        if (e1 == cudaSuccess && a->dweight)
            e1 = launch_pdl(rmsnorm_dweight_kernel<DT>, dim3((unsigned)((a->dim + 31) / 32)), dim3(512), 0, stream, k);
        return e1;
    });
    return ce == cudaSuccess ? RAR_OK : cuda_fail(h, ce, "launching the residual norm's gradient");
}

}  // namespace
}  // namespace rar

extern "C" {

int rar_add_rmsnorm(rar_handle h, const rar_rmsnorm_args *a, void *stream) {
    return rar::guarded(h, [&] {
        if (!h) return rar::fail(nullptr, RAR_EINVAL, "handle is NULL");
        return rar::add_rmsnorm(h, a, (cudaStream_t)stream);
    });
}

size_t rar_add_rmsnorm_grad_workspace(size_t rows, size_t dim) {
    if (dim < 1 || dim > RAR_NORM_MAX_DIM) return 0;
    return rar::grad_plan(nullptr, rows, dim, nullptr);
}

int rar_add_rmsnorm_grad(rar_handle h, const rar_rmsnorm_grad_args *a, void *stream) {
    return rar::guarded(h, [&] {
        if (!h) return rar::fail(nullptr, RAR_EINVAL, "handle is NULL");
        return rar::add_rmsnorm_grad(h, a, (cudaStream_t)stream);
    });
}

}  // extern "C"

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

#include "op_elem.cuh"
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
    int group_vecs;  // 16-byte vectors of a group, where they are 1, 2, ... 32
    int warps;       // warps a row
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

// Rows that 16-byte accesses reach: `warps` warps hold a row in registers, V
// vectors a thread (vector v of a thread: tid + v n), in 32 bits.  Every input is
// read once, and before anything is written (in-place outputs).
// QUANT: 0 none; 1 a group is `group_vecs` aligned lanes of a warp, its maximum a
// shuffle; 2 any group, maxima in shared memory (a maximum does not depend on
// the order, so neither do the codes).
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
    const long long i0 = t * a.dim;
    // the row's first chunk, and where it ends
    const int c_row = live ? chunks.of(i0) : 0;
    const long long c_end = chunk_start(c_row + 1, chunks.base, chunks.extra);
    auto first_rank = [&](long long j) { return i0 + j < c_end ? c_row : chunks.of(i0 + j); };

    float s[V][VE];
    float ss = 0.0f;
#pragma unroll
    for (int v = 0; v < V; v++) {
        const int vec = tid + v * n;
        const bool has = vec < vecs;
        const long long j = (long long)vec * VE;
        RowBits<DT> res;
        if (a.residual) res.load(row_of<DT>(a.residual, t, a.residual_stride), vec, has);
        int r = has ? first_rank(j) : 0;
        if (!has || r == first_rank(j + VE - 1)) {
            for (int k0 = 0; k0 < a.p; k0 += kNormRanks) {
                RowBits<DT> w[kNormRanks];
#pragma unroll
                for (int k = 0; k < kNormRanks; k++)
                    if (k0 + k < a.p) {
                        w[k].load(row_of<DT>(rank_ptr(a.parts, a.p, r), t, a.part_stride), vec, has);
                        r = r + 1 == a.p ? 0 : r + 1;
                    }
#pragma unroll
                for (int k = 0; k < kNormRanks; k++)
                    if (k0 + k < a.p)
#pragma unroll
                        for (int e = 0; e < VE; e++) s[v][e] = k0 + k ? s[v][e] + w[k].get(e) : w[k].get(e);
            }
        } else {  // the vector crosses a chunk boundary: each element in its own order
            float f[VE];
#pragma unroll 1
            for (int e = 0; e < VE; e++) {
                const float x = fold_element<DT>(a, first_rank(j + e), t * a.part_stride + j + e);
#pragma unroll
                for (int q = 0; q < VE; q++) f[q] = q == e ? x : e ? f[q] : 0.0f;
            }
#pragma unroll
            for (int e = 0; e < VE; e++) s[v][e] = f[e];
        }
#pragma unroll
        for (int e = 0; e < VE; e++) {
            if (a.residual) s[v][e] += res.get(e);
            if (has) ss = fmaf(s[v][e], s[v][e], ss);
        }
    }
    ss = row_sum(ss, red, a.warps);
    const float rstd = __fdiv_rn(1.0f, __fsqrt_rn(__fdiv_rn(ss, (float)a.dim) + a.eps));
    if (live && a.rstd && tid == 0) a.rstd[t] = rstd;
    if (QUANT == 2) __syncthreads();  // group_max is clear
    unsigned *gmax = group_max + in_cta * a.n_groups;
#pragma unroll
    for (int v = 0; v < V; v++) {
        const int vec = tid + v * n;
        const bool has = vec < vecs;
        if (a.sum && has) store_vec<DT>(row_of<DT>(a.sum, t, a.sum_stride), vec, s[v]);
        RowBits<DT> w;
        if (a.weight) w.load(a.weight, vec, has);
        float amax = 0.0f;
#pragma unroll
        for (int e = 0; e < VE; e++) {
            s[v][e] *= rstd;
            if (a.weight) s[v][e] *= w.get(e);
            if (QUANT && has) amax = fmaxf(amax, fabsf(s[v][e]));
        }
        if (a.out && has) store_vec<DT>(row_of<DT>(a.out, t, a.out_stride), vec, s[v]);
        if (QUANT == 1) {
            for (int o = a.group_vecs / 2; o; o /= 2) amax = fmaxf(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, o));
            const float scale = scale_of(amax);
            if (has) {
                if (vec % a.group_vecs == 0) a.scales[t * a.n_groups + vec / a.group_vecs] = scale;
                store_codes(a.out8 + t * a.out8_stride + (long long)vec * VE, s[v], scale);
            }
        }
        // (a vector lies in one group: a multiple of 32 columns, or the row)
        if (QUANT == 2 && has) atomicMax(gmax + (unsigned)(vec * VE) / (unsigned)a.group, __float_as_uint(amax));
    }
    if (QUANT == 2) {
        __syncthreads();
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
    const float rstd = __fdiv_rn(1.0f, __fsqrt_rn(__fdiv_rn(ss, (float)a.dim) + a.eps));
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
};

// A CTA walks rows blockIdx, blockIdx + n_partial, ...; dout, sum and dsum of a
// row stay in registers as they were read (dx may be dout or dsum), and so does
// the CTA's part of dweight, a fixed set of columns a thread.
template <int DT, int V>
__global__ void __launch_bounds__(kNormMaxThreads, V == 1 ? 2 : 1) rmsnorm_grad_kernel(const __grid_constant__ NormGradArgs a) {
    constexpr int VE = RowBits<DT>::VE;
    __shared__ float red[2][kNormMaxThreads / 32];
    pdl_wait();
    pdl_launch_dependents();
    const int n = blockDim.x, vecs = (int)(a.dim / VE);
    float dw[V][VE] = {};
    int turn = 0;
    for (long long t = blockIdx.x; t < a.rows; t += gridDim.x, turn ^= 1) {
        RowBits<DT> dy[V], x[V], ds[V];
        float dot = 0.0f;
        const float rstd = a.rstd[t];
#pragma unroll
        for (int v = 0; v < V; v++) {
            const int vec = threadIdx.x + v * n;
            dy[v].load(row_of<DT>(a.dout, t, a.dout_stride), vec, vec < vecs);
            x[v].load(row_of<DT>(a.sum, t, a.sum_stride), vec, vec < vecs);
            if (a.dsum) ds[v].load(row_of<DT>(a.dsum, t, a.dsum_stride), vec, vec < vecs);
        }
#pragma unroll
        for (int v = 0; v < V; v++) {
            const int vec = threadIdx.x + v * n;
            RowBits<DT> w;
            if (a.weight) w.load(a.weight, vec, vec < vecs);
#pragma unroll
            for (int e = 0; e < VE; e++) {
                const float g = dy[v].get(e), f = x[v].get(e);
                dw[v][e] = fmaf(g, f * rstd, dw[v][e]);
                dot = fmaf(a.weight ? w.get(e) * g : g, f, dot);
            }
        }
        if (!a.dx) continue;
        dot = row_sum(dot, red[turn], n / 32);  // two buffers: one barrier a row
        const float c = __fdiv_rn(dot * rstd * rstd, (float)a.dim);
#pragma unroll
        for (int v = 0; v < V; v++) {
            const int vec = threadIdx.x + v * n;
            RowBits<DT> w;
            if (a.weight) w.load(a.weight, vec, vec < vecs);
            float d[VE];
#pragma unroll
            for (int e = 0; e < VE; e++) {
                const float g = dy[v].get(e);
                d[e] = rstd * fmaf(-x[v].get(e), c, a.weight ? w.get(e) * g : g);
                if (a.dsum) d[e] += ds[v].get(e);
            }
            if (vec < vecs) store_vec<DT>(row_of<DT>(a.dx, t, a.dx_stride), vec, d);
        }
    }
    if (a.dweight) {
        float4 *part = reinterpret_cast<float4 *>(a.partial + (long long)blockIdx.x * a.dim);
#pragma unroll
        for (int v = 0; v < V; v++) {
            const int vec = threadIdx.x + v * n;
            if (vec < vecs)
#pragma unroll
                for (int e = 0; e < VE; e += 4) part[vec * (VE / 4) + e / 4] = make_float4(dw[v][e], dw[v][e + 1], dw[v][e + 2], dw[v][e + 3]);
        }
    }
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
// 16 warps of one vector, then up to 4 vectors; v is 0 where that does not hold the row.
struct RowShape {
    int v, warps;
};
RowShape row_shape(size_t vecs) {
    RowShape r{1, 1};
    while ((size_t)r.warps * 32 < vecs && r.warps * 32 < kNormMaxThreads) r.warps *= 2;
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
        k.group_vecs = lanes ? (int)gv : 0;
        k.warps = shape.warps;
        const size_t rows_cta = (size_t)std::max(1, 4 / shape.warps);
        const dim3 grid((unsigned)((a->rows + rows_cta - 1) / rows_cta)), block((unsigned)(rows_cta * shape.warps * 32));
        const size_t smem = quant == 2 ? sizeof(unsigned) * rows_cta * n_groups : 0;
        ce = dispatch_float(a->dtype, [&](auto dt) {
            return dispatch_v(shape.v, [&](auto vv) {
                constexpr int DT = decltype(dt)::value, V = decltype(vv)::value;
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
    const dim3 grid((unsigned)k.n_partial);
    cudaError_t ce = dispatch_float(a->dtype, [&](auto dt) {
        constexpr int DT = decltype(dt)::value;
        cudaError_t e1 = cudaSuccess;
        if (a->rows && vec && shape.v)
            e1 = dispatch_v(shape.v, [&](auto vv) {
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

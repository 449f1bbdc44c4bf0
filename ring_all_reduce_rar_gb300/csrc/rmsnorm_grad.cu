// rmsnorm_grad.cu -- the gradient of the residual norm (rar_add_rmsnorm_grad).
//
//   dx = dsum + rstd (weight dout - s rstd^2 mean(weight dout s))
//   dweight = sum over the rows of dout s rstd
//
// Bound by memory: 3 reads and a write an element against 9 operations.
#include "rmsnorm.cuh"

namespace rar {

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
template <int DT, int V, bool ODD>
__device__ __forceinline__ void grad_outputs(const NormGradArgs &a, long long t, const RowView<DT, ODD> &view, int tid, int n, const RowBits<DT> (&dy)[V], const RowBits<DT> (&x)[V],
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
        if (view.has(vec)) view.store(row_of<DT>(a.dx, t, a.dx_stride), vec, d);
    }
}
template <int DT, int V, bool ODD>
__device__ __forceinline__ void grad_part(const NormGradArgs &a, const RowView<DT, ODD> &view, int tid, int n, const float (&dw)[V][RowBits<DT>::VE]) {
    constexpr int VE = RowBits<DT>::VE;
    if (!a.dweight) return;
    float *part = a.partial + (long long)blockIdx.x * a.dim;
#pragma unroll
    for (int v = 0; v < V; v++) {
        const int vec = tid + v * n;
        if (!view.has(vec)) continue;
        if (!ODD) {
#pragma unroll
            for (int e = 0; e < VE; e += 4) *reinterpret_cast<float4 *>(part + vec * VE + e) = make_float4(dw[v][e], dw[v][e + 1], dw[v][e + 2], dw[v][e + 3]);
        } else {
#pragma unroll
            for (int e = 0; e < VE; e++)
                if (view.has(vec, e)) part[view.column(vec, e)] = dw[v][e];
        }
    }
}

// A CTA walks rows blockIdx, blockIdx + n_partial, ...; dout, sum and dsum of a
// row stay in registers as they were read (dx may be dout or dsum), and so does
// the CTA's part of dweight, a fixed set of columns a thread.  ODD: rows that begin
// anywhere in a 16-byte vector; n_partial is a multiple of a vector's elements
// (or every CTA has one row), so that all of a CTA's rows begin at the same place.
// Bound by latency at few rows: 1027 x 1001 float32 takes 13 us with the sum of dweight's
// parts; 8192 x 1001 40 us (against 129 by single elements).  8192 x 4096 bf16 took 63 us
// here: a row's loads, reduction and stores follow one another.
template <int DT, int V, bool ODD>
__global__ void __launch_bounds__(kNormMaxThreads, V == 1 ? 2 : 1) rmsnorm_grad_kernel(const __grid_constant__ NormGradArgs a) {
    constexpr int VE = RowBits<DT>::VE;
    __shared__ float red[2][kNormMaxThreads / 32];
    pdl_wait();
    pdl_launch_dependents();
    const int n = blockDim.x, tid = threadIdx.x;
    RowView<DT, ODD> view{0, (int)a.dim};
    if (ODD) {
        view.lo = (int)((uintptr_t)row_of<DT>(a.dout, blockIdx.x, a.dout_stride) % 16) / ElemInfo<DT>::bytes;
        view.hi += view.lo;
    }
    float dw[V][VE] = {};
    RowBits<DT> w[V];
#pragma unroll
    for (int v = 0; v < V; v++)
        if (a.weight) view.load_columns(a.weight, tid + v * n, w[v]);
    int turn = 0;
    for (long long t = blockIdx.x; t < a.rows; t += gridDim.x, turn ^= 1) {
        RowBits<DT> dy[V], x[V], ds[V];
        const float rstd = a.rstd[t];
#pragma unroll
        for (int v = 0; v < V; v++) {
            const int vec = tid + v * n;
            view.load(row_of<DT>(a.dout, t, a.dout_stride), vec, dy[v]);
            view.load(row_of<DT>(a.sum, t, a.sum_stride), vec, x[v]);
            if (a.dsum) view.load(row_of<DT>(a.dsum, t, a.dsum_stride), vec, ds[v]);
        }
        float dot = grad_sums<DT, V>(a, dy, x, w, rstd, dw);
        if (!a.dx) continue;
        dot = row_sum(dot, red[turn], n / 32);  // two buffers: one barrier a row
        grad_outputs<DT, V, ODD>(a, t, view, tid, n, dy, x, ds, w, rstd, dot);
    }
    grad_part<DT, V, ODD>(a, view, tid, n, dw);
}

// The same for many rows, brought `stages` rows ahead by a warp of its own (see
// add_rmsnorm_ring_kernel).  needs dx.  8192 x 4096 bf16: 47 us with dweight's join, 5.7 TB/s.
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
            if (lane < matrices && lane != a.limits.mute)
                bulk_load(ring + (size_t)st * stage_bytes + (size_t)lane * row_bytes,
                          lane == 0 ? row_of<DT>(a.dout, t, a.dout_stride) : lane == 1 ? row_of<DT>(a.sum, t, a.sum_stride) : row_of<DT>(a.dsum, t, a.dsum_stride),
                          row_bytes, &full[st]);
        }
        for (unsigned q = k > (unsigned)a.stages ? k - (unsigned)a.stages : 0; q < k; q++)
            if (!mbar_drain(&full[q % (unsigned)a.stages], (q / (unsigned)a.stages) & 1)) break;
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
        if (tid % 32 == 0) free_stage(&failed, &empty[st]);
        float dot = warp_sum(grad_sums<DT, V>(a, dy, x, w, rstd, dw));
        if (tid % 32 == 0) red[parity][tid / 32] = dot;  // two buffers: one barrier a row
        row_threads_sync(1, n);
        dot = warp_sum(tid % 32 < n / 32 ? red[parity][tid % 32] : 0.0f);
        grad_outputs<DT, V, false>(a, t, RowView<DT, false>{0, (int)a.dim}, tid, n, dy, x, ds, w, rstd, dot);
    }
    grad_part<DT, V, false>(a, RowView<DT, false>{0, (int)a.dim}, tid, n, dw);
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
// side by side and then in order (no atomics: the order is fixed).  6 to 8 us alone, for 608 parts
// of 1001 and 304 of 4096 columns: latency; its start overlaps the row kernel.
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

// CTAs of the gradient's row kernel at most, each with a part of dweight: four
// per SM of a GB300 (the workspace has to be sized without a handle).
constexpr size_t kNormGradCtas = 608;

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
    bool vec = a->dim % ve == 0 && (uintptr_t)k.weight % 16 == 0, alike = true;  // (as in add_rmsnorm)
    auto look = [&](const void *ptr, long long st) {
        if (!ptr) return;
        vec = vec && vec16(ptr, a->rows, st, e);
        alike = alike && ((uintptr_t)ptr - (uintptr_t)k.dout) % 16 == 0 && (a->rows <= 1 || (size_t)(st - k.dout_stride) * e % 16 == 0);
    };
    look(k.dout, k.dout_stride);
    look(k.dsum, k.dsum_stride);
    look(k.sum, k.sum_stride);
    look(k.dx, k.dx_stride);
    const RowShape shape = row_shape(vec ? a->dim / ve : (a->dim + ve - 1) / ve + 1);
    const size_t stage_bytes = (k.dsum ? 3 : 2) * a->dim * e;
    RingShape ring = vec && k.dx ? ring_shape(h, a->rows, shape, shape.warps * 32 + 32, shape.v == 1 ? 1088 : 544, 1, stage_bytes) : RingShape{0, 0};
    // 1024 threads an SM, and parts of dweight as the workspace has them
    const int ctas = std::min<int>(ring.ctas ? ring.ctas : std::max(1, 1024 / (shape.warps * 32)), (int)kNormGradCtas / h->sm_count);
    k.stages = ring.stages;
    k.limits = {h->status, op_timeout_ns(h), op_muted_rank(h)};
    k.n_partial = (int)std::min<size_t>(k.n_partial, (size_t)h->sm_count * ctas);
    const bool odd = !vec && alike && ((size_t)k.n_partial == a->rows || k.n_partial % 8 == 0);
    const dim3 grid((unsigned)k.n_partial);
    cudaError_t ce = dispatch_float(a->dtype, [&](auto dt) {
        constexpr int DT = decltype(dt)::value;
        cudaError_t e1 = cudaSuccess;
        if (a->rows && (vec || odd) && shape.v)
            e1 = dispatch_v(shape.v, [&](auto vv) {
                constexpr int V = decltype(vv)::value;
                if (ring.ctas) return launch_any(rmsnorm_grad_ring_kernel<DT, V>, grid, shape.warps * 32 + 32, ring.stages * stage_bytes, stream, k);
                return launch_pdl(vec ? rmsnorm_grad_kernel<DT, V, false> : rmsnorm_grad_kernel<DT, V, true>, grid, dim3((unsigned)shape.warps * 32), 0,
                                  stream, k);
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

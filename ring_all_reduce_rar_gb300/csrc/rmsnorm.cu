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
};

// A CTA takes a row at a time; the row's s stays in shared memory in 32
// bits, so that every input is read before anything is written (in-place
// outputs) and the norm needs no second read.
template <int DT>
__global__ void __launch_bounds__(256) add_rmsnorm_kernel(const __grid_constant__ NormArgs a) {
    extern __shared__ float row[];
    __shared__ float red[8];
    pdl_wait();
    const long long n = a.rows * a.dim, base = n / a.p, extra = n % a.p;
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    for (long long t = blockIdx.x; t < a.rows; t += gridDim.x) {
        float ss = 0.0f;
        for (long long j = threadIdx.x; j < a.dim; j += blockDim.x) {
            int r = chunk_of(t * a.dim + j, base, extra);
            float s = load_f<DT>(rank_ptr(a.parts, a.p, r), t * a.part_stride + j);
            for (int k = 1; k < a.p; k++) {
                r = r + 1 == a.p ? 0 : r + 1;
                s += load_f<DT>(rank_ptr(a.parts, a.p, r), t * a.part_stride + j);
            }
            if (a.residual) s += load_f<DT>(a.residual, t * a.residual_stride + j);
            row[j] = s;
            ss = fmaf(s, s, ss);
        }
        ss = block_sum(ss, red);  // its barrier also publishes `row`
        const float rstd = __frcp_rn(__fsqrt_rn(__fdiv_rn(ss, (float)a.dim) + a.eps));
        if (a.rstd && threadIdx.x == 0) a.rstd[t] = rstd;
        auto norm = [&](long long j) {
            const float w = a.weight ? load_f<DT>(a.weight, j) : 1.0f;
            return row[j] * rstd * w;
        };
        for (long long j = threadIdx.x; j < a.dim; j += blockDim.x) {
            if (a.sum) store_f<DT>(a.sum, t * a.sum_stride + j, row[j]);
            if (a.out) store_f<DT>(a.out, t * a.out_stride + j, norm(j));
        }
        if (a.out8) {
            for (long long g = warp; g < a.n_groups; g += blockDim.x / 32) {
                const long long lo = g * a.group, hi = lo + a.group < a.dim ? lo + a.group : a.dim;
                float amax = 0.0f;
                for (long long j = lo + lane; j < hi; j += 32) amax = fmaxf(amax, fabsf(norm(j)));
                const float scale = scale_of(warp_max(amax));
                if (lane == 0) a.scales[t * a.n_groups + g] = scale;
                for (long long j = lo + lane; j < hi; j += 32)
                    a.out8[t * a.out8_stride + j] = to_e4m3(__fdiv_rn(norm(j), scale));
            }
        }
        __syncthreads();  // `row` and `red` are reused
    }
}

struct NormGradArgs {
    long long rows, dim;
    long long dout_stride, dsum_stride, sum_stride, dx_stride;
    const void *dout, *dsum, *sum, *weight;
    const float *rstd;
    void *dx, *dweight;
    float *partial;  // [n_partial][dim]
    int n_partial;
};

template <int DT>
__global__ void __launch_bounds__(256) rmsnorm_dx_kernel(const __grid_constant__ NormGradArgs a) {
    __shared__ float red[8];
    pdl_wait();
    for (long long t = blockIdx.x; t < a.rows; t += gridDim.x) {
        float dot = 0.0f;
        for (long long j = threadIdx.x; j < a.dim; j += blockDim.x) {
            const float w = a.weight ? load_f<DT>(a.weight, j) : 1.0f;
            dot = fmaf(w * load_f<DT>(a.dout, t * a.dout_stride + j), load_f<DT>(a.sum, t * a.sum_stride + j), dot);
        }
        dot = block_sum(dot, red);
        const float rstd = a.rstd[t];
        const float c = __fdiv_rn(dot * rstd * rstd, (float)a.dim);
        for (long long j = threadIdx.x; j < a.dim; j += blockDim.x) {
            const float w = a.weight ? load_f<DT>(a.weight, j) : 1.0f;
            const float s = load_f<DT>(a.sum, t * a.sum_stride + j);
            float d = rstd * fmaf(-s, c, w * load_f<DT>(a.dout, t * a.dout_stride + j));
            if (a.dsum) d += load_f<DT>(a.dsum, t * a.dsum_stride + j);
            store_f<DT>(a.dx, t * a.dx_stride + j, d);
        }
        __syncthreads();  // `red` is reused
    }
}

// Rows [k rows / n_partial, (k + 1) rows / n_partial) of dweight's sum.
template <int DT>
__global__ void __launch_bounds__(256) rmsnorm_dweight_kernel(const __grid_constant__ NormGradArgs a) {
    pdl_wait();
    const long long j = (long long)blockIdx.x * blockDim.x + threadIdx.x;
    if (j >= a.dim) return;
    const long long lo = a.rows * blockIdx.y / a.n_partial, hi = a.rows * (blockIdx.y + 1) / a.n_partial;
    float d = 0.0f;
    for (long long t = lo; t < hi; t++)
        d = fmaf(load_f<DT>(a.dout, t * a.dout_stride + j), load_f<DT>(a.sum, t * a.sum_stride + j) * a.rstd[t], d);
    a.partial[blockIdx.y * a.dim + j] = d;
}
template <int DT>
__global__ void __launch_bounds__(256) rmsnorm_dweight_join_kernel(const __grid_constant__ NormGradArgs a) {
    pdl_wait();
    const long long j = (long long)blockIdx.x * blockDim.x + threadIdx.x;
    if (j >= a.dim) return;
    float d = 0.0f;
    for (int k = 0; k < a.n_partial; k++) d += a.partial[k * a.dim + j];
    store_f<DT>(a.dweight, j, d);
}

namespace {

constexpr int kNormPartials = 64;

size_t grad_plan(void *base, size_t rows, size_t dim, NormGradArgs *a) {
    WorkspacePlan w(base);
    const size_t k = rows < (size_t)kNormPartials ? (rows ? rows : 1) : (size_t)kNormPartials;
    float *partial = w.take<float>(k * dim);
    if (a) {
        a->partial = partial;
        a->n_partial = (int)k;
    }
    return w.used;
}

int grid_rows(const rar_ctx *h, size_t rows) {
    const size_t most = (size_t)h->sm_count * 8;
    return (int)(rows < most ? rows : most);
}

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
    const size_t smem = sizeof(float) * a->dim;
    cudaError_t ce = dispatch_float(a->dtype, [&](auto dt) {
        auto kern = add_rmsnorm_kernel<decltype(dt)::value>;
        cudaError_t e1 = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                              (int)(sizeof(float) * RAR_NORM_MAX_DIM));
        return e1 != cudaSuccess ? e1 : launch_pdl(kern, dim3(grid_rows(h, a->rows)), dim3(256), smem, stream, k);
    });
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
    cudaError_t ce = dispatch_float(a->dtype, [&](auto dt) {
        constexpr int DT = decltype(dt)::value;
        const dim3 cols((unsigned)((a->dim + 255) / 256));
        cudaError_t e1 = cudaSuccess;
        // dweight first: dx may be dout itself
        if (a->dweight) {
            e1 = launch_pdl(rmsnorm_dweight_kernel<DT>, dim3(cols.x, k.n_partial), dim3(256), 0, stream, k);
            if (e1 == cudaSuccess) e1 = launch_pdl(rmsnorm_dweight_join_kernel<DT>, cols, dim3(256), 0, stream, k);
        }
        if (e1 == cudaSuccess && a->dx && a->rows)
            e1 = launch_pdl(rmsnorm_dx_kernel<DT>, dim3(grid_rows(h, a->rows)), dim3(256), 0, stream, k);
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

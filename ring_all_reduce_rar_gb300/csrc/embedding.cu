// embedding.cu -- scaled lookup in a table held in p pieces, and the table's
// gradient (rar_embedding, rar_embedding_grad).
//
//   out[t] = scale table[tokens[t]]
//   dtables[v] = scale sum over the t with tokens[t] = v, in the order of t,
//                of dout[t]   (+ what dtables[v] held, with accumulate)
//
// Bound by memory: a read and a write an element.
#include "op_elem.cuh"
#include "op_host.h"

namespace rar {

struct EmbedArgs {
    RankPtrs pieces;
    int p;
    long long vocab, dim, n_tokens;
    long long table_stride, row_stride;  // row_stride: of out or dout
    const void *tokens;
    int index_bytes;
    float scale;
    void *out;         // lookup
    const void *dout;  // gradient
    int accumulate;
};

// Row v of a table in pieces (chunk_bounds over the vocabulary).
__device__ __forceinline__ char *table_row(const EmbedArgs &a, long long v, int elem_size) {
    const long long base = a.vocab / a.p, extra = a.vocab % a.p;
    const int r = chunk_of(v, base, extra);
    return rank_ptr(a.pieces, a.p, r) + (v - chunk_start(r, base, extra)) * a.table_stride * elem_size;
}

template <int DT>
__global__ void __launch_bounds__(256) embedding_kernel(const __grid_constant__ EmbedArgs a) {
    pdl_wait();
    for (long long t = blockIdx.x; t < a.n_tokens; t += gridDim.x) {
        const long long v = load_index(a.tokens, a.index_bytes, t);
        const bool valid = v >= 0 && v < a.vocab;
        const char *row = valid ? table_row(a, v, ElemInfo<DT>::bytes) : nullptr;
        for (long long j = threadIdx.x; j < a.dim; j += blockDim.x)
            store_f<DT>(a.out, t * a.row_stride + j, valid ? load_f<DT>(row, j) * a.scale : 0.0f);
    }
}

// A CTA per row of the table looks through all tokens.
template <int DT>
__global__ void __launch_bounds__(256) embedding_grad_kernel(const __grid_constant__ EmbedArgs a) {
    pdl_wait();
    for (long long v = blockIdx.x; v < a.vocab; v += gridDim.x) {
        char *row = table_row(a, v, ElemInfo<DT>::bytes);
        for (long long j0 = 0; j0 < a.dim; j0 += blockDim.x) {
            const long long j = j0 + threadIdx.x;
            float sum = 0.0f;
            bool any = false;
            for (long long t0 = 0; t0 < a.n_tokens; t0 += blockDim.x) {
                __shared__ unsigned hits[8];
                const long long t = t0 + threadIdx.x;
                const unsigned hit =
                    __ballot_sync(0xFFFFFFFFu, t < a.n_tokens && load_index(a.tokens, a.index_bytes, t) == v);
                __syncthreads();
                if (threadIdx.x % 32 == 0) hits[threadIdx.x / 32] = hit;
                __syncthreads();
                for (int w = 0; w < 8; w++)
                    for (unsigned m = hits[w]; m; m &= m - 1) {
                        any = true;
                        if (j < a.dim) sum += load_f<DT>(a.dout, (t0 + w * 32 + __ffs(m) - 1) * a.row_stride + j);
                    }
            }
            if (j < a.dim && (any || !a.accumulate))
                store_f<DT>(row, j, a.accumulate ? fmaf(sum, a.scale, load_f<DT>(row, j)) : sum * a.scale);
        }
    }
}

namespace {

// Checks the p pieces of a table with `vocab` rows.
template <typename Add>
int check_pieces(OpCheck &c, const char *name, const void *const *pieces, int p, size_t vocab, size_t dim, size_t stride,
                 size_t e, Add &&add) {
    if (!pieces) return c.bad(std::string(name) + " is NULL");
    for (int r = 0; r < p; r++) {
        MatrixSpan s;
        const size_t rows = vocab / p + ((size_t)r < vocab % p ? 1 : 0);
        const int rc = c.matrix(name, pieces[r], rows, dim, stride, e, e, &s);
        if (rc != RAR_OK) return rc;
        add(s);
    }
    return RAR_OK;
}

int embedding(rar_ctx *h, const rar_embedding_args *a, cudaStream_t stream) {
    OpCheck c(h, "rar_embedding");
    if (!a) return c.bad("args is NULL");
    int rc = c.dtype(a->dtype, true);
    if (rc != RAR_OK) return rc;
    if (a->p < 1 || a->p > RAR_MAX_P) return c.bad("p must be in [1, RAR_MAX_P]");
    if (a->vocab < 1 || a->dim < 1) return c.bad("vocab and dim must be at least 1");
    if (a->index_bytes != 4 && a->index_bytes != 8) return c.bad("index_bytes must be 4 or 8");
    if (a->n_tokens == 0) return RAR_OK;
    const size_t e = (size_t)elem_bytes(a->dtype);
    MatrixSpan s;
    rc = check_pieces(c, "a table piece", a->tables, a->p, a->vocab, a->dim, a->table_stride, e,
                      [&](const MatrixSpan &m) { c.input(m); });
    if (rc != RAR_OK) return rc;
    const size_t ib = (size_t)a->index_bytes;
    if ((rc = c.matrix("tokens", a->tokens, 1, a->n_tokens, 0, ib, ib, &s)) != RAR_OK) return rc;
    c.input(s);
    if ((rc = c.matrix("out", a->out, a->n_tokens, a->dim, a->out_stride, e, e, &s)) != RAR_OK) return rc;
    c.output(s);
    if ((rc = c.overlaps([](const MatrixSpan &, const MatrixSpan &) { return false; })) != RAR_OK) return rc;

    DeviceGuard dg(h->device);
    if (dg.err != cudaSuccess) return cuda_fail(h, dg.err, "selecting the device");
    EmbedArgs k{};
    if ((rc = fill_ptrs(h, k.pieces, const_cast<void *const *>(a->tables), a->p, stream)) != RAR_OK) return rc;
    k.p = a->p;
    k.vocab = (long long)a->vocab;
    k.dim = (long long)a->dim;
    k.n_tokens = (long long)a->n_tokens;
    k.table_stride = (long long)(a->table_stride ? a->table_stride : a->dim);
    k.row_stride = (long long)(a->out_stride ? a->out_stride : a->dim);
    k.tokens = a->tokens;
    k.index_bytes = a->index_bytes;
    k.scale = a->scale;
    k.out = a->out;
    note_op_call(h, a->p, stream);
    const size_t most = (size_t)h->sm_count * 8;
    const dim3 grid((unsigned)(a->n_tokens < most ? a->n_tokens : most));
    cudaError_t ce = dispatch_float(a->dtype, [&](auto dt) {
        return launch_pdl(embedding_kernel<decltype(dt)::value>, grid, dim3(256), 0, stream, k);
    });
    return ce == cudaSuccess ? RAR_OK : cuda_fail(h, ce, "launching the lookup");
}

size_t grad_workspace(size_t, size_t, size_t) { return 0; }

int embedding_grad(rar_ctx *h, const rar_embedding_grad_args *a, cudaStream_t stream) {
    OpCheck c(h, "rar_embedding_grad");
    if (!a) return c.bad("args is NULL");
    int rc = c.dtype(a->dtype, true);
    if (rc != RAR_OK) return rc;
    if (a->p < 1 || a->p > RAR_MAX_P) return c.bad("p must be in [1, RAR_MAX_P]");
    if (a->vocab < 1 || a->dim < 1) return c.bad("vocab and dim must be at least 1");
    if (a->vocab > 0x7FFFFFFFu) return c.bad("vocab must be at most 2^31 - 1");
    if (a->n_tokens > (size_t)1 << 24) return c.bad("n_tokens must be at most 2^24");
    if (a->index_bytes != 4 && a->index_bytes != 8) return c.bad("index_bytes must be 4 or 8");
    const size_t e = (size_t)elem_bytes(a->dtype);
    MatrixSpan s;
    rc = check_pieces(c, "a table piece", a->dtables, a->p, a->vocab, a->dim, a->dtable_stride, e,
                      [&](const MatrixSpan &m) { c.output(m); });
    if (rc != RAR_OK) return rc;
    const size_t ib = (size_t)a->index_bytes;
    if ((rc = c.matrix("tokens", a->tokens, 1, a->n_tokens, 0, ib, ib, &s)) != RAR_OK) return rc;
    c.input(s);
    if ((rc = c.matrix("dout", a->dout, a->n_tokens, a->dim, a->dout_stride, e, e, &s)) != RAR_OK) return rc;
    c.input(s);
    rc = c.workspace(a->workspace, a->workspace_bytes, grad_workspace(a->n_tokens, a->vocab, a->dim));
    if (rc != RAR_OK) return rc;
    if ((rc = c.overlaps([](const MatrixSpan &, const MatrixSpan &) { return false; })) != RAR_OK) return rc;

    if (a->n_tokens == 0 && a->accumulate) return RAR_OK;
    DeviceGuard dg(h->device);
    if (dg.err != cudaSuccess) return cuda_fail(h, dg.err, "selecting the device");
    EmbedArgs k{};
    if ((rc = fill_ptrs(h, k.pieces, a->dtables, a->p, stream)) != RAR_OK) return rc;
    k.p = a->p;
    k.vocab = (long long)a->vocab;
    k.dim = (long long)a->dim;
    k.n_tokens = (long long)a->n_tokens;
    k.table_stride = (long long)(a->dtable_stride ? a->dtable_stride : a->dim);
    k.row_stride = (long long)(a->dout_stride ? a->dout_stride : a->dim);
    k.tokens = a->tokens;
    k.index_bytes = a->index_bytes;
    k.scale = a->scale;
    k.dout = a->dout;
    k.accumulate = a->accumulate;
    note_op_call(h, a->p, stream);
    const size_t most = (size_t)h->sm_count * 8;
    const dim3 grid((unsigned)(a->vocab < most ? a->vocab : most));
    cudaError_t ce = dispatch_float(a->dtype, [&](auto dt) {
        return launch_pdl(embedding_grad_kernel<decltype(dt)::value>, grid, dim3(256), 0, stream, k);
    });
    return ce == cudaSuccess ? RAR_OK : cuda_fail(h, ce, "launching the lookup's gradient");
}

}  // namespace
}  // namespace rar

extern "C" {

int rar_embedding(rar_handle h, const rar_embedding_args *a, void *stream) {
    return rar::guarded(h, [&] {
        if (!h) return rar::fail(nullptr, RAR_EINVAL, "handle is NULL");
        return rar::embedding(h, a, (cudaStream_t)stream);
    });
}

size_t rar_embedding_grad_workspace(size_t n_tokens, size_t vocab, size_t dim) {
    return rar::grad_workspace(n_tokens, vocab, dim);
}

int rar_embedding_grad(rar_handle h, const rar_embedding_grad_args *a, void *stream) {
    return rar::guarded(h, [&] {
        if (!h) return rar::fail(nullptr, RAR_EINVAL, "handle is NULL");
        return rar::embedding_grad(h, a, (cudaStream_t)stream);
    });
}

}  // extern "C"

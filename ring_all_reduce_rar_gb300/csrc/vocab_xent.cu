// vocab_xent.cu -- softmax cross entropy over a vocabulary in p pieces, from
// the hidden states, with its gradients (rar_vocab_xent).
//
//   z = hidden W^T,  lse = log sum exp(z),  loss = lse - z[target]
//   G = (exp(z - lse) - onehot(target)) token_weight
//   dhidden = G W,  dweights = G^T hidden
//
// The vocabulary is walked in blocks of kBlock rows, none of which crosses
// a piece.  Pass 1 computes each logit tile and keeps its row maxima and sums
// of exponentials; they are joined to lse.  Pass 2 takes a window of blocks at a
// time: the logit tiles again, G in the 16-bit type into the workspace, and
// the two products with it.  dhidden adds up over the windows in 32 bits.
//
// All four products run on the tensor cores through one kernel (vocab_tiles.cuh):
// a pair of CTAs computes a 256 x 256 tile, and the epilogue of a tile overlaps the
// next tile's product (two accumulators).  G is rounded once, to the
// type of the products that it enters: an error of half a unit in its last place, of the
// size that rounding dhidden and dweights has anyway.
//
// Bound by the tensor cores for many tokens (8 tokens x vocab x dim operations
// against 6 if the logits were kept): 8192 tokens by 65536 x 4096 bf16 take 2.5 ms forward
// (1.76 PFLOP/s; 2.7 ms back to back) and 10.8 ms with gradients (1.63 PFLOP/s) at the power
// limit (1.37 kW, which leaves 1725 of 2070 MHz).  For few tokens by the fill of full tiles in two
// uneven waves: 16 by 32768 x 2048 take 38 us, as 256 do (134 MB of weights, 3.5 TB/s).
#include "vocab_tiles.cuh"

namespace rar {

// Joins the blocks of some tokens, a warp a token, to lse and loss; with gradients also their
// weights and hidden states, cleared where a token is left out (0 x NaN is not 0
// in dweights' sum).  Without gradients a CTA is small enough to stand beside one of
// the tile kernel and wait there for its end: 256 tokens by 32768 x 2048 took 37 us
// so and 48 us with 8 tokens a CTA; with gradients 8 tokens, whose loads are in flight
// together, took 262 us of a whole call against 281 (1024 by 32000 x 1024; the call takes 230 now).
template <bool GRAD>
constexpr int kJoinTokens = GRAD ? 8 : 4;
template <int DT, bool GRAD>
__global__ void __launch_bounds__(32 * kJoinTokens<GRAD>, GRAD ? 1 : 16) xent_join_kernel(const __grid_constant__ VocabArgs a) {
    constexpr int kTokens = kJoinTokens<GRAD>;
    __shared__ int counts[kTokens];
    pdl_wait();
    pdl_launch_dependents();
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, n = 2 * a.n_blocks;
    const long long t0 = (long long)blockIdx.x * kTokens, t = t0 + warp;
    float m = -INFINITY, s = 0.0f;
    if (t < a.tokens) {
        const long long y = load_index(a.targets, a.index_bytes, t);
        const bool ok = y >= 0 && y < a.vocab;
        const float z = a.z_target[t], tw = !ok ? 0.0f : a.token_weight ? a.token_weight[t] : 1.0f;
        for (int b0 = lane; b0 < n; b0 += 32 * 8) {
            float2 v[8];  // loads in flight together
#pragma unroll
            for (int k = 0; k < 8; k++) v[k] = __ldcg(a.stats + (long long)min(b0 + 32 * k, n - 1) * a.tokens + t);
#pragma unroll
            for (int k = 0; k < 8; k++)
                if (b0 + 32 * k < n) add_exp(m, s, v[k].x, v[k].y);
        }
#pragma unroll
        for (int o = 1; o < 32; o *= 2) {  // lanes in order: the same bits in every lane
            const float om = __shfl_xor_sync(0xFFFFFFFFu, m, o), os = __shfl_xor_sync(0xFFFFFFFFu, s, o);
            float lm = lane & o ? om : m, ls = lane & o ? os : s;
            add_exp(lm, ls, lane & o ? m : om, lane & o ? s : os);
            m = lm;
            s = ls;
        }
        if (lane == 0) {
            const float lse = m + logf(s);
            if (a.lse) a.lse[t] = lse;
            if (a.loss) a.loss[t] = ok ? lse - z : 0.0f;
            if (GRAD) {
                a.lse_ws[t] = lse;
                a.row_weight[t] = tw;
                if (isfinite(tw)) atomicMax(a.w_max, __float_as_uint(fabsf(tw)));
            }
            counts[warp] = ok;
        }
    }
    if (!GRAD) return;
    __syncthreads();
    const int vecs = (int)(a.dim / 8), total = vecs * (int)(a.tokens - t0 < kTokens ? a.tokens - t0 : kTokens);
    for (int i0 = threadIdx.x; i0 < total; i0 += 4 * 32 * kTokens) {
        uint4 q[4];  // loads in flight together
#pragma unroll
        for (int u = 0; u < 4; u++) {
            const int i = min(i0 + u * 32 * kTokens, total - 1), k = i / vecs;
            q[u] = *(reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(a.hidden) + (t0 + k) * a.hidden_stride) + (i - k * vecs));
        }
#pragma unroll
        for (int u = 0; u < 4; u++) {
            const int i = i0 + u * 32 * kTokens, k = i / vecs;
            if (i < total)
                *(reinterpret_cast<uint4 *>(static_cast<uint16_t *>(a.hidden_used) + (t0 + k) * a.dim) + (i - k * vecs)) =
                    counts[k] ? q[u] : make_uint4(0, 0, 0, 0);
        }
    }
}

namespace {

size_t plan(void *base, size_t tokens, size_t dim, size_t vocab, int p, bool grad, VocabArgs *k) {
    WorkspacePlan w(base);
    plan_blocks(vocab, p, k);
    k->stats = w.take<float2>(2 * (size_t)k->n_blocks * tokens);
    k->z_target = w.take<float>(tokens);
    k->w_max = w.take<unsigned>(1);
    k->window = 0;
    if (grad) {
        k->lse_ws = w.take<float>(tokens);
        k->row_weight = w.take<float>(tokens);
        plan_grad(w, tokens, dim, 2, k);
    }
    return w.used;
}

int vocab_xent(rar_ctx *h, const rar_vocab_xent_args *a, cudaStream_t stream) {
    OpCheck c(h, "rar_vocab_xent");
    if (!a) return c.bad("args is NULL");
    int rc = c.dtype(a->dtype, false);
    if (rc != RAR_OK) return rc;
    if (a->p < 1 || a->p > kInlineP) return c.bad("p must be in [1, 64]");
    if (a->dim < 1 || a->vocab < 1) return c.bad("dim and vocab must be at least 1");
    if (a->dim % 8) return c.bad("dim must be a multiple of 8");
    if (a->index_bytes != 4 && a->index_bytes != 8) return c.bad("index_bytes must be 4 or 8");
    if (!sizes_ok(a->tokens, a->dim, a->vocab, a->p)) return c.bad("the sizes are too large");
    const bool grad = a->dhidden || a->dweights;
    MatrixSpan s;
    if ((rc = c.matrix("hidden", a->hidden, a->tokens, a->dim, a->hidden_stride, 2, 16, &s)) != RAR_OK) return rc;
    c.input(s);
    if (!a->weights) return c.bad("weights is NULL");
    for (int r = 0; r < a->p; r++) {
        const size_t rows = a->vocab / a->p + ((size_t)r < a->vocab % a->p ? 1 : 0);
        if ((rc = c.matrix("a weight piece", a->weights[r], rows, a->dim, a->weight_stride, 2, 16, &s)) != RAR_OK) return rc;
        c.input(s);
        if (a->dweights) {
            if ((rc = c.matrix("a dweight piece", a->dweights[r], rows, a->dim, a->dweight_stride, 2, 16, &s)) != RAR_OK)
                return rc;
            c.output(s);
        }
    }
    const size_t ib = (size_t)a->index_bytes;
    if ((rc = c.matrix("targets", a->targets, 1, a->tokens, 0, ib, ib, &s)) != RAR_OK) return rc;
    c.input(s);
    if (a->token_weight) {
        if ((rc = c.matrix("token_weight", a->token_weight, 1, a->tokens, 0, 4, 4, &s)) != RAR_OK) return rc;
        c.input(s);
    }
    struct Out { const char *name; void *ptr; size_t rows, cols, stride, eb, align; };
    const Out outs[] = {{"loss", a->loss, 1, a->tokens, 0, 4, 4}, {"lse", a->lse, 1, a->tokens, 0, 4, 4},
                        {"dhidden", a->dhidden, a->tokens, a->dim, a->dhidden_stride, 2, 16}};
    for (const Out &o : outs)
        if (o.ptr) {
            if ((rc = c.matrix(o.name, o.ptr, o.rows, o.cols, o.stride, o.eb, o.align, &s)) != RAR_OK) return rc;
            c.output(s);
        }
    VocabArgs k{};
    const size_t need = plan(nullptr, a->tokens, a->dim, a->vocab, a->p, grad, &k);
    if ((rc = c.workspace(a->workspace, a->workspace_bytes, need)) != RAR_OK) return rc;
    if ((rc = c.overlaps([](const MatrixSpan &, const MatrixSpan &) { return false; })) != RAR_OK) return rc;
    if (a->tokens == 0 && !a->dweights) return RAR_OK;

    DeviceGuard dg(h->device);
    if (dg.err != cudaSuccess) return cuda_fail(h, dg.err, "selecting the device");
    plan(a->workspace, a->tokens, a->dim, a->vocab, a->p, grad, &k);
    auto stride = [&](size_t st) { return (long long)(st ? st : a->dim); };
    for (int r = 0; r < a->p; r++) {
        k.w.inl[r] = const_cast<void *>(a->weights[r]);
        k.dw.inl[r] = a->dweights ? a->dweights[r] : nullptr;
    }
    k.p = a->p;
    k.tokens = (long long)a->tokens;
    k.dim = (long long)a->dim;
    k.vocab = (long long)a->vocab;
    k.hidden_stride = stride(a->hidden_stride);
    k.weight_stride = stride(a->weight_stride);
    k.dhidden_stride = stride(a->dhidden_stride);
    k.dweight_stride = stride(a->dweight_stride);
    k.hidden = a->hidden;
    k.targets = a->targets;
    k.index_bytes = a->index_bytes;
    k.token_weight = a->token_weight;
    k.scale = 1.0f;
    k.loss = a->loss;
    k.lse = a->lse;
    k.dhidden = a->dhidden;
    k.want_dw = a->dweights != nullptr;
    note_op_call(h, a->p, stream);

    k.limits = {h->status, op_timeout_ns(h), op_muted_rank(h)};

    CallMaps m;
    if (k.tokens && !make_maps(a->dtype, k, &m)) return fail(h, RAR_ECUDA, "rar_vocab_xent: the driver refused a tensor map");

    auto run = [&](auto dt) {
        constexpr int DT = decltype(dt)::value;
        cudaError_t e = cudaSuccess;
        if (!k.tokens) return clear_dweights(k, stream);
        const bool sums = k.dim > 64 * kStepsPerSum;
        e = sums ? launch_tiles<TILES_STATS_SUMS, DT>(h, k, m.logits, 0, k.n_blocks, stream)
                 : launch_tiles<TILES_STATS, DT>(h, k, m.logits, 0, k.n_blocks, stream);
        const int join = grad ? kJoinTokens<true> : kJoinTokens<false>;
        if (e == cudaSuccess)
            e = launch_pdl(grad ? xent_join_kernel<DT, true> : xent_join_kernel<DT, false>, dim3((unsigned)((k.tokens + join - 1) / join)), dim3(32 * join), 0, stream, k);
        if (e != cudaSuccess || !grad) return e;
        return sums ? launch_gradients<TILES_G_SUMS, DT>(h, k, m, stream) : launch_gradients<TILES_G, DT>(h, k, m, stream);
    };
    cudaError_t ce = a->dtype == RAR_BFLOAT16 ? run(IntC<DT_BF16>{}) : run(IntC<DT_F16>{});
    return ce == cudaSuccess ? RAR_OK : cuda_fail(h, ce, "launching the cross entropy");
}

}  // namespace
}  // namespace rar

extern "C" {

size_t rar_vocab_xent_workspace(size_t tokens, size_t dim, size_t vocab, int p, int grad) {
    if (!rar::sizes_ok(tokens, dim, vocab, p)) return 0;
    rar::VocabArgs k{};
    return rar::plan(nullptr, tokens, dim, vocab, p, grad != 0, &k);
}

int rar_vocab_xent(rar_handle h, const rar_vocab_xent_args *a, void *stream) {
    return rar::guarded(h, [&] {
        if (!h) return rar::fail(nullptr, RAR_EINVAL, "handle is NULL");
        return rar::vocab_xent(h, a, (cudaStream_t)stream);
    });
}

}  // extern "C"

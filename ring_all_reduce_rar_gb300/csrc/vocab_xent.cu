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
// Bound by the tensor cores for many tokens (8 tokens x vocab x dim
// operations against 6 if the logits were kept), by memory for few.
#include <algorithm>

#include "op_elem.cuh"
#include "op_host.h"

namespace rar {

constexpr int kBlock = 256;  // vocabulary rows of a block

struct XentArgs {
    RankPtrs w, dw;  // pieces
    int p;
    long long tokens, dim, vocab;
    long long hidden_stride, weight_stride, dhidden_stride, dweight_stride;
    const void *hidden, *targets;
    int index_bytes;
    const float *token_weight;
    float *loss, *lse;
    void *dhidden;
    bool want_dw;
    // blocks
    long long base, extra;     // chunk_bounds(vocab, p)
    long long nb_big, nb_small;  // blocks of a piece of base + 1 / base rows
    long long n_blocks;
    // workspace
    float2 *stats;        // [n_blocks][tokens]: max, sum of exp(z - max)
    float *z_target;      // [tokens]
    float *lse_ws;        // [tokens]
    float *row_weight;    // [tokens] scaled token_weight, 0 where left out
    unsigned *w_max;      // bits of the largest finite |token_weight|
    void *hidden_used;    // [tokens][dim]: hidden, zeros where left out
    void *g;              // [tokens][window * kBlock]
    float *dh_acc;        // [tokens][dim]
    long long window;     // blocks of a window
};

struct BlockOf {
    int piece;
    long long row;   // first row in the piece
    int rows;        // 1 .. kBlock
    long long first;  // its index in the vocabulary
};
__device__ __forceinline__ BlockOf block_of(const XentArgs &a, long long b) {
    BlockOf o;
    const long long big = a.extra * a.nb_big;
    long long k;
    if (b < big) {
        o.piece = (int)(b / a.nb_big);
        k = b % a.nb_big;
    } else {
        o.piece = (int)(a.extra + (b - big) / a.nb_small);
        k = (b - big) % a.nb_small;
    }
    o.row = k * kBlock;
    const long long piece_rows = a.base + (o.piece < a.extra ? 1 : 0);
    o.rows = (int)(piece_rows - o.row < kBlock ? piece_rows - o.row : kBlock);
    o.first = chunk_start(o.piece, a.base, a.extra) + o.row;
    return o;
}

// fp16 holds nothing below 6e-8, so G is scaled by a power of two that puts the
// largest token weight near 2^14; the products undo it.  bf16 needs none.
template <int DT>
__device__ __forceinline__ int g_exponent(const XentArgs &a) {
    if constexpr (DT != DT_F16) return 0;
    const float m = __uint_as_float(*a.w_max);
    if (!(m > 0.0f)) return 0;
    const int e = 14 - ilogbf(m);
    return e > 120 ? 120 : e < -120 ? -120 : e;
}

// C[64][64] of one CTA of 256 threads, 4 x 4 a thread: sum over k of
// A(i, k) B(j, k).
template <typename FA, typename FB>
__device__ __forceinline__ void tile_product(float (&acc)[4][4], long long K, FA &&fa, FB &&fb) {
    __shared__ float sa[16][65], sb[16][65];
    const int ti = threadIdx.x / 16, tj = threadIdx.x % 16;
    for (long long k0 = 0; k0 < K; k0 += 16) {
        for (int x = threadIdx.x; x < 64 * 16; x += 256) {
            const int i = x / 16, k = x % 16;
            sa[k][i] = k0 + k < K ? fa(i, k0 + k) : 0.0f;
            sb[k][i] = k0 + k < K ? fb(i, k0 + k) : 0.0f;
        }
        __syncthreads();
#pragma unroll
        for (int k = 0; k < 16; k++)
#pragma unroll
            for (int i = 0; i < 4; i++)
#pragma unroll
                for (int j = 0; j < 4; j++) acc[i][j] = fmaf(sa[k][ti * 4 + i], sb[k][tj * 4 + j], acc[i][j]);
        __syncthreads();
    }
}

// The logits of 64 tokens x 64 rows of a block; rows beyond it are -inf.
template <int DT>
__device__ __forceinline__ void logits_tile(const XentArgs &a, long long t0, const BlockOf &b, int j0, float (&acc)[4][4]) {
    const char *w = rank_ptr(a.w, a.p, b.piece);
    tile_product(
        acc, a.dim, [&](int i, long long k) { return t0 + i < a.tokens ? load_f<DT>(a.hidden, (t0 + i) * a.hidden_stride + k) : 0.0f; },
        [&](int j, long long k) { return j0 + j < b.rows ? load_f<DT>(w, (b.row + j0 + j) * a.weight_stride + k) : 0.0f; });
    const int tj = threadIdx.x % 16;
    for (int i = 0; i < 4; i++)
        for (int j = 0; j < 4; j++)
            if (j0 + tj * 4 + j >= b.rows) acc[i][j] = -INFINITY;
}

// Pass 1: row maxima and sums of exponentials of a block, and the target's logit.
template <int DT>
__global__ void __launch_bounds__(256) xent_stats_kernel(const __grid_constant__ XentArgs a) {
    pdl_wait();
    if (blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x == 0) *a.w_max = 0u;
    const BlockOf b = block_of(a, blockIdx.x);
    const int ti = threadIdx.x / 16, tj = threadIdx.x % 16;
    for (long long t0 = (long long)blockIdx.y * 64; t0 < a.tokens; t0 += (long long)gridDim.y * 64) {
        float m[4], s[4];
        for (int i = 0; i < 4; i++) m[i] = -INFINITY, s[i] = 0.0f;
        for (int j0 = 0; j0 < b.rows; j0 += 64) {
            float acc[4][4] = {};
            logits_tile<DT>(a, t0, b, j0, acc);
            for (int i = 0; i < 4; i++) {
                const long long t = t0 + ti * 4 + i;
                if (t < a.tokens) {
                    const long long y = load_index(a.targets, a.index_bytes, t) - b.first - j0 - tj * 4;
                    for (int j = 0; j < 4; j++)
                        if (y == j && j0 + tj * 4 + j < b.rows) a.z_target[t] = acc[i][j];
                }
                for (int j = 0; j < 4; j++) {
                    const float z = acc[i][j], top = fmaxf(m[i], z);
                    if (z == -INFINITY) continue;
                    s[i] = s[i] * expf(m[i] - top) + expf(z - top);
                    m[i] = top;
                }
            }
        }
        for (int i = 0; i < 4; i++) {
            for (int o = 1; o < 16; o *= 2) {
                const float om = __shfl_xor_sync(0xFFFFFFFFu, m[i], o), os = __shfl_xor_sync(0xFFFFFFFFu, s[i], o);
                const float top = fmaxf(m[i], om);
                s[i] = top == -INFINITY ? s[i] + os : s[i] * expf(m[i] - top) + os * expf(om - top);
                m[i] = top;
            }
            const long long t = t0 + ti * 4 + i;
            if (tj == 0 && t < a.tokens) a.stats[(long long)blockIdx.x * a.tokens + t] = make_float2(m[i], s[i]);
        }
    }
}

// Joins a token's blocks to lse and loss; with gradients also its weight and
// its hidden state, cleared where the token is left out (0 x NaN is not 0 in
// dweights' sum).  A CTA a token.
template <int DT, bool GRAD>
__global__ void __launch_bounds__(256) xent_join_kernel(const __grid_constant__ XentArgs a) {
    __shared__ float red[8], redm[8];
    pdl_wait();
    const long long t = blockIdx.x;
    float m = -INFINITY;
    for (long long b = threadIdx.x; b < a.n_blocks; b += blockDim.x) m = fmaxf(m, a.stats[b * a.tokens + t].x);
    m = warp_max(m);
    if (threadIdx.x % 32 == 0) redm[threadIdx.x / 32] = m;
    __syncthreads();
    for (int w = 0; w < 8; w++) m = fmaxf(m, redm[w]);
    float s = 0.0f;
    for (long long b = threadIdx.x; b < a.n_blocks; b += blockDim.x) {
        const float2 v = a.stats[b * a.tokens + t];
        if (v.y != 0.0f) s = fmaf(v.y, expf(v.x - m), s);  // (a NaN sum of a block of NaN is kept)
    }
    s = block_sum(s, red);
    const float lse = m + logf(s);
    const long long y = load_index(a.targets, a.index_bytes, t);
    const bool counts = y >= 0 && y < a.vocab;
    if (threadIdx.x == 0) {
        if (a.lse) a.lse[t] = lse;
        if (a.loss) a.loss[t] = counts ? lse - a.z_target[t] : 0.0f;
        if (GRAD) {
            const float w = !counts ? 0.0f : a.token_weight ? a.token_weight[t] : 1.0f;
            a.lse_ws[t] = lse;
            a.row_weight[t] = w;
            if (isfinite(w)) atomicMax(a.w_max, __float_as_uint(fabsf(w)));
        }
    }
    if (GRAD)
        for (long long j = threadIdx.x; j < a.dim; j += blockDim.x)
            store_f<DT>(a.hidden_used, t * a.dim + j, counts ? load_f<DT>(a.hidden, t * a.hidden_stride + j) : 0.0f);
}

// Pass 2: G of a window.
template <int DT>
__global__ void __launch_bounds__(256) xent_g_kernel(const __grid_constant__ XentArgs a, long long b0) {
    pdl_wait();
    const BlockOf b = block_of(a, b0 + blockIdx.x);
    const int ti = threadIdx.x / 16, tj = threadIdx.x % 16, ge = g_exponent<DT>(a);
    for (long long t0 = (long long)blockIdx.y * 64; t0 < a.tokens; t0 += (long long)gridDim.y * 64)
        for (int j0 = 0; j0 < kBlock; j0 += 64) {
            float acc[4][4] = {};
            logits_tile<DT>(a, t0, b, j0, acc);
            for (int i = 0; i < 4; i++) {
                const long long t = t0 + ti * 4 + i;
                if (t >= a.tokens) continue;
                const float w = ldexpf(a.row_weight[t], ge), lse = a.lse_ws[t];
                const long long y = load_index(a.targets, a.index_bytes, t) - b.first - j0 - tj * 4;
                for (int j = 0; j < 4; j++) {
                    const int col = j0 + tj * 4 + j;
                    float g = 0.0f;
                    if (col < b.rows && w != 0.0f) g = (expf(acc[i][j] - lse) - (y == j ? 1.0f : 0.0f)) * w;
                    store_f<DT>(a.g, (t * a.window + blockIdx.x) * kBlock + col, g);
                }
            }
        }
}

// dhidden's sum over a window of nb blocks.
template <int DT>
__global__ void __launch_bounds__(256) xent_dh_kernel(const __grid_constant__ XentArgs a, long long b0, long long nb) {
    pdl_wait();
    const long long d0 = (long long)blockIdx.x * 64;
    const float undo = ldexpf(1.0f, -g_exponent<DT>(a));
    const int ti = threadIdx.x / 16, tj = threadIdx.x % 16;
    for (long long t0 = (long long)blockIdx.y * 64; t0 < a.tokens; t0 += (long long)gridDim.y * 64) {
        float acc[4][4] = {};
        for (long long k = 0; k < nb; k++) {
            const BlockOf b = block_of(a, b0 + k);
            const char *w = rank_ptr(a.w, a.p, b.piece);
            tile_product(
                acc, b.rows,
                [&](int i, long long v) { return t0 + i < a.tokens ? load_f<DT>(a.g, ((t0 + i) * a.window + k) * kBlock + v) : 0.0f; },
                [&](int j, long long v) { return d0 + j < a.dim ? load_f<DT>(w, (b.row + v) * a.weight_stride + d0 + j) : 0.0f; });
        }
        for (int i = 0; i < 4; i++)
            for (int j = 0; j < 4; j++) {
                const long long t = t0 + ti * 4 + i, d = d0 + tj * 4 + j;
                if (t >= a.tokens || d >= a.dim) continue;
                float v = acc[i][j] * undo + (b0 ? a.dh_acc[t * a.dim + d] : 0.0f);
                if (b0 + nb < a.n_blocks) a.dh_acc[t * a.dim + d] = v;
                else store_f<DT>(a.dhidden, t * a.dhidden_stride + d, v);
            }
    }
}

// dweights of a window: a block's 64-row quarter x 64 columns a CTA.
template <int DT>
__global__ void __launch_bounds__(256) xent_dw_kernel(const __grid_constant__ XentArgs a, long long b0) {
    pdl_wait();
    const long long k = blockIdx.x, d0 = (long long)blockIdx.y * 64;
    const BlockOf b = block_of(a, b0 + k);
    const float undo = ldexpf(1.0f, -g_exponent<DT>(a));
    const int ti = threadIdx.x / 16, tj = threadIdx.x % 16;
    for (int v0 = 0; v0 < b.rows; v0 += 64) {
        float acc[4][4] = {};
        tile_product(
            acc, a.tokens,
            [&](int i, long long t) { return load_f<DT>(a.g, (t * a.window + k) * kBlock + v0 + i); },
            [&](int j, long long t) { return d0 + j < a.dim ? load_f<DT>(a.hidden_used, t * a.dim + d0 + j) : 0.0f; });
        for (int i = 0; i < 4; i++)
            for (int j = 0; j < 4; j++) {
                const int v = v0 + ti * 4 + i;
                const long long d = d0 + tj * 4 + j;
                if (v < b.rows && d < a.dim)
                    store_f<DT>(rank_ptr(a.dw, a.p, b.piece), (b.row + v) * a.dweight_stride + d, acc[i][j] * undo);
            }
    }
}

namespace {

constexpr size_t kWindowBytes = (size_t)256 << 20;  // of G

void plan_blocks(size_t vocab, int p, XentArgs *k) {
    k->base = (long long)(vocab / p);
    k->extra = (long long)(vocab % p);
    k->nb_big = (k->base + 1 + kBlock - 1) / kBlock;
    k->nb_small = (k->base + kBlock - 1) / kBlock;
    k->n_blocks = k->extra * k->nb_big + (p - k->extra) * k->nb_small;
}

size_t plan(void *base, size_t tokens, size_t dim, size_t vocab, int p, bool grad, XentArgs *k) {
    WorkspacePlan w(base);
    plan_blocks(vocab, p, k);
    const size_t n_blocks = (size_t)k->n_blocks;
    k->stats = w.take<float2>(n_blocks * tokens);
    k->z_target = w.take<float>(tokens);
    k->w_max = w.take<unsigned>(1);
    k->window = 0;
    if (grad) {
        k->lse_ws = w.take<float>(tokens);
        k->row_weight = w.take<float>(tokens);
        k->hidden_used = w.take<uint16_t>(tokens * dim);
        size_t window = kWindowBytes / (sizeof(uint16_t) * kBlock * std::max<size_t>(tokens, 1));
        window = std::min(std::max<size_t>(window, 1), n_blocks);
        k->window = (long long)window;
        k->g = w.take<uint16_t>(tokens * window * kBlock);
        k->dh_acc = w.take<float>(window < n_blocks ? tokens * dim : 0);
    }
    return w.used;
}

bool sizes_ok(size_t tokens, size_t dim, size_t vocab, int p) {
    const size_t most = (size_t)1 << 40;
    return p >= 1 && p <= kInlineP && dim >= 1 && vocab >= 1 && tokens <= most && dim <= most / 1024 && vocab <= 0x7FFFFFFFu &&
           tokens <= (((size_t)1 << 58) / std::max(dim, vocab)) && dim % 8 == 0;
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
    XentArgs k{};
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
    k.loss = a->loss;
    k.lse = a->lse;
    k.dhidden = a->dhidden;
    k.want_dw = a->dweights != nullptr;
    note_op_call(h, a->p, stream);

    auto run = [&](auto dt) {
        constexpr int DT = decltype(dt)::value;
        const unsigned ty = (unsigned)std::min<long long>((k.tokens + 63) / 64, 4096);
        const unsigned dx = (unsigned)((k.dim + 63) / 64);
        cudaError_t e = cudaSuccess;
        if (k.tokens) {
            e = launch_pdl(xent_stats_kernel<DT>, dim3((unsigned)k.n_blocks, ty), dim3(256), 0, stream, k);
            if (e == cudaSuccess)
                e = launch_pdl(grad ? xent_join_kernel<DT, true> : xent_join_kernel<DT, false>, dim3((unsigned)k.tokens), dim3(256), 0, stream, k);
        }
        if (!grad) return e;
        for (long long b0 = 0; b0 < k.n_blocks && e == cudaSuccess; b0 += k.window) {
            const long long nb = std::min(k.window, k.n_blocks - b0);
            if (k.tokens) e = launch_pdl(xent_g_kernel<DT>, dim3((unsigned)nb, ty), dim3(256), 0, stream, k, b0);
            if (e == cudaSuccess && k.dhidden && k.tokens)
                e = launch_pdl(xent_dh_kernel<DT>, dim3(dx, ty), dim3(256), 0, stream, k, b0, nb);
            if (e == cudaSuccess && k.want_dw)
                e = launch_pdl(xent_dw_kernel<DT>, dim3((unsigned)nb, dx), dim3(256), 0, stream, k, b0);
        }
        return e;
    };
    cudaError_t ce = a->dtype == RAR_BFLOAT16 ? run(IntC<DT_BF16>{}) : run(IntC<DT_F16>{});
    return ce == cudaSuccess ? RAR_OK : cuda_fail(h, ce, "launching the cross entropy");
}

}  // namespace
}  // namespace rar

extern "C" {

size_t rar_vocab_xent_workspace(size_t tokens, size_t dim, size_t vocab, int p, int grad) {
    if (!rar::sizes_ok(tokens, dim, vocab, p)) return 0;
    rar::XentArgs k{};
    return rar::plan(nullptr, tokens, dim, vocab, p, grad != 0, &k);
}

int rar_vocab_xent(rar_handle h, const rar_vocab_xent_args *a, void *stream) {
    return rar::guarded(h, [&] {
        if (!h) return rar::fail(nullptr, RAR_EINVAL, "handle is NULL");
        return rar::vocab_xent(h, a, (cudaStream_t)stream);
    });
}

}  // extern "C"

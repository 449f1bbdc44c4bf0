// rmsnorm.cu -- the residual stream's join with the ranks' partial results and
// its RMS norm with an optional 8-bit output (rar_add_rmsnorm).
//
//   s = residual + x_c + x_(c+1) + ...   (c: the element's chunk, ring order)
//   rstd = 1 / sqrt(mean(s^2) + eps),  y = s rstd weight
//
// Bound by memory: (p + 1) reads and 2 writes an element against p + 6
// operations.  Few rows are bound by latency: 4 rows of 2048 with 8 parts and 8-bit output
// take 6 us, and a call in a stream of calls 11.7, or 10.4 without the check of its pointers, which is
// the host's time for one.
#include "rmsnorm.cuh"

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

// What a row's threads do once they hold its s: the norm and every output.
// QUANT: 0 none; 1 a group is 2^group_shift aligned lanes of a warp, its maximum a
// shuffle; 2 any group, maxima in shared memory (a maximum does not depend on
// the order, so neither do the codes).  n threads a row; gmax: the row's maxima,
// clear (QUANT 2).  All threads that sync() joins come here.
template <int DT, int V, int QUANT, bool ODD, typename SYNC>
__device__ __forceinline__ void norm_outputs(const NormArgs &a, long long t, const RowView<DT, ODD> &view, int tid, int n, float rstd,
                                             float (&s)[V][RowBits<DT>::VE], const RowBits<DT> (&w)[V], unsigned *gmax, SYNC &&sync) {
    constexpr int VE = RowBits<DT>::VE;
    static_assert(!ODD || QUANT != 1, "groups of an odd row are not aligned vectors");
    const bool live = view.hi > 0;
    auto group_of = [&](int vec, int e) { return (unsigned)view.column(vec, e) / (unsigned)a.group; };
    if (live && a.rstd && tid == 0) a.rstd[t] = rstd;
#pragma unroll
    for (int v = 0; v < V; v++) {
        const int vec = tid + v * n;
        const bool has = view.has(vec);
        if (a.sum && has) view.store(row_of<DT>(a.sum, t, a.sum_stride), vec, s[v]);
        float amax = 0.0f;
#pragma unroll
        for (int e = 0; e < VE; e++) {
            s[v][e] *= rstd;
            if (a.weight) s[v][e] *= w[v].get(e);
            if (QUANT && view.has(vec, e)) amax = fmaxf(amax, fabsf(s[v][e]));
        }
        if (a.out && has) view.store(row_of<DT>(a.out, t, a.out_stride), vec, s[v]);
        if (QUANT == 1) {
            for (int o = 1 << a.group_shift >> 1; o; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, o));
            const float scale = scale_of(amax);
            if (has) {
                if ((vec & ((1 << a.group_shift) - 1)) == 0) a.scales[t * a.n_groups + (vec >> a.group_shift)] = scale;
                store_codes(a.out8 + t * a.out8_stride + (long long)vec * VE, s[v], scale);
            }
        }
        if (QUANT == 2 && has) {
            // (groups are multiples of 32 columns, or the row: an aligned vector lies in
            // one, an odd one in two at most)
            if (!ODD) {
                atomicMax(gmax + group_of(vec, 0), __float_as_uint(amax));
            } else {
#pragma unroll
                for (int e = 0; e < VE; e++)
                    if (view.has(vec, e) && (e == VE - 1 || !view.has(vec, e + 1) || group_of(vec, e) != group_of(vec, e + 1))) {
                        float part = 0.0f;
#pragma unroll
                        for (int q = 0; q <= e; q++)
                            if (view.has(vec, q) && group_of(vec, q) == group_of(vec, e)) part = fmaxf(part, fabsf(s[v][q]));
                        atomicMax(gmax + group_of(vec, e), __float_as_uint(part));
                    }
            }
        }
    }
    if (QUANT == 2) {
        sync();
        if (live)
            for (int k = tid; k < (int)a.n_groups; k += n) a.scales[t * a.n_groups + k] = scale_of(__uint_as_float(gmax[k]));
#pragma unroll
        for (int v = 0; v < V; v++) {
            const int vec = tid + v * n;
            if (!view.has(vec)) continue;
            uint8_t *to = a.out8 + t * a.out8_stride + view.column(vec, 0);
            if (!ODD) {
                store_codes(to, s[v], scale_of(__uint_as_float(gmax[group_of(vec, 0)])));
            } else {
#pragma unroll
                for (int e = 0; e < VE; e++)
                    if (view.has(vec, e)) to[e] = CodeOf(scale_of(__uint_as_float(gmax[group_of(vec, e)]))).one(s[v][e]);
            }
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
// The vector at global index i of a row [lo, hi) that lies in chunk `chunk` alone, or
// (-1) over a boundary: its elements in each chunk take that chunk's order.
template <int DT, int RANKS, typename LOAD>
__device__ __forceinline__ void fold_vector(const NormArgs &a, const Chunks &chunks, int chunk, long long i, long long lo, long long hi,
                                            float (&s)[RowBits<DT>::VE], LOAD &&load) {
    constexpr int VE = RowBits<DT>::VE;
    int c = chunk, last = chunk;
    if (chunk < 0) c = chunks.of(i > lo ? i : lo), last = chunks.of(i + VE < hi ? i + VE - 1 : hi - 1);
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

// `warps` warps hold a row in registers, V vectors a thread (vector v of a
// thread: tid + v n), in 32 bits.  Every input is read once, and before anything is
// written (in-place outputs).  ODD: rows that begin anywhere in a 16-byte vector, at
// the same place in all matrices.  One CTA a row and many of them: 8 x 4096 x 4096 bf16 with
// 8-bit output took 76 us (4.6 TB/s) here, the ramp of each CTA's loads exposed; it
// stays for rows too few for the ring to turn, too long for it or not of whole vectors.
template <int DT, int V, int QUANT, bool ODD>
__global__ void __launch_bounds__(kNormMaxThreads, V == 1 ? 2 : 1) add_rmsnorm_kernel(const __grid_constant__ NormArgs a) {
    constexpr int VE = RowBits<DT>::VE;
    extern __shared__ unsigned group_max[];  // QUANT 2: [rows of the CTA][n_groups], bits of floats >= 0
    __shared__ float red[kNormMaxThreads / 32];
    pdl_wait();
    pdl_launch_dependents();
    const int n = a.warps * 32, in_cta = threadIdx.x / n, tid = threadIdx.x % n;
    const long long t = (long long)blockIdx.x * (blockDim.x / n) + in_cta;
    const bool live = t < a.rows;
    RowView<DT, ODD> view{0, live ? (int)a.dim : 0};
    if (ODD && live) {
        view.lo = (int)((uintptr_t)row_of<DT>((const void *)rank_ptr(a.parts, a.p, 0), t, a.part_stride) % 16) / ElemInfo<DT>::bytes;
        view.hi += view.lo;
    }
    if (QUANT == 2)
        for (int i = threadIdx.x; i < (int)(blockDim.x / n * a.n_groups); i += blockDim.x) group_max[i] = 0u;
    const Chunks chunks(a.rows * a.dim, a.p);
    const long long i0 = t * a.dim;
    int chunk = live ? chunks.of(i0) : 0;
    if (i0 + a.dim > chunk_start(chunk + 1, chunks.base, chunks.extra)) chunk = -1;  // the row lies over a boundary

    float s[V][VE] = {};
    RowBits<DT> w[V];
    float ss = 0.0f;
#pragma unroll
    for (int v = 0; v < V; v++) {
        const int vec = tid + v * n;
        const bool has = view.has(vec);
        RowBits<DT> res;
        if (a.residual) view.load(row_of<DT>(a.residual, t, a.residual_stride), vec, res);
        fold_vector<DT, kNormRanks>(a, chunks, has ? chunk : 0, i0 + view.column(vec, 0), i0, i0 + a.dim, s[v],
                                    [&](int r, RowBits<DT> &b) { view.load(row_of<DT>((const void *)rank_ptr(a.parts, a.p, r), t, a.part_stride), vec, b); });
        if (a.weight) view.load_columns(a.weight, vec, w[v]);
        if (a.residual) add_vec<DT>(s[v], res);
#pragma unroll
        for (int e = 0; e < VE; e++)
            if (view.has(vec, e)) ss = fmaf(s[v][e], s[v][e], ss);
    }
    ss = row_sum(ss, red, a.warps);
    if (QUANT == 2) __syncthreads();  // group_max is clear
    norm_outputs<DT, V, QUANT, ODD>(a, t, view, tid, n, rstd_of(a, ss), s, w, group_max + in_cta * a.n_groups, [] { __syncthreads(); });
}

// The same for many rows: persistent CTAs, to which a warp of its own brings the rows
// blockIdx, blockIdx + gridDim, ... of all ranks and the residual by bulk copies, `stages`
// rows ahead, a lane a matrix.  Two groups of `warps` warps take the rows in turn: one
// row's reduction is a chain of waits, and a second row in the works fills them
// (the ring alone holds too few rows for two CTAs an SM when p is 8).  Up to 256 threads a row:
// what a thread does once a row is then shared by two vectors or more.
// 8 x 4096 x 4096 bf16 with 8-bit output: 59 us, 5.9 TB/s of the 6.7 that a copy reaches
// (68 us with one row in the works).
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
            row_chunk[s] = 0;  // (read also after a wait that ran out)
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
            for (int r = tid; r < matrices; r += 32) {
                if (r == a.limits.mute) continue;
                bulk_load(ring + (size_t)st * stage_bytes + (size_t)r * row_bytes,
                          r < a.p ? row_of<DT>((const void *)rank_ptr(a.parts, a.p, r), t, a.part_stride) : row_of<DT>(a.residual, t, a.residual_stride),
                          row_bytes, &full[st]);
            }
        }
        // the CTA stays until its copies have landed
        for (unsigned q = k > (unsigned)a.stages ? k - (unsigned)a.stages : 0; q < k; q++)
            if (!mbar_drain(&full[q % (unsigned)a.stages], (q / (unsigned)a.stages) & 1)) break;
        return;
    }
    const int vecs = (int)(a.dim / VE), bar = 1 + group;
    unsigned *gmax = reinterpret_cast<unsigned *>(ring + (size_t)a.stages * stage_bytes) + 2 * group * (int)a.n_groups;
    RowBits<DT> w[V];
#pragma unroll
    for (int v = 0; v < V; v++)
        if (a.weight) w[v].load(a.weight, tid + v * n, tid + v * n < vecs);
    int parity = 0;
    unsigned st = (unsigned)group, turn = 0;  // (stages is even: a stage is one group's)
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
                fold_vector<DT, 1>(a, chunks, has ? -1 : 0, t * a.dim + (long long)vec * VE, t * a.dim, (t + 1) * a.dim, s[v], get);
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
        if (tid % 32 == 0) free_stage(&failed, &empty[st]);
        // the row's sum over the warps (two buffers: one barrier a row)
        ss = warp_sum(ss);
        if (tid % 32 == 0) red[group][parity][tid / 32] = ss;
        row_threads_sync(bar, n);
        ss = warp_sum(tid % 32 < a.warps ? red[group][parity][tid % 32] : 0.0f);
        if (QUANT == 2)  // the last row's maxima have been used
            for (int g = tid; g < (int)a.n_groups; g += n) gmax[(parity ^ 1) * (int)a.n_groups + g] = 0u;
        norm_outputs<DT, V, QUANT, false>(a, t, RowView<DT, false>{0, (int)a.dim}, tid, n, rstd_of(a, ss), s, w, gmax + parity * (int)a.n_groups,
                                          [&] { row_threads_sync(bar, n); });
        st += 2;
        if (st >= (unsigned)a.stages) st = (unsigned)group, turn++;
    }
}

// Any other row (matrices whose rows begin at different places in a vector, rows too
// long for the registers):
// s in shared memory in 32 bits, single elements, a CTA a row: 8 x 4096 x 4096 bf16 takes
// 391 us.
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

namespace {

int add_rmsnorm(rar_ctx *h, const rar_rmsnorm_args *a, cudaStream_t stream) {
    OpCheck c(h, "rar_add_rmsnorm");
    if (!a) return c.bad("args is NULL");
    int rc = c.dtype(a->dtype, true);
    if (rc != RAR_OK) return rc;
    if (a->p < 1 || a->p > RAR_MAX_P) return c.bad("p must be in [1, RAR_MAX_P]");
    if (a->dim < 1 || a->dim > RAR_NORM_MAX_DIM) return c.bad("dim must be in [1, RAR_NORM_MAX_DIM]");
    if (!(a->eps >= 0.0f)) return c.bad("eps must be at least 0");
    if (a->group % 32) return c.bad("group must be a multiple of 32");
    if (a->rows > 0x7FFFFFFFu) return c.bad("rows must be at most 2^31 - 1");  // (a CTA a row)
    if (a->rows == 0) return RAR_OK;
    if (!a->parts) return c.bad("parts is NULL");
    if (a->out8 && !a->scales) return c.bad("scales is NULL");
    const size_t e = (size_t)elem_bytes(a->dtype);
    // (one longer than any row is the row's; the kernels count columns in 32 bits)
    const size_t group = a->group ? std::min<size_t>(a->group, RAR_NORM_MAX_DIM) : a->dim, n_groups = (a->dim + group - 1) / group;
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
    // whether the rows of every matrix are whole 16-byte vectors, or at least begin
    // at the same place in one
    bool vec = a->dim % ve == 0, alike = true;
    auto look = [&](const void *ptr, long long st) {
        if (!ptr) return;
        vec = vec && vec16(ptr, a->rows, st, e);
        alike = alike && ((uintptr_t)ptr - (uintptr_t)a->parts[0]) % 16 == 0 && (a->rows <= 1 || (size_t)(st - k.part_stride) * e % 16 == 0);
    };
    for (int r = 0; r < a->p; r++) look(a->parts[r], k.part_stride);
    look(k.residual, k.residual_stride);
    look(k.sum, k.sum_stride);
    look(k.out, k.out_stride);
    vec = vec && (uintptr_t)k.weight % 16 == 0 &&
          (!k.out8 || ((uintptr_t)k.out8 % ve == 0 && (a->rows <= 1 || (size_t)k.out8_stride % ve == 0)));
    const RowShape shape = row_shape(vec ? a->dim / ve : (a->dim + ve - 1) / ve + 1);
    cudaError_t ce;
    if ((vec || alike) && shape.v) {
        const size_t gv = group / ve;
        // a group's maximum by shuffles: its vectors are aligned lanes of one warp
        const bool lanes = vec && group % ve == 0 && gv <= 32 && (gv & (gv - 1)) == 0;
        const int quant = !k.out8 ? 0 : lanes ? 1 : 2;
        k.group_shift = 0;
        while (lanes && ((size_t)1 << k.group_shift) < gv) k.group_shift++;
        k.warps = shape.warps;
        const size_t stage_bytes = (size_t)(a->p + (k.residual ? 1 : 0)) * a->dim * e;
        const RowShape ring_row = row_shape(a->dim / ve, kRingRowThreads);
        const int ring_threads = 2 * ring_row.warps * 32 + 32;
        const RingShape ring = vec ? ring_shape(h, a->rows, ring_row, ring_threads, 682, 2, stage_bytes) : RingShape{0, 0};
        if (ring.ctas) k.warps = ring_row.warps;
        k.stages = ring.stages;
        k.limits = {h->status, op_timeout_ns(h), op_muted_rank(h)};
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
                if (!vec)
                    return launch_pdl(quant == 0 ? add_rmsnorm_kernel<DT, V, 0, true> : add_rmsnorm_kernel<DT, V, 2, true>, grid, block, smem, stream, k);
                return launch_pdl(quant == 0   ? add_rmsnorm_kernel<DT, V, 0, false>
                                  : quant == 1 ? add_rmsnorm_kernel<DT, V, 1, false>
                                               : add_rmsnorm_kernel<DT, V, 2, false>,
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

}  // namespace
}  // namespace rar

extern "C" {

int rar_add_rmsnorm(rar_handle h, const rar_rmsnorm_args *a, void *stream) {
    return rar::guarded(h, [&] {
        if (!h) return rar::fail(nullptr, RAR_EINVAL, "handle is NULL");
        return rar::add_rmsnorm(h, a, (cudaStream_t)stream);
    });
}

}  // extern "C"

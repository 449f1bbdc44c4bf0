// grad_norm.cu -- the norm of many tensors together and of each (rar_grad_norm), and
// tensors scaled down to a largest norm (rar_grad_clip).
//
//   norms[i] = sqrt(sum x^2 over tensor i),  norm = sqrt(sum of all)
//   out = x min(1, max_norm / (norm + eps))
//
// The tensors are cut into chunks of equally many elements, a CTA a chunk; the chunks'
// sums go to the workspace and are added in a fixed order (no atomics).  Bound by
// memory: one read of everything, and a read and a write.  The norm of 1.07 G bf16 elements takes 296 us
// (7.2 TB/s, a read alone runs above a copy's rate), of 157 M float32 in 440 tensors 95 us; clipping the 1.07 G into 32 bits
// 1.01 ms more for 6.4 GB, two thirds of them written (a write alone runs at 4.1 TB/s), in place 0.62 (7.0 TB/s).
#include <algorithm>

#include "op_elem.cuh"
#include "op_host.h"

namespace rar {

// A tensor as the kernels see it: `rows` of `cols` elements, one row where it is dense.
struct GradEntry {
    const void *data;
    void *out;
    long long n, cols, stride, out_stride;
    short dtype, out_dtype;
};
// The tensors of a launch travel in the kernel's parameters.
template <int N>
struct GradTable {
    GradEntry entry[N];
    unsigned start[N + 1];  // a tensor's first chunk (apart from the rest: it is what is searched); its end
    int n;
    unsigned first, chunks;  // of this launch
    long long chunk;         // elements of a chunk
    double *sums;            // [chunks of all launches]
    double *total;
    float *norm, *norms;
    bool begins, ends;       // the first launch, the last
    // clipping
    const float *clip_norm;
    float max_norm, eps;
};
constexpr int kFewTensors = 64, kManyTensors = 512;
constexpr int kGradThreads = 256;

// The tensor that a chunk belongs to (tensors without elements have none).
template <int N>
__device__ __forceinline__ int tensor_of(const GradTable<N> &a, unsigned chunk) {
    int lo = 0, hi = a.n - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) / 2;
        if (a.start[mid] <= chunk) lo = mid;
        else hi = mid - 1;
    }
    return lo;
}

template <int DT>
__device__ __forceinline__ float element(const GradEntry &t, long long i) {
    if (t.cols == t.n) return load_f<DT>(t.data, i);
    const long long r = i / t.cols;
    return load_f<DT>(t.data, r * t.stride + (i - r * t.cols));
}

// Calls f for the 16-byte vectors of elements [e0, e1) that lie one after the other from `base` (element
// 0) on, kAhead of them read together and `after` called after these, and g for the elements at the ends that
// fill none; as thread `tid` of n, at least a vector's elements.
template <int DT, int kAhead, typename F, typename G, typename H>
__device__ __forceinline__ void walk(const char *base, long long e0, long long e1, int tid, int n, F &&f, G &&g, H &&after) {
    constexpr int VE = RowBits<DT>::VE, EB = ElemInfo<DT>::bytes;
    const uintptr_t at = (uintptr_t)(base + e0 * EB);
    const long long lead = min((long long)((0 - at) % 16 / EB), e1 - e0);
    const long long v0 = e0 + lead, vecs = (e1 - v0) / VE, tail = v0 + vecs * VE;
    if (tid < lead) g(e0 + tid);
    if (tid < e1 - tail) g(tail + tid);
    const char *from = base + v0 * EB;
    long long v = tid;
    for (; v + (kAhead - 1) * n < vecs; v += kAhead * n) {
        RowBits<DT> b[kAhead];
#pragma unroll
        for (int k = 0; k < kAhead; k++) b[k].load(from + (v + k * n) * 16, 0, true);
#pragma unroll
        for (int k = 0; k < kAhead; k++) f(v0 + (v + k * n) * VE, b[k]);
        after();
    }
    for (; v < vecs; v += n) {
        RowBits<DT> b;
        b.load(from + v * 16, 0, true);
        f(v0 + v * VE, b);
    }
}
// The same for elements [e0, e1) of a matrix with gaps, a warp a row: f(row, first and last element) of its parts.
// (Rows longer than an eighth of a chunk leave warps without one: the norm of 8192 x 8192 bf16 takes 86 us with gaps, 60
// without, clipping in place 61 and 47.)
template <typename F>
__device__ __forceinline__ void walk_rows(const GradEntry &t, long long e0, long long e1, F &&f) {
    for (long long r = e0 / t.cols + threadIdx.x / 32; r * t.cols < e1; r += kGradThreads / 32) f(r, max(e0, r * t.cols), min(e1, (r + 1) * t.cols));
}
// Rows of fewer elements go one by one, a thread each, with a division for its row.
constexpr int kShortRow = 64;

// Sum over the CTA, in every thread.
__device__ __forceinline__ float cta_sum(float v, float *red) {
    v = warp_sum(v);
    __syncthreads();
    if (threadIdx.x % 32 == 0) red[threadIdx.x / 32] = v;
    __syncthreads();
    v = 0.0f;
    for (int w = 0; w < kGradThreads / 32; w++) v += red[w];
    return v;
}
__device__ __forceinline__ float cta_max(float v, float *red) {
    for (int o = 16; o; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xFFFFFFFFu, v, o));
    __syncthreads();
    if (threadIdx.x % 32 == 0) red[threadIdx.x / 32] = v;
    __syncthreads();
    v = 0.0f;
    for (int w = 0; w < kGradThreads / 32; w++) v = fmaxf(v, red[w]);
    return v;
}

// A thread's sum of squares.  A long run of additions to one sum of squares loses more than their rounding's
// share (small squares, which come more often than large ones, are rounded away from a sum that has grown): those of
// 256 bf16 values come out 2.5e-7 low, of 2048 3.9e-6, of 16 1e-8.  So what a few loads bring is added up
// first, and these batches with their additions' remainders (Knuth's two-sum), however many there are.
struct Squares {
    float s[4] = {}, total = 0.0f, rest = 0.0f;
    __device__ __forceinline__ void add(int k, float x) { s[k] = fmaf(x, x, s[k]); }
    __device__ __forceinline__ void batch() {
        const float x = (s[0] + s[1]) + (s[2] + s[3]), t = total + x, y = t - total;
        rest += (total - (t - y)) + (x - y);
        total = t;
        s[0] = s[1] = s[2] = s[3] = 0.0f;
    }
    __device__ __forceinline__ float sum() const { return total + rest; }  // (NaN where it passes binary32)
};

template <int DT>
__device__ __forceinline__ double chunk_sum(const GradEntry &t, long long e0, long long e1) {
    __shared__ float red[kGradThreads / 32];
    Squares own;
    auto batch = [&] { own.batch(); };
    uint32_t bits = 0;  // of all elements
    auto one = [&](float x) {
        bits |= __float_as_uint(x) << 1;
        own.add(0, x);
    };
    auto eight = [&](long long, const RowBits<DT> &b) {
#pragma unroll
        for (int e = 0; e < RowBits<DT>::VE; e++) own.add(e % 4, b.get(e));
        // (not the signs)
        bits |= DT == DT_F32 ? (b.w[0] | b.w[1] | b.w[2] | b.w[3]) << 1 : (b.w[0] | b.w[1] | b.w[2] | b.w[3]) & 0x7FFF7FFFu;
    };
    const char *data = static_cast<const char *>(t.data);
    if (t.cols == t.n) {
        walk<DT, 8>(data, e0, e1, threadIdx.x, kGradThreads, eight, [&](long long i) { one(load_f<DT>(data, i)); }, batch);
    } else if (t.cols >= kShortRow) {
        walk_rows(t, e0, e1, [&](long long r, long long r0, long long r1) {
            const char *row = data + r * (t.stride - t.cols) * ElemInfo<DT>::bytes;
            walk<DT, 4>(row, r0, r1, threadIdx.x % 32, 32, eight, [&](long long i) { one(load_f<DT>(row, i)); }, batch);
            batch();
        });
    } else {
        for (long long i = e0 + threadIdx.x; i < e1; i += kGradThreads) {
            one(element<DT>(t, i));
            if ((i / kGradThreads) % 16 == 15) batch();
        }
    }
    batch();
    const float sum = cta_sum(own.sum(), red);
    const bool any = __syncthreads_or(bits != 0);
    // Squares that pass binary32 or vanish in it: the chunk once more, relative to its largest
    // element (in these bounds what was lost is below 2^-24 of the sum for a chunk of 2^30 elements)
    if (!any || (sum >= 0x1p-90f && sum <= 0x1p126f)) return (double)sum;
    float most = 0.0f;
    bool finite = true, nan = false;
    for (long long i = e0 + threadIdx.x; i < e1; i += kGradThreads) {
        const float x = fabsf(element<DT>(t, i));
        finite = finite && isfinite(x);
        nan = nan || isnan(x);
        most = fmaxf(most, x);
    }
    if (__syncthreads_or(!finite)) return (double)(__syncthreads_or(nan) ? NAN : INFINITY);
    most = cta_max(most, red);
    const int e = ilogbf(most);
    Squares v;
    for (long long i = e0 + threadIdx.x; i < e1; i += kGradThreads) {
        v.add(0, ldexpf(element<DT>(t, i), -e));
        if ((i / kGradThreads) % 16 == 15) v.batch();
    }
    v.batch();
    return ldexp((double)cta_sum(v.sum(), red), 2 * e);
}

template <int N>
__global__ void __launch_bounds__(kGradThreads) grad_norm_kernel(const __grid_constant__ GradTable<N> a) {
    pdl_wait();
    pdl_launch_dependents();
    const unsigned chunk = a.first + blockIdx.x;
    const int i = tensor_of(a, chunk);
    const GradEntry &t = a.entry[i];
    const long long e0 = (long long)(chunk - a.start[i]) * a.chunk, e1 = min(e0 + a.chunk, t.n);
    const double s = t.dtype == DT_F32 ? chunk_sum<DT_F32>(t, e0, e1) : t.dtype == DT_BF16 ? chunk_sum<DT_BF16>(t, e0, e1) : chunk_sum<DT_F16>(t, e0, e1);
    if (threadIdx.x == 0) a.sums[chunk] = s;
}

// The root of a sum of squares, rounded to binary32: that of its significand times an even power of two, in
// binary32 (half a unit in the last place for the rounding, half for the root).  A root in binary64
// takes some 30 operations at 2 a clock and SM, for 440 tensors most of the join's 13 us.
__device__ __forceinline__ float norm_of(double s) {
    if (!(s > 0.0) || isinf(s)) return (float)s;
    const int hi = __double2hiint(s), e = ((hi >> 20) - 1023) & ~1;
    return ldexpf(sqrtf((float)__hiloint2double(hi - e * (1 << 20), __double2loint(s))), e / 2);
}

// Sum over groups of n lanes, in each of them.
__device__ __forceinline__ double lanes_sum(double v, int n) {
    for (int o = n / 2; o; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    return v;
}

// The chunks' sums by tensor, and the tensors': one CTA, a group of lanes a tensor, so that the latency of
// a tensor's few loads is not paid for one after the other.
template <int N>
__global__ void __launch_bounds__(1024) grad_norm_join_kernel(const __grid_constant__ GradTable<N> a) {
    __shared__ double tensor[N];
    __shared__ unsigned start[N + 1];
    for (int i = threadIdx.x; i <= a.n; i += 1024) start[i] = a.start[i];
    __syncthreads();
    pdl_wait();
    pdl_launch_dependents();
    int lanes = 32;
    while (lanes > 4 && a.n * lanes > 1024) lanes /= 2;
    const int sub = threadIdx.x % lanes;
    for (int i0 = 0; i0 < a.n; i0 += 1024 / lanes) {
        const int i = i0 + threadIdx.x / lanes;
        double s = 0.0;
        if (i < a.n) {
            const unsigned hi = start[i + 1];
#pragma unroll 8
            for (unsigned c = start[i] + sub; c < hi; c += lanes) s += __ldcg(a.sums + c);
        }
        s = lanes_sum(s, lanes);
        if (i < a.n && sub == 0) {
            tensor[i] = s;
            if (a.norms) a.norms[i] = norm_of(s);
        }
    }
    __syncthreads();
    if (threadIdx.x >= 32) return;
    double s = 0.0;
    for (int i = threadIdx.x; i < a.n; i += 32) s += tensor[i];
    s = lanes_sum(s, 32);
    if (threadIdx.x) return;
    if (!a.begins) s += *a.total;
    if (!a.ends) *a.total = s;
    else if (a.norm) *a.norm = norm_of(s);
}

template <int DT, int OUT>
__device__ __forceinline__ void scale_chunk(const GradEntry &t, long long e0, long long e1, float f) {
    constexpr int VE = RowBits<DT>::VE, EB = ElemInfo<DT>::bytes, OB = ElemInfo<OUT>::bytes;
    const char *data = static_cast<const char *>(t.data);
    char *out = static_cast<char *>(t.out);
    // elements [i0, i1) of runs that begin (element 0) at `from` and `to`
    auto run = [&](const char *from, char *to, long long i0, long long i1, int tid, int n) {
        const long long lead = (0 - (uintptr_t)(from + i0 * EB)) % 16 / EB;
        if ((uintptr_t)(to + (i0 + lead) * OB) % 16) {  // vectors that are read go to no whole ones (268 M bf16 into 32 bits 988 us, else 404)
            for (long long i = i0 + tid; i < i1; i += n) store_f<OUT>(to, i, load_f<DT>(from, i) * f);
            return;
        }
        walk<DT, 4>(from, i0, i1, tid, n, [&](long long i, const RowBits<DT> &b) {
            float v[VE];
#pragma unroll
            for (int e = 0; e < VE; e++) v[e] = b.get(e) * f;
#pragma unroll
            for (int q = 0; q < VE * OB / 16; q++) store_vec<OUT>(to + i * OB, q, v + q * (16 / OB));
        }, [&](long long i) { store_f<OUT>(to, i, load_f<DT>(from, i) * f); }, [] {});
    };
    if (t.cols == t.n) {
        run(data, out, e0, e1, threadIdx.x, kGradThreads);
    } else if (t.cols >= kShortRow) {
        walk_rows(t, e0, e1, [&](long long r, long long r0, long long r1) {
            run(data + r * (t.stride - t.cols) * EB, out + r * (t.out_stride - t.cols) * OB, r0, r1, threadIdx.x % 32, 32);
        });
    } else {
        for (long long i = e0 + threadIdx.x; i < e1; i += kGradThreads) {
            const long long r = i / t.cols;
            store_f<OUT>(out, r * t.out_stride + (i - r * t.cols), element<DT>(t, i) * f);
        }
    }
}

// From the last chunk to the first: what the norm read last is still in L2.
template <int N>
__global__ void __launch_bounds__(kGradThreads) grad_clip_kernel(const __grid_constant__ GradTable<N> a) {
    pdl_wait();
    pdl_launch_dependents();
    const float d = *a.clip_norm + a.eps;
    const float f = d <= a.max_norm ? 1.0f : __fdiv_rn(a.max_norm, d);  // (a NaN is passed on)
    const unsigned chunk = a.first + a.chunks - 1 - blockIdx.x;
    const int i = tensor_of(a, chunk);
    const GradEntry &t = a.entry[i];
    if (f == 1.0f && t.out == t.data) return;
    const long long e0 = (long long)(chunk - a.start[i]) * a.chunk, e1 = min(e0 + a.chunk, t.n);
    if (t.dtype == DT_F32) scale_chunk<DT_F32, DT_F32>(t, e0, e1, f);
    else if (t.dtype == DT_BF16) t.out_dtype == DT_F32 ? scale_chunk<DT_BF16, DT_F32>(t, e0, e1, f) : scale_chunk<DT_BF16, DT_BF16>(t, e0, e1, f);
    else t.out_dtype == DT_F32 ? scale_chunk<DT_F16, DT_F32>(t, e0, e1, f) : scale_chunk<DT_F16, DT_F16>(t, e0, e1, f);
}

namespace {

size_t elements(const rar_tensor &t) { return t.rows * t.cols; }

// Elements of a chunk: a power of two, 8192 or more (at 4096, 10 M fp16 elements took 24 us to clip, 17 at
// 8192), so that there are at most `most` chunks, and one more a tensor.  For the norm 4096, whose sums one CTA
// joins: 1.07 G elements bf16 take 296 us with 512 to 4096 of them, 310 with up to 16384, 334 with 65536;
// 157 M float32 99 us with up to 4096, 102 and 191.  Clipping has nothing to join: the 1.07 G into 32 bits take
// 1683 us with up to 512, 1447 with 2048, 1356 with 16384, 1300 with 65536, with the norm before it.
constexpr size_t kLeastChunk = 8192, kNormChunks = 4096, kClipChunks = 65536;
size_t chunk_elements(const rar_tensor *tensors, size_t n, size_t most) {
    size_t total = 0, chunk = kLeastChunk;
    for (size_t i = 0; i < n; i++) total += elements(tensors[i]);
    while (total / chunk > most) chunk *= 2;
    return chunk;
}
size_t count_chunks(const rar_tensor *tensors, size_t n, size_t chunk) {
    size_t chunks = 0;
    for (size_t i = 0; i < n; i++) chunks += (elements(tensors[i]) + chunk - 1) / chunk;
    return chunks;
}
size_t plan(void *base, const rar_tensor *tensors, size_t n, double **sums, double **total) {
    WorkspacePlan w(base);
    *total = w.take<double>(1);
    *sums = w.take<double>(count_chunks(tensors, n, chunk_elements(tensors, n, kNormChunks)));
    return w.used;
}

// Sizes alone, without a handle.
const char *sizes_wrong(const rar_tensor *tensors, size_t n) {
    constexpr size_t kMost = (size_t)1 << 40;
    size_t total = 0;
    if (!tensors && n) return "tensors is NULL";
    if (n > (size_t)1 << 24) return "there are too many tensors";
    for (size_t i = 0; i < n; i++) {
        const rar_tensor &t = tensors[i];
        if (t.cols > kMost || (t.cols && t.rows > kMost / t.cols)) return "a tensor is too large";
        if ((total += elements(t)) > kMost) return "the tensors are too large";
    }
    return nullptr;
}

// Checks one list; spans of its tensors are added to `spans`.
int check_list(OpCheck &c, const char *what, const rar_tensor *tensors, size_t n, std::vector<MatrixSpan> *spans) {
    if (const char *wrong = sizes_wrong(tensors, n)) return c.bad(wrong);
    for (size_t i = 0; i < n; i++) {
        const rar_tensor &t = tensors[i];
        int rc = c.dtype(t.dtype, true);
        if (rc != RAR_OK) return rc;
        const size_t e = (size_t)elem_bytes(t.dtype);
        MatrixSpan s;
        if ((rc = c.matrix(what, t.data, t.rows, t.cols, t.stride, e, e, &s)) != RAR_OK) return rc;
        if (t.rows && t.cols) spans->push_back(s);
    }
    return RAR_OK;
}

bool dense(const rar_tensor &t) { return t.rows <= 1 || t.stride == 0 || t.stride == t.cols; }

// Calls f(table, its first tensor) with tables of up to N tensors, in order.
template <int N, typename F>
cudaError_t for_tables(const rar_tensor *tensors, const rar_tensor *out, size_t n, size_t chunk, F &&f) {
    cudaError_t e = cudaSuccess;
    unsigned chunks = 0;
    GradTable<N> a;
    for (size_t i0 = 0; (i0 < n || i0 == 0) && e == cudaSuccess; i0 += N) {
        a.n = (int)std::min<size_t>(n - i0, N);
        a.first = chunks;
        for (int i = 0; i < a.n; i++) {
            const rar_tensor &t = tensors[i0 + i], &o = out ? out[i0 + i] : t;
            GradEntry &g = a.entry[i];
            // a matrix without gaps is one row, and where its copy has some, it is not
            const bool one = dense(t) && dense(o);
            g.data = t.data;
            g.out = o.data;
            g.n = (long long)elements(t);
            g.cols = one ? g.n : (long long)t.cols;
            g.stride = one ? g.n : (long long)(t.stride ? t.stride : t.cols);
            g.out_stride = one ? g.n : (long long)(o.stride ? o.stride : o.cols);
            a.start[i] = chunks;
            g.dtype = (short)t.dtype;
            g.out_dtype = (short)o.dtype;
            chunks += (unsigned)((elements(t) + chunk - 1) / chunk);
        }
        a.start[a.n] = chunks;
        a.chunks = chunks - a.first;
        a.chunk = (long long)chunk;
        a.begins = i0 == 0;
        a.ends = i0 + N >= n;
        e = f(a, i0);
    }
    return e;
}

int grad_norm(rar_ctx *h, const rar_grad_norm_args *a, cudaStream_t stream) {
    OpCheck c(h, "rar_grad_norm");
    if (!a) return c.bad("args is NULL");
    std::vector<MatrixSpan> spans;
    int rc = check_list(c, "a tensor", a->tensors, a->n, &spans);
    if (rc != RAR_OK) return rc;
    if (!a->norm && !a->norms) return c.bad("norm and norms are NULL");
    MatrixSpan s;
    for (const MatrixSpan &in : spans) c.input(in);
    if (a->norm) {
        if ((rc = c.matrix("norm", a->norm, 1, 1, 0, 4, 4, &s)) != RAR_OK) return rc;
        c.output(s);
    }
    if (a->norms) {
        if ((rc = c.matrix("norms", a->norms, 1, a->n, 0, 4, 4, &s)) != RAR_OK) return rc;
        c.output(s);
    }
    double *sums, *total;
    if ((rc = c.workspace(a->workspace, a->workspace_bytes, plan(nullptr, a->tensors, a->n, &sums, &total))) != RAR_OK) return rc;
    if ((rc = c.overlaps([](const MatrixSpan &, const MatrixSpan &) { return false; })) != RAR_OK) return rc;

    DeviceGuard dg(h->device);
    if (dg.err != cudaSuccess) return cuda_fail(h, dg.err, "selecting the device");
    plan(a->workspace, a->tensors, a->n, &sums, &total);
    note_op_call(h, 1, stream);
    auto run = [&](auto most) {
        constexpr int N = decltype(most)::value;
        return for_tables<N>(a->tensors, nullptr, a->n, chunk_elements(a->tensors, a->n, kNormChunks), [&](GradTable<N> &t, size_t i0) {
            t.sums = sums;
            t.total = total;
            t.norm = a->norm;
            t.norms = a->norms ? a->norms + i0 : nullptr;
            cudaError_t e = cudaSuccess;
            if (t.chunks) e = launch_pdl(grad_norm_kernel<N>, dim3(t.chunks), dim3(kGradThreads), 0, stream, t);
            if (e == cudaSuccess) e = launch_pdl(grad_norm_join_kernel<N>, dim3(1), dim3(1024), 0, stream, t);
            return e;
        });
    };
    const cudaError_t ce = a->n <= kFewTensors ? run(IntC<kFewTensors>{}) : run(IntC<kManyTensors>{});
    return ce == cudaSuccess ? RAR_OK : cuda_fail(h, ce, "launching the norm");
}

int grad_clip(rar_ctx *h, const rar_grad_clip_args *a, cudaStream_t stream) {
    OpCheck c(h, "rar_grad_clip");
    if (!a) return c.bad("args is NULL");
    if (!(a->max_norm >= 0.0f && a->max_norm <= 3.402823466e38f)) return c.bad("max_norm must be finite and not negative");
    if (!(a->eps >= 0.0f && a->eps <= 3.402823466e38f)) return c.bad("eps must be finite and not negative");
    std::vector<MatrixSpan> spans, outs;
    int rc = check_list(c, "a tensor", a->tensors, a->n, &spans);
    if (rc != RAR_OK) return rc;
    if (a->out) {
        if ((rc = check_list(c, "an output", a->out, a->n, &outs)) != RAR_OK) return rc;
        for (size_t i = 0; i < a->n; i++) {
            const rar_tensor &t = a->tensors[i], &o = a->out[i];
            if (o.rows != t.rows || o.cols != t.cols) return c.bad("an output differs from its tensor in its sizes");
            if (o.dtype != t.dtype && o.dtype != RAR_FLOAT32) return c.bad("an output has neither its tensor's dtype nor float32");
        }
    }
    MatrixSpan s;
    if ((rc = c.matrix("norm", a->norm, 1, 1, 0, 4, 4, &s)) != RAR_OK) return rc;
    if ((rc = c.list_overlaps(spans, a->out ? &outs : nullptr, s)) != RAR_OK) return rc;

    DeviceGuard dg(h->device);
    if (dg.err != cudaSuccess) return cuda_fail(h, dg.err, "selecting the device");
    note_op_call(h, 1, stream);
    auto run = [&](auto most) {
        constexpr int N = decltype(most)::value;
        return for_tables<N>(a->tensors, a->out, a->n, chunk_elements(a->tensors, a->n, kClipChunks), [&](GradTable<N> &t, size_t) {
            t.clip_norm = a->norm;
            t.max_norm = a->max_norm;
            t.eps = a->eps;
            return t.chunks ? launch_pdl(grad_clip_kernel<N>, dim3(t.chunks), dim3(kGradThreads), 0, stream, t) : cudaSuccess;
        });
    };
    const cudaError_t ce = a->n <= kFewTensors ? run(IntC<kFewTensors>{}) : run(IntC<kManyTensors>{});
    return ce == cudaSuccess ? RAR_OK : cuda_fail(h, ce, "launching the clipping");
}

}  // namespace
}  // namespace rar

extern "C" {

size_t rar_grad_norm_workspace(const rar_tensor *tensors, size_t n) {
    if (rar::sizes_wrong(tensors, n)) return 0;
    double *sums, *total;
    return rar::plan(nullptr, tensors, n, &sums, &total);
}

int rar_grad_norm(rar_handle h, const rar_grad_norm_args *a, void *stream) {
    return rar::guarded(h, [&] {
        if (!h) return rar::fail(nullptr, RAR_EINVAL, "handle is NULL");
        return rar::grad_norm(h, a, (cudaStream_t)stream);
    });
}

int rar_grad_clip(rar_handle h, const rar_grad_clip_args *a, void *stream) {
    return rar::guarded(h, [&] {
        if (!h) return rar::fail(nullptr, RAR_EINVAL, "handle is NULL");
        return rar::grad_clip(h, a, (cudaStream_t)stream);
    });
}

}  // extern "C"

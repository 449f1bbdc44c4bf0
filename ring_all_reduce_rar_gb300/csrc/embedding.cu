// embedding.cu -- scaled lookup in a table held in p pieces, and the table's
// gradient (rar_embedding, rar_embedding_grad).
//
//   out[t] = scale table[tokens[t]]
//   dtables[v] = scale sum over the t with tokens[t] = v of dout[t]
//                (+ what dtables[v] held, with accumulate), in a fixed order
//
// Bound by memory: a read and a write an element.
#include <algorithm>
#include <utility>

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

// Row v of a table in pieces.
__device__ __forceinline__ char *table_row(const EmbedArgs &a, const Chunks &c, long long v, int elem_size) {
    const int r = c.of(v);
    return rank_ptr(a.pieces, a.p, r) + (v - chunk_start(r, c.base, c.extra)) * a.table_stride * elem_size;
}

// The lookup: the out matrix as one run of 16-byte vectors (VEC) or single elements,
// U of them a thread with their loads in flight together.  8192 rows of 4096 bf16: 27 us,
// 5.0 TB/s of rows read (half of them, repeated, from L2) and written; 63 us with one element
// a thread.
template <int DT, bool VEC, int U>
__global__ void __launch_bounds__(256) embedding_kernel(const __grid_constant__ EmbedArgs a) {
    constexpr int VE = VEC ? RowBits<DT>::VE : 1, EB = ElemInfo<DT>::bytes;
    pdl_wait();
    pdl_launch_dependents();
    const Chunks chunks(a.vocab, a.p);
    const long long per_row = a.dim / VE, total = a.n_tokens * per_row;
    const long long i0 = (long long)blockIdx.x * (256 * U) + threadIdx.x;
    const char *from[U];
    long long t[U];
    int j[U];
    bool has[U];
#pragma unroll
    for (int u = 0; u < U; u++) {
        const long long i = i0 + u * 256;
        has[u] = i < total;
        t[u] = total < 0x7FFFFFFF ? (long long)((uint32_t)i / (uint32_t)per_row) : i / per_row;
        j[u] = (int)(i - t[u] * per_row);
        const long long v = has[u] ? load_index(a.tokens, a.index_bytes, t[u]) : -1;
        from[u] = v >= 0 && v < a.vocab ? table_row(a, chunks, v, EB) : nullptr;
    }
    if constexpr (VEC) {
        RowBits<DT> w[U];
#pragma unroll
        for (int u = 0; u < U; u++) w[u].load(from[u], j[u], from[u] != nullptr);
#pragma unroll
        for (int u = 0; u < U; u++) {
            float f[VE];
#pragma unroll
            for (int e = 0; e < VE; e++) f[e] = w[u].get(e) * a.scale;
            if (!from[u])  // (0 x an infinite scale)
#pragma unroll
                for (int e = 0; e < VE; e++) f[e] = 0.0f;
            if (has[u]) store_vec<DT>(static_cast<char *>(a.out) + t[u] * a.row_stride * EB, j[u], f);
        }
    } else {
        uint32_t w[U];
#pragma unroll
        for (int u = 0; u < U; u++) w[u] = from[u] ? load_elem<DT>(from[u], j[u]) : 0u;
#pragma unroll
        for (int u = 0; u < U; u++)
            if (has[u]) store_f<DT>(a.out, t[u] * a.row_stride + j[u], from[u] ? widen<DT>(w[u]) * a.scale : 0.0f);
    }
}

// ---- gradient
//
// 1. The tokens are sorted by index, equal ones in the order of their places
//    (radix sort by one cluster), while the table is cleared.
// 2. The sorted places are cut into chunks.  A CTA adds up the runs of its chunk in
//    order; a run inside the chunk is written to the table, one that goes
//    on beyond it into the workspace.
// 3. Runs over several chunks are joined: groups of threads add every groups-th
//    chunk, and then the groups' sums in order.
// So a frequent token costs no more than others, and no sum depends on timing.

struct SortArgs {
    EmbedArgs e;
    uint2 *items[2];    // (index, place), from one pass to the next
    int bits, passes;   // of an index; of the sort
    int chunk, n_chunks;
    float *part;        // [n_chunks][2][dim]: sums of runs that began before the chunk, that go on after it
};

constexpr int kSortThreads = 1024, kSortWarps = kSortThreads / 32;
constexpr int kSortMaxBits = 9;       // of a pass
constexpr int kSortCluster = 8;       // CTAs that sort, for more than kSortOneCta tokens
constexpr int kSortHeld = 8;          // items a thread in flight
constexpr int kSortOneCta = 2 * kSortThreads;
constexpr int kSortPitch = kSortWarps + 1;  // counts of a digit, one a warp (odd: no bank conflicts)
constexpr int kSortSmem = (kSortPitch + 2) * (1 << kSortMaxBits) * (int)sizeof(unsigned);

__device__ __forceinline__ uint32_t dsmem_load(const void *p, int rank) {
    uint32_t addr = (uint32_t)__cvta_generic_to_shared(p), v;
    asm volatile("mapa.shared::cluster.u32 %0, %0, %1;" : "+r"(addr) : "r"(rank));
    asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
    return v;
}
__device__ __forceinline__ void sort_cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// Least significant digit first.  A warp owns a run of places, so that equal
// digits keep their order; it counts its digits, the counts of all warps and
// CTAs are summed up in (digit, CTA, warp) order, and the warp moves its
// items there.  One cluster, because every pass needs all counts: bound by latency, 18 us
// at 8192 tokens of 65536 rows (two passes) and 13 us at 4095 of 10007, beside the clearing where
// the table is written whole.
__device__ __forceinline__ void sort_tokens(const SortArgs &s, unsigned *smem, int cta, int ctas) {
    const EmbedArgs &a = s.e;
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const unsigned n = (unsigned)a.n_tokens, warps = (unsigned)(ctas * kSortWarps);
    const unsigned run = ((n + warps - 1) / warps + 31) / 32 * 32;
    const unsigned lo = min(n, run * (unsigned)(cta * kSortWarps + warp)), hi = min(n, lo + run);
    const int width = (s.bits + s.passes - 1) / s.passes;
    const unsigned bins = 1u << width;
    unsigned *count = smem;                       // [bins][kSortPitch]
    unsigned *total = smem + bins * kSortPitch;   // [bins] of this CTA
    unsigned *start = total + bins;               // [bins] of this CTA's items
    __shared__ unsigned warp_sums[kSortWarps];
    const bool held = run <= 32 * kSortHeld;      // the run's items stay in registers
    for (int pass = 0; pass < s.passes; pass++) {
        const uint2 *in = s.items[pass & 1];
        uint2 *out = s.items[(pass & 1) ^ 1];
        const int shift = pass * width;
        uint2 it[kSortHeld];
        // the items of kSortHeld rounds of 32 from place i0, loads in flight together
        auto load = [&](unsigned i0) {
#pragma unroll
            for (int k = 0; k < kSortHeld; k++) {
                const unsigned i = i0 + 32 * k + lane;
                it[k] = make_uint2(0, 0);
                if (i >= hi) continue;
                if (pass) {
                    it[k] = __ldcg(in + i);
                } else {
                    const long long v = load_index(a.tokens, a.index_bytes, i);
                    it[k] = make_uint2(v >= 0 && v < a.vocab ? (unsigned)v : (unsigned)a.vocab, i);
                }
            }
        };
        auto digit = [&](int k) { return it[k].x >> shift & (bins - 1); };
        // the lanes with the same digit in each round (a vote a bit: matching all
        // lanes' values in one instruction takes longer), 0 where the lane has no item
        unsigned peers[kSortHeld];
        auto match = [&](unsigned i0) {
#pragma unroll
            for (int k = 0; k < kSortHeld; k++) {
                peers[k] = 0u;
                if (i0 + 32 * k >= hi) continue;
                const unsigned d = digit(k);
                const bool has = i0 + 32 * k + lane < hi;
                unsigned same = __ballot_sync(0xFFFFFFFFu, has);
#pragma unroll
                for (int b = 0; b < kSortMaxBits; b++) {
                    const unsigned with = __ballot_sync(0xFFFFFFFFu, d >> b & 1);
                    same &= d >> b & 1 ? with : ~with;
                }
                peers[k] = has ? same : 0u;
            }
        };
        load(lo);
        for (unsigned i = threadIdx.x; i < bins * kSortPitch; i += kSortThreads) count[i] = 0u;
        __syncthreads();
        for (unsigned i0 = lo; i0 < hi; i0 += 32 * kSortHeld) {
            if (i0 != lo) load(i0);
            match(i0);
#pragma unroll
            for (int k = 0; k < kSortHeld; k++) {
                if (i0 + 32 * k >= hi) break;
                if (peers[k] && lane == __ffs(peers[k]) - 1) count[digit(k) * kSortPitch + warp] += __popc(peers[k]);
                __syncwarp();
            }
        }
        __syncthreads();
        // a digit's warps: a warp a digit, lane = warp; four digits side by side
        for (unsigned d0 = warp; d0 < bins; d0 += 4 * kSortWarps) {
            unsigned c[4], x[4];
#pragma unroll
            for (int k = 0; k < 4; k++) x[k] = c[k] = d0 + k * kSortWarps < bins ? count[(d0 + k * kSortWarps) * kSortPitch + lane] : 0u;
#pragma unroll
            for (int o = 1; o < 32; o *= 2)
#pragma unroll
                for (int k = 0; k < 4; k++) {
                    const unsigned y = __shfl_up_sync(0xFFFFFFFFu, x[k], o);
                    if (lane >= o) x[k] += y;
                }
#pragma unroll
            for (int k = 0; k < 4; k++) {
                if (d0 + k * kSortWarps >= bins) break;
                count[(d0 + k * kSortWarps) * kSortPitch + lane] = x[k] - c[k];
                if (lane == 31) total[d0 + k * kSortWarps] = x[k];
            }
        }
        __syncthreads();
        if (ctas > 1) sort_cluster_sync();
        // where the digit's items begin, and this CTA's among them
        unsigned all = 0, before = 0;
        if (threadIdx.x < bins) {
            if (ctas == 1) {
                all = total[threadIdx.x];
            } else {
                unsigned t[kSortCluster];  // (ctas is kSortCluster: loads in flight together)
#pragma unroll
                for (int c = 0; c < kSortCluster; c++) t[c] = dsmem_load(total + threadIdx.x, c);
#pragma unroll
                for (int c = 0; c < kSortCluster; c++) {
                    all += t[c];
                    if (c < cta) before += t[c];
                }
            }
        }
        unsigned x = all;
#pragma unroll
        for (int o = 1; o < 32; o *= 2) {
            const unsigned y = __shfl_up_sync(0xFFFFFFFFu, x, o);
            if (lane >= o) x += y;
        }
        if (lane == 31) warp_sums[warp] = x;
        __syncthreads();
        unsigned base = lane < warp ? warp_sums[lane] : 0u;
#pragma unroll
        for (int o = 16; o; o /= 2) base += __shfl_xor_sync(0xFFFFFFFFu, base, o);
        if (threadIdx.x < bins) start[threadIdx.x] = base + x - all + before;
        __syncthreads();
        for (unsigned i0 = lo; i0 < hi; i0 += 32 * kSortHeld) {
            if (!held) load(i0), match(i0);
#pragma unroll
            for (int k = 0; k < kSortHeld; k++) {
                if (i0 + 32 * k >= hi) break;
                const unsigned d = digit(k), ahead = __popc(peers[k] & ((1u << lane) - 1));
                const unsigned at = peers[k] ? count[d * kSortPitch + warp] : 0u;
                __syncwarp();
                if (peers[k]) {
                    out[start[d] + at + ahead] = it[k];
                    if (ahead == 0) count[d * kSortPitch + warp] = at + __popc(peers[k]);
                }
                __syncwarp();
            }
        }
        // the items, and every CTA's reads of the totals, before the next pass
        if (ctas > 1) {
            __threadfence();
            sort_cluster_sync();
        } else {
            __syncthreads();
        }
    }
}

// The sort, one cluster.  After a clearing launch (`beside`) it runs beside it: that
// launch lets it start once all work before it is done, and it ends only when the clearing
// has, so that what follows finds both done.
template <int DT>
__global__ void __launch_bounds__(kSortThreads) embedding_sort_kernel(const __grid_constant__ SortArgs s, bool beside) {
    extern __shared__ unsigned sort_smem[];
    if (!beside) pdl_wait();
    pdl_launch_dependents();
    sort_tokens(s, sort_smem, blockIdx.x, gridDim.x);
    if (beside) pdl_wait();
}

constexpr int kClearBytes = 16384;  // zeros in shared memory, the source of the bulk stores
// CTAs an SM: they leave room for the sort.  (Fewer warps to issue the stores clear more
// slowly beside other work: 65536 x 4096 bf16 with the gradient of 8192 tokens 110 us,
// with 4 x 128 threads 171, with 128 threads 333.)
constexpr int kClearThreads = 512, kClearCtas = 2;

// The warps clear the table: 16 KB of a piece at a time where its rows are
// packed, else a row.  65536 x 4096 bf16: 512 MB in 82 us, 6.5 TB/s; a write-only stream is bound by
// memory.  The 16-byte lines inside go by one bulk store, the elements before and
// after them one by one.
template <int DT>
__global__ void __launch_bounds__(kClearThreads) embedding_clear_kernel(const __grid_constant__ EmbedArgs a) {
    __shared__ __align__(128) unsigned zero_smem[kClearBytes / 4];
    constexpr int EB = ElemInfo<DT>::bytes;
    for (int i = threadIdx.x; i < kClearBytes / 16; i += kClearThreads) reinterpret_cast<uint4 *>(zero_smem)[i] = make_uint4(0, 0, 0, 0);
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    __syncthreads();
    pdl_wait();
    pdl_launch_dependents();
    const uint32_t zeros = (uint32_t)__cvta_generic_to_shared(zero_smem);
    const int lane = threadIdx.x % 32;
    const long long warps = (long long)gridDim.x * (kClearThreads / 32), me = (long long)blockIdx.x * (kClearThreads / 32) + threadIdx.x / 32;
    auto clear = [&](char *from, long long bytes) {
        for (long long at = 0; at < bytes; at += kClearBytes) {
            const uintptr_t p0 = (uintptr_t)from + at, p1 = p0 + (bytes - at < kClearBytes ? bytes - at : kClearBytes);
            const uintptr_t a0 = min((p0 + 15) & ~(uintptr_t)15, p1), a1 = max(p1 & ~(uintptr_t)15, a0);
            if (lane == 0 && a1 > a0)
                asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(a0), "r"(zeros), "r"((uint32_t)(a1 - a0)) : "memory");
            if (lane < (int)(a0 - p0) / EB) store_elem<DT>(reinterpret_cast<char *>(p0), lane, 0u);
            if (lane < (int)(p1 - a1) / EB) store_elem<DT>(reinterpret_cast<char *>(a1), lane, 0u);
        }
    };
    if (a.table_stride == a.dim) {
        const long long base = a.vocab / a.p, extra = a.vocab % a.p, row = a.dim * EB;
        const long long per_big = ((base + 1) * row + kClearBytes - 1) / kClearBytes, per_small = (base * row + kClearBytes - 1) / kClearBytes;
        const long long big = extra * per_big, units = big + (a.p - extra) * per_small;
        for (long long u = me; u < units; u += warps) {
            const long long r = u < big ? u / per_big : extra + (u - big) / per_small, k = u < big ? u % per_big : (u - big) % per_small;
            const long long left = (base + (r < extra ? 1 : 0)) * row - k * kClearBytes;
            clear(rank_ptr(a.pieces, a.p, (int)r) + k * kClearBytes, left < kClearBytes ? left : kClearBytes);
        }
    } else {
        const Chunks chunks(a.vocab, a.p);
        for (long long v = me; v < a.vocab; v += warps) clear(table_row(a, chunks, v, EB), a.dim * EB);
    }
    if (lane == 0) {
        asm volatile("cp.async.bulk.commit_group;" ::: "memory");
        asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
    }
}

constexpr int kReduceThreads = 256;
constexpr int kReduceAhead = 8;  // rows whose loads are in flight together
constexpr int kMinChunk = 16;

// Columns of a thread of `n` threads: a 16-byte vector, or 4 single elements n apart.
// Rows are held as they were read.
template <int DT, bool VEC>
struct GradCols {
    static constexpr int N = VEC ? RowBits<DT>::VE : 4;
    long long dim, first;
    int tid, n;
    struct Bits {
        RowBits<DT> v;
        __device__ __forceinline__ float get(int e) const { return VEC ? v.get(e) : widen<DT>(v.w[e]); }
    };
    __device__ __forceinline__ long long at(int e) const { return VEC ? first + (long long)tid * N + e : first + tid + (long long)e * n; }
    __device__ __forceinline__ bool has(int e) const { return at(VEC ? 0 : e) < dim; }
    __device__ __forceinline__ Bits load(const char *row, bool wanted) const {  // (coherent: a row of the table is written later)
        Bits b;
        if constexpr (VEC) {
            const uint4 q = wanted && has(0) ? *reinterpret_cast<const uint4 *>(row + at(0) * ElemInfo<DT>::bytes) : make_uint4(0, 0, 0, 0);
            b.v.w[0] = q.x, b.v.w[1] = q.y, b.v.w[2] = q.z, b.v.w[3] = q.w;
        } else {
#pragma unroll
            for (int e = 0; e < N; e++) b.v.w[e] = wanted && has(e) ? load_elem<DT>(row, at(e)) : 0u;
        }
        return b;
    }
    // a row of the workspace's sums
    __device__ __forceinline__ void load_part(const float *part, float (&f)[N]) const {
        if constexpr (VEC) {
#pragma unroll
            for (int e = 0; e < N; e += 4) {
                const float4 q = has(0) ? *reinterpret_cast<const float4 *>(part + at(e)) : make_float4(0, 0, 0, 0);
                f[e] = q.x, f[e + 1] = q.y, f[e + 2] = q.z, f[e + 3] = q.w;
            }
        } else {
#pragma unroll
            for (int e = 0; e < N; e++) f[e] = has(e) ? part[at(e)] : 0.0f;
        }
    }
    __device__ __forceinline__ void store_part(float *part, const float (&f)[N]) const {
        if constexpr (VEC) {
            if (has(0))
#pragma unroll
                for (int e = 0; e < N; e += 4) *reinterpret_cast<float4 *>(part + at(e)) = make_float4(f[e], f[e + 1], f[e + 2], f[e + 3]);
        } else {
#pragma unroll
            for (int e = 0; e < N; e++)
                if (has(e)) part[at(e)] = f[e];
        }
    }
    // a row of the table: the sum, scaled, added to what the row held, rounded once
    __device__ __forceinline__ void finish(char *row, const float (&sum)[N], float scale, bool add, const Bits &old) const {
        float f[N];
#pragma unroll
        for (int e = 0; e < N; e++) f[e] = add ? fmaf(sum[e], scale, old.get(e)) : sum[e] * scale;
        if constexpr (VEC) {
            if (has(0)) store_vec<DT>(row, (int)(at(0) / N), f);
        } else {
#pragma unroll
            for (int e = 0; e < N; e++)
                if (has(e)) store_f<DT>(row, at(e), f[e]);
        }
    }
};

// What is done with an item of a chunk: its row of dout is added, and, where
// its run leaves the chunk, the sum goes to `to`.
struct RunStep {
    const char *from;  // NULL: left out
    char *to;          // NULL: the run goes on
    bool table;        // `to` is the run's row of the table, else of the workspace
};

// ADD: accumulate.  The row that a run is added to is read together with the
// run's last row of dout.  Bound by memory for wide rows (8192 tokens added into
// 65536 x 4096 bf16: 47 us with the sort; 256 MB), by the sort's latency for others
// (4095 x 1001 float32 into 10007 rows: 24.5 us).
template <int DT, bool VEC, bool ADD>
__global__ void __launch_bounds__(kReduceThreads, 3) embedding_runs_kernel(const __grid_constant__ SortArgs s) {
    using Cols = GradCols<DT, VEC>;
    constexpr int N = Cols::N, EB = ElemInfo<DT>::bytes;
    __shared__ RunStep steps[kMinChunk];
    const EmbedArgs &a = s.e;
    pdl_wait();
    pdl_launch_dependents();
    const Chunks chunks(a.vocab, a.p);
    const uint2 *items = s.items[s.passes & 1];
    const Cols cols{a.dim, (long long)blockIdx.y * blockDim.x * N, (int)threadIdx.x, (int)blockDim.x};
    const int lo = blockIdx.x * s.chunk, hi = (int)min((long long)lo + s.chunk, a.n_tokens);
    float sum[N] = {};
    for (int i0 = lo; i0 < hi; i0 += kMinChunk) {
        if (threadIdx.x < kMinChunk) {
            const int i = i0 + threadIdx.x;
            const uint2 it = items[min(i, hi - 1)];
            const unsigned none = (unsigned)a.vocab;  // left out: sorted last
            const unsigned after = i + 1 < a.n_tokens ? items[i + 1].x : none + 1, before = lo ? items[lo - 1].x : none + 1;
            const bool ends = it.x != after, began = it.x != before;  // the run, in this chunk
            RunStep st{nullptr, nullptr, ends && began};
            if (i < hi && it.x != none) {
                st.from = static_cast<const char *>(a.dout) + it.y * a.row_stride * EB;
                if (ends || i + 1 == hi)
                    st.to = st.table ? table_row(a, chunks, it.x, EB) : reinterpret_cast<char *>(s.part + ((long long)blockIdx.x * 2 + (began ? 1 : 0)) * a.dim);
            }
            steps[threadIdx.x] = st;
        }
        __syncthreads();
#pragma unroll 1
        for (int k0 = 0; k0 < kMinChunk; k0 += kReduceAhead) {
            typename Cols::Bits f[kReduceAhead], old[ADD ? kReduceAhead : 1];
#pragma unroll
            for (int u = 0; u < kReduceAhead; u++) {
                const RunStep &st = steps[k0 + u];
                f[u] = cols.load(st.from, st.from != nullptr);
                if (ADD) old[u] = cols.load(st.to, st.to && st.table);
            }
#pragma unroll
            for (int u = 0; u < kReduceAhead; u++) {
                const RunStep &st = steps[k0 + u];
                if (!st.from) continue;
#pragma unroll
                for (int e = 0; e < N; e++) sum[e] += f[u].get(e);
                if (!st.to) continue;
                if (st.table) cols.finish(st.to, sum, a.scale, ADD, old[ADD ? u : 0]);
                else cols.store_part(reinterpret_cast<float *>(st.to), sum);
#pragma unroll
                for (int e = 0; e < N; e++) sum[e] = 0.0f;
            }
        }
        __syncthreads();
    }
}

// A run that begins in chunk blockIdx.x and goes on beyond it.  `width` threads
// have the columns; the CTA's kReduceThreads / width groups of them take the run's
// chunks in turn, and their sums are added in order.
template <int DT, bool VEC, bool ADD>
__global__ void __launch_bounds__(kReduceThreads, 4) embedding_join_kernel(const __grid_constant__ SortArgs s, int width) {
    using Cols = GradCols<DT, VEC>;
    constexpr int N = Cols::N;
    __shared__ float sums[N][kReduceThreads];
    const EmbedArgs &a = s.e;
    pdl_wait();
    pdl_launch_dependents();
    const uint2 *items = s.items[s.passes & 1];
    const int c0 = blockIdx.x;
    const long long lo = (long long)c0 * s.chunk, hi = min(lo + s.chunk, a.n_tokens);
    if (hi == a.n_tokens) return;
    const unsigned key = items[hi - 1].x, next = items[hi].x, before = lo ? items[lo - 1].x : (unsigned)a.vocab;
    // (one that reaches back before the chunk is the business of an earlier CTA)
    if (key == (unsigned)a.vocab || next != key || before == key) return;
    // the chunk that it ends in: the chunks after c0 that begin with its key
    int last = c0;
    for (int c = c0 + 1;; c += kReduceThreads) {
        const int mine = c + (int)threadIdx.x;
        const int more = __syncthreads_count(mine < s.n_chunks && items[(long long)mine * s.chunk].x == key);
        last += more;
        if (more < kReduceThreads) break;
    }
    const int group = threadIdx.x / width, groups = kReduceThreads / width;
    const Cols cols{a.dim, (long long)blockIdx.y * width * N, (int)threadIdx.x % width, width};
    char *row = table_row(a, Chunks(a.vocab, a.p), key, ElemInfo<DT>::bytes);
    const typename Cols::Bits old = cols.load(row, ADD && group == 0);
    float sum[N] = {};
    // part 1 of the first chunk, part 0 of the others
    auto part_of = [&](int c) { return s.part + ((long long)c * 2 + (c == c0 ? 1 : 0)) * a.dim; };
    constexpr int kAhead = 4;  // chunks whose loads are in flight together
#pragma unroll 1
    for (int c = c0 + group; c <= last; c += kAhead * groups) {
        float f[kAhead][N];
#pragma unroll
        for (int u = 0; u < kAhead; u++) cols.load_part(part_of(min(c + u * groups, last)), f[u]);
#pragma unroll
        for (int u = 0; u < kAhead; u++)
            if (c + u * groups <= last)
#pragma unroll
                for (int e = 0; e < N; e++) sum[e] += f[u][e];
    }
#pragma unroll
    for (int e = 0; e < N; e++) sums[e][threadIdx.x] = sum[e];
    __syncthreads();
    if (group) return;
    for (int w = 1; w < groups; w++)
#pragma unroll
        for (int e = 0; e < N; e++) sum[e] += sums[e][w * width + threadIdx.x];
    cols.finish(row, sum, a.scale, ADD, old);
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
    if (a->dim > 0x7FFFFFFFu) return c.bad("dim must be at most 2^31 - 1");  // (columns are counted in 32 bits)
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

    const long long table_stride = (long long)(a->table_stride ? a->table_stride : a->dim), row_stride = (long long)(a->out_stride ? a->out_stride : a->dim);
    const size_t ve = 16 / e;
    bool vec = a->dim % ve == 0 && vec16(a->out, a->n_tokens, row_stride, e);
    for (int r = 0; r < a->p && vec; r++) vec = vec16(a->tables[r], a->vocab / a->p + 1, table_stride, e);
    // 4 loads in flight a thread where that still leaves 4 CTAs an SM, else one
    const size_t count = vec ? a->n_tokens * (a->dim / ve) : a->n_tokens * a->dim;
    const bool many = count >= (size_t)h->sm_count * 4 * 1024;
    const size_t ctas = many ? (count + 1023) / 1024 : (count + 255) / 256;
    if (ctas > 0x7FFFFFFFu) return c.bad("the lookup is too large");

    DeviceGuard dg(h->device);
    if (dg.err != cudaSuccess) return cuda_fail(h, dg.err, "selecting the device");
    EmbedArgs k{};
    if ((rc = fill_ptrs(h, k.pieces, const_cast<void *const *>(a->tables), a->p, stream)) != RAR_OK) return rc;
    k.p = a->p;
    k.vocab = (long long)a->vocab;
    k.dim = (long long)a->dim;
    k.n_tokens = (long long)a->n_tokens;
    k.table_stride = table_stride;
    k.row_stride = row_stride;
    k.tokens = a->tokens;
    k.index_bytes = a->index_bytes;
    k.scale = a->scale;
    k.out = a->out;
    note_op_call(h, a->p, stream);
    cudaError_t ce = dispatch_float(a->dtype, [&](auto dt) {
        constexpr int DT = decltype(dt)::value;
        return launch_pdl(vec ? (many ? embedding_kernel<DT, true, 4> : embedding_kernel<DT, true, 1>)
                              : (many ? embedding_kernel<DT, false, 4> : embedding_kernel<DT, false, 1>),
                          dim3((unsigned)ctas), dim3(256), 0, stream, k);
    });
    return ce == cudaSuccess ? RAR_OK : cuda_fail(h, ce, "launching the lookup");
}

size_t grad_plan(void *base, size_t n_tokens, size_t vocab, size_t dim, SortArgs *s) {
    WorkspacePlan w(base);
    // chunks of 16 to 64 places while that makes about 1024 of them, and never
    // more than 4096, so that their sums stay small against dout
    const size_t chunk = std::max({(size_t)kMinChunk, std::min<size_t>(64, n_tokens / 1024), (n_tokens + 4095) / 4096}), n = (n_tokens + chunk - 1) / chunk;
    s->chunk = (int)chunk;
    s->n_chunks = (int)n;
    s->items[0] = w.take<uint2>(n_tokens);
    s->items[1] = w.take<uint2>(n_tokens);
    s->part = w.take<float>(n > 1 ? n * 2 * dim : 0);
    s->bits = 1;
    while (((size_t)1 << s->bits) <= vocab) s->bits++;  // 0 .. vocab, which stands for left out
    s->passes = (s->bits + kSortMaxBits - 1) / kSortMaxBits;
    return w.used;
}

// The launch of the sorting cluster.
template <typename... Params, typename... Args>
cudaError_t launch_sort(void (*kern)(Params...), unsigned cluster, cudaStream_t stream, Args &&...args) {
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kSortSmem);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(cluster);
    cfg.blockDim = dim3(kSortThreads);
    cfg.dynamicSmemBytes = kSortSmem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = cluster;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = cluster > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kern, std::forward<Args>(args)...);
}

int embedding_grad(rar_ctx *h, const rar_embedding_grad_args *a, cudaStream_t stream) {
    OpCheck c(h, "rar_embedding_grad");
    if (!a) return c.bad("args is NULL");
    int rc = c.dtype(a->dtype, true);
    if (rc != RAR_OK) return rc;
    if (a->p < 1 || a->p > RAR_MAX_P) return c.bad("p must be in [1, RAR_MAX_P]");
    if (a->vocab < 1 || a->dim < 1) return c.bad("vocab and dim must be at least 1");
    if (a->vocab > 0x7FFFFFFFu) return c.bad("vocab must be at most 2^31 - 1");
    if (a->n_tokens > (size_t)1 << 24) return c.bad("n_tokens must be at most 2^24");
    if (a->dim > (size_t)1 << 22) return c.bad("dim must be at most 2^22");
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
    SortArgs sort{};
    rc = c.workspace(a->workspace, a->workspace_bytes, grad_plan(nullptr, a->n_tokens, a->vocab, a->dim, &sort));
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
    grad_plan(a->workspace, a->n_tokens, a->vocab, a->dim, &sort);
    sort.e = k;
    const size_t ve = 16 / e;
    bool vec = a->dim % ve == 0 && vec16(a->dout, a->n_tokens, k.row_stride, e);
    for (int r = 0; r < a->p && vec; r++) vec = vec16(a->dtables[r], a->vocab / a->p + 1, k.table_stride, e);
    const unsigned sorters = a->n_tokens <= (size_t)kSortOneCta ? 1 : kSortCluster;
    cudaError_t ce = dispatch_float(a->dtype, [&](auto dt) {
        constexpr int DT = decltype(dt)::value;
        auto steps = [&](auto vv) {
            constexpr bool VEC = decltype(vv)::value != 0;
            cudaError_t e1 = cudaSuccess;
            if (!a->accumulate)
                e1 = launch_pdl(embedding_clear_kernel<DT>, dim3((unsigned)(h->sm_count * kClearCtas)), dim3(kClearThreads), 0, stream, k);
            if (e1 != cudaSuccess || a->n_tokens == 0) return e1;
            e1 = launch_sort(embedding_sort_kernel<DT>, sorters, stream, sort, !a->accumulate);
            if (e1 != cudaSuccess) return e1;
            constexpr int N = GradCols<DT, VEC>::N;
            // no more threads than the row has columns for
            const int threads = (int)std::min<size_t>(((a->dim + N - 1) / N + 31) / 32 * 32, kReduceThreads);
            const dim3 grid((unsigned)sort.n_chunks, (unsigned)((a->dim + threads * N - 1) / (threads * N)));
            e1 = launch_pdl(a->accumulate ? embedding_runs_kernel<DT, VEC, true> : embedding_runs_kernel<DT, VEC, false>, grid, dim3((unsigned)threads),
                            0, stream, sort);
            const int width = threads >= 128 ? 128 : threads >= 64 ? 64 : 32;  // divides the CTA
            const dim3 joins((unsigned)sort.n_chunks, (unsigned)((a->dim + width * N - 1) / (width * N)));
            if (e1 == cudaSuccess && sort.n_chunks > 1)
                e1 = launch_pdl(a->accumulate ? embedding_join_kernel<DT, VEC, true> : embedding_join_kernel<DT, VEC, false>, joins,
                                dim3(kReduceThreads), 0, stream, sort, width);
            return e1;
        };
        return vec ? steps(IntC<1>{}) : steps(IntC<0>{});
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
    if (vocab < 1 || vocab > 0x7FFFFFFFu || dim < 1 || n_tokens > (size_t)1 << 24) return 0;
    rar::SortArgs s{};
    return rar::grad_plan(nullptr, n_tokens, vocab, dim, &s);
}

int rar_embedding_grad(rar_handle h, const rar_embedding_grad_args *a, void *stream) {
    return rar::guarded(h, [&] {
        if (!h) return rar::fail(nullptr, RAR_EINVAL, "handle is NULL");
        return rar::embedding_grad(h, a, (cudaStream_t)stream);
    });
}

}  // extern "C"

// vocab_stream.cuh -- logits of a few tokens: the pieces of the vocabulary streamed
// once, with the vocabulary along the tensor cores' 128 rows and the tokens along
// their columns.
//
// Bound by memory: 2 vocab x dim bytes.  65536 x 4096 bf16 take 85 us for 16 tokens and 89 for 64 (6.0 to 6.3
// TB/s, 0.9 of a copy); 32768 x 2048 26 us, of which some 5 are the first loads' and the last epilogue's.  A CTA an SM takes passes of up to 256
// vocabulary rows, as many in each as give all CTAs the same share; a stage of its
// ring holds 64 columns of dim of all the pass's rows, one box, and of the hidden states, so
// that these are read once a pass.  A sum of 1024 of dim has accumulators of its own (see
// kStepsPerSum in vocab_tiles.cuh), which are added in registers at the end; where tensor memory has
// room for a second set of them, that takes the next pass meanwhile.
#pragma once

#include "vocab_tiles.cuh"

namespace rar {

struct StreamArgs {
    int base, extra;       // chunk_bounds(vocab, p)
    int rows;              // of a pass
    int nb_big, nb_small;  // passes of a piece of base + 1 / base rows
    int passes;
    int tokens, columns;   // columns of the product: tokens, to a multiple of 16
    int steps;             // of 64 along dim
    int sums;              // accumulators of a tile
    int tiles;             // of 128 rows in a pass, 1 or 2
    int sets;              // of accumulators, 1 or 2
    int stages, stage_bytes;
    float *logits;         // [tokens][pitch], by index in the vocabulary
    long long pitch;
    WaitLimits limits;
};

constexpr int kStreamMaxTokens = 128, kStreamMaxStages = 12, kStreamEpilogueWarps = 8;
constexpr int kStreamThreads = 32 * (kStreamEpilogueWarps + 2);
constexpr int kStreamSmem = 225 * 1024;

struct StreamShared {
    uint64_t full[kStreamMaxStages], empty[kStreamMaxStages], acc_full[2], acc_empty[2];
    uint32_t tmem;
    int failed;
};

struct PassOf {
    int piece, row, rows, first;  // as BlockOf
};
__device__ __forceinline__ PassOf pass_of(const StreamArgs &a, int i) {
    PassOf o;
    const int big = a.extra * a.nb_big;
    int k;
    if (i < big) {
        o.piece = i / a.nb_big;
        k = i - o.piece * a.nb_big;
    } else {
        o.piece = a.extra + (i - big) / a.nb_small;
        k = (i - big) % a.nb_small;
    }
    o.row = k * a.rows;
    o.rows = min(a.base + (o.piece < a.extra ? 1 : 0) - o.row, a.rows);
    o.first = o.piece * a.base + min(o.piece, a.extra) + o.row;
    return o;
}

__device__ __forceinline__ void stream_load_box(const CUtensorMap *map, uint32_t dst, uint64_t *bar, int x, int y) {
    asm volatile("cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(dst), "l"(map),
                 "r"(x), "r"(y), "r"(smem_u32(bar))
                 : "memory");
}
__device__ __forceinline__ void stream_mma(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool accumulate) {
    asm volatile(
        "{\n\t.reg .pred P;\n\tsetp.ne.u32 P, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, P;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(accumulate ? 1u : 0u)
        : "memory");
}
__device__ __forceinline__ void stream_commit(uint64_t *bar) {
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
}

// Warps 0 to 7: epilogue, two for each 32 lanes of an accumulator, one for each tile; 8: loads,
// 9: products.
template <int DT>
__global__ void __launch_bounds__(kStreamThreads, 1) vocab_stream_kernel(const __grid_constant__ StreamArgs a, const __grid_constant__ VocabMaps maps) {
    extern __shared__ unsigned char dyn[];
    __shared__ StreamShared sh;
    const uint32_t ring = (smem_u32(dyn) + 1023u) & ~1023u;
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    auto wait = [&](uint64_t *bar, uint32_t parity, int role) { return mbar_wait(&sh.failed, a.limits, bar, parity, WAIT_OF_XENT, role); };
    if (threadIdx.x == 0) {
        sh.failed = 0;
        for (int s = 0; s < a.stages; s++) {
            mbar_init(&sh.full[s], 1);
            mbar_init(&sh.empty[s], 1);
        }
        for (int s = 0; s < 2; s++) {
            mbar_init(&sh.acc_full[s], 1);
            mbar_init(&sh.acc_empty[s], kStreamEpilogueWarps);
        }
        mbar_fence_init();
    }
    if (warp == kStreamEpilogueWarps) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_u32(&sh.tmem)) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    pdl_wait();
    pdl_launch_dependents();
    const int hidden_bytes = a.columns * 128;  // of a stage, before its rows of the vocabulary
    if (warp == kStreamEpilogueWarps && lane == 0) {
        unsigned step = 0;
        int st = 0;
        uint32_t phase = 0;
        bool ok = true;
        for (int i = blockIdx.x; i < a.passes && ok; i += gridDim.x) {
            const PassOf b = pass_of(a, i);
            for (int s = 0; s < a.steps; s++) {
                // (a new barrier's preceding phase counts as complete: the first turn does not wait)
                if (!(ok = wait(&sh.empty[st], phase ^ 1, 0))) break;
                const uint32_t to = ring + st * a.stage_bytes;
                mbar_expect_tx(&sh.full[st], (uint32_t)(hidden_bytes + a.rows * 128));
                stream_load_box(&maps.w[b.piece], to + hidden_bytes, &sh.full[st], s * 64, b.row);
                stream_load_box(&maps.one, to, &sh.full[st], s * 64, 0);
                step++;
                if (++st == a.stages) st = 0, phase ^= 1;
            }
        }
        // the CTA may not end, nor give its tensor memory back, while loads or products are under way
        for (unsigned k = step > (unsigned)a.stages ? step - a.stages : 0; k < step; k++) {
            const unsigned s = k % (unsigned)a.stages, turn = k / (unsigned)a.stages;
            if (!mbar_drain(&sh.full[s], turn & 1) || !mbar_drain(&sh.empty[s], turn & 1)) break;
        }
    } else if (warp == kStreamEpilogueWarps + 1 && lane == 0) {
        const uint64_t hidden = tc_operand(ring, 16, 1024), rows = tc_operand(ring + hidden_bytes, 16, 1024);
        const uint32_t type = DT == DT_BF16 ? 1u : 0u, idesc = 1u << 4 | type << 7 | type << 10 | (uint32_t)(a.columns >> 3) << 17 | (128u >> 4) << 24;
        int st = 0;
        uint32_t phase = 0;
        unsigned turn = 0;
        bool ok = true;
        for (int i = blockIdx.x; i < a.passes && ok; i += gridDim.x, turn++) {
            const unsigned set = turn % a.sets, use = turn / a.sets;
            if (use && !wait(&sh.acc_empty[set], (use - 1) & 1, 2)) break;
            tc_fence_after();
            const uint32_t acc = sh.tmem + set * 256;
            for (int s = 0; s < a.steps; s++) {
                if (!(ok = wait(&sh.full[st], phase, 3))) break;
                tc_fence_after();
                const uint64_t off = (uint64_t)(st * (a.stage_bytes / 16));
                const int sum = s / kStepsPerSum;
                for (int t = 0; t < a.tiles; t++)
#pragma unroll
                    for (int k = 0; k < 4; k++)
                        stream_mma(acc + (t * a.sums + sum) * a.columns, rows + off + t * 1024 + k * 2, hidden + off + k * 2, idesc, s % kStepsPerSum || k);
                stream_commit(&sh.empty[st]);
                if (++st == a.stages) st = 0, phase ^= 1;
            }
            if (ok) stream_commit(&sh.acc_full[set]);
        }
    } else if (warp < kStreamEpilogueWarps) {
        const int quarter = warp % 4, tile = warp / 4, row = tile * 128 + quarter * 32 + lane;
        unsigned turn = 0;
        for (int i = blockIdx.x; i < a.passes; i += gridDim.x, turn++) {
            const PassOf b = pass_of(a, i);
            const unsigned set = turn % a.sets, use = turn / a.sets;
            if (!__all_sync(0xFFFFFFFFu, wait(&sh.acc_full[set], use & 1, 4))) break;
            tc_fence_after();
            const uint32_t acc = sh.tmem + ((uint32_t)quarter << 21) + set * 256 + tile * a.sums * a.columns;
            if (tile < a.tiles)
                for (int c0 = 0; c0 < a.tokens; c0 += 8) {
                    float z[8] = {};
                    for (int s = 0; s < a.sums; s++) {
                        float v[8];
                        tc_read8(acc + s * a.columns + c0, v);
                        tc_read_wait();
#pragma unroll
                        for (int c = 0; c < 8; c++) z[c] += v[c];
                    }
                    float *out = a.logits + c0 * a.pitch + b.first + row;
#pragma unroll
                    for (int c = 0; c < 8; c++)
                        if (row < b.rows && c0 + c < a.tokens) out[c * a.pitch] = z[c];
                }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&sh.acc_empty[set]);
        }
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == kStreamEpilogueWarps) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(sh.tmem) : "memory");
}

namespace {

// Whether a call is one of these: the accumulators of two tiles fit into the tensor memory, or those of
// one for up to 64 tokens.
bool stream_fits(size_t tokens, size_t dim) {
    const size_t columns = (tokens + 15) / 16 * 16, sums = (dim + 64 * kStepsPerSum - 1) / (64 * kStepsPerSum);
    return tokens >= 1 && tokens <= kStreamMaxTokens && columns * sums <= (tokens <= 64 ? 512 : 256);
}

size_t stream_pitch(size_t vocab) { return (vocab + 3) / 4 * 4; }

// The shape of a launch on `sms` SMs.
void stream_shape(StreamArgs *s, int tokens, long long dim, int base, int extra, int p, int sms) {
    s->base = base;
    s->extra = extra;
    s->tokens = tokens;
    s->columns = (tokens + 15) / 16 * 16;
    s->steps = (int)((dim + 63) / 64);
    s->sums = (s->steps + kStepsPerSum - 1) / kStepsPerSum;
    // rows of a pass: the fewest for the CTA that has most of them (and, for equal ones, the fewest passes)
    const int tile = s->sums * s->columns, most = 2 * tile <= 512 ? 256 : 128;
    long long least = 0;
    for (int rows = most; rows >= 8; rows -= 8) {
        const int big = (base + 1 + rows - 1) / rows, small = (base + rows - 1) / rows;
        const long long passes = (long long)extra * big + (long long)(p - extra) * small, cost = (passes + sms - 1) / sms * rows;
        if (rows != most && cost >= least) continue;
        least = cost;
        s->rows = rows;
        s->nb_big = big;
        s->nb_small = std::max(small, 1);
        s->passes = (int)passes;
    }
    s->tiles = s->rows > 128 ? 2 : 1;
    s->sets = s->tiles * tile <= 256 ? 2 : 1;
    s->stage_bytes = s->columns * 128 + (s->rows * 128 + 1023) / 1024 * 1024;
    // (a product reads 128 rows of a tile, whatever lies behind the pass's last)
    const int behind = s->tiles * 16384 - (s->stage_bytes - s->columns * 128);
    s->stages = std::min(kStreamMaxStages, (kStreamSmem - 1024 - behind) / s->stage_bytes);
}

bool stream_maps(int dtype, const VocabArgs &k, const StreamArgs &s, VocabMaps *m) {
    bool mapped = make_map(&m->one, dtype, k.hidden, k.tokens, k.dim, k.hidden_stride, s.columns);
    for (int r = 0; r < k.p && mapped; r++) {
        const long long rows = k.base + (r < k.extra ? 1 : 0);
        // (a box without its last row completes no stage)
        if (rows) mapped = make_map(&m->w[r], dtype, k.w.inl[r], rows, k.dim, k.weight_stride, s.rows - (r == k.limits.mute ? 1 : 0));
    }
    return mapped;
}

template <int DT>
cudaError_t launch_stream(const rar_ctx *h, const StreamArgs &s, const VocabMaps &maps, cudaStream_t stream) {
    auto kern = vocab_stream_kernel<DT>;
    const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kStreamSmem);
    if (e != cudaSuccess) return e;
    return launch_pdl(kern, dim3((unsigned)std::min(s.passes, h->sm_count)), dim3(kStreamThreads), kStreamSmem, stream, s, maps);
}

}  // namespace
}  // namespace rar

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
// All four products run on the tensor cores through one kernel (tc_gemm.cuh):
// a pair of CTAs computes a 256 x 256 tile, and the epilogue of a tile overlaps the
// next tile's product (two accumulators).  G is rounded once, to the
// type of the products that it enters: an error of half a unit in its last place, of the
// size that rounding dhidden and dweights has anyway.
//
// Bound by the tensor cores for many tokens (8 tokens x vocab x dim operations
// against 6 if the logits were kept): 8192 tokens by 65536 x 4096 bf16 take 2.5 ms forward
// (1.76 PFLOP/s; 2.7 ms back to back) and 11.4 ms with gradients (1.54 PFLOP/s) at the power
// limit (1.37 kW, which leaves 1725 of 2070 MHz).  For few tokens by the fill of full tiles in two
// uneven waves: 16 by 32768 x 2048 take 38 us, as 256 do (134 MB of weights, 3.5 TB/s).
#include <algorithm>

#include "op_host.h"
#include "tc_gemm.cuh"

namespace rar {

constexpr int kBlock = 256;  // vocabulary rows of a block: a tile's columns
constexpr int kTile = 256;   // rows and columns of a tile

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
    int base, extra;       // chunk_bounds(vocab, p)
    int nb_big, nb_small;  // blocks of a piece of base + 1 / base rows
    int n_blocks;
    // workspace
    float2 *stats;        // [2 n_blocks][tokens]: a half block's max, sum of exp(z - max)
    float *z_target;      // [tokens]
    float *lse_ws;        // [tokens]
    float *row_weight;    // [tokens] scaled token_weight, 0 where left out
    unsigned *w_max;      // bits of the largest finite |token_weight|
    void *hidden_used;    // [tokens][dim]: hidden, zeros where left out
    void *g;              // [tokens][window * kBlock]
    float *dh_part;       // [splits][tokens][dim]
    int window;           // blocks of a window
    int splits;           // of dhidden's sum over a window
    bool direct;          // one split: the last window writes dhidden itself
    WaitLimits limits;
};

// Tensor maps of a launch: `one` is the operand that is one matrix (hidden or G),
// `w` the pieces of W, or hidden as XENT_DWEIGHT's second operand.  Boxes are 64
// elements of 128 rows where K runs along the rows, else of 64.
struct XentMaps {
    CUtensorMap one, w[kInlineP];
};

struct BlockOf {
    int piece;
    int row;    // first row in the piece
    int rows;   // 1 .. kBlock
    int first;  // its index in the vocabulary
};
__device__ __forceinline__ BlockOf block_of(const XentArgs &a, int b) {
    BlockOf o;
    const unsigned big = (unsigned)(a.extra * a.nb_big), u = (unsigned)b;
    unsigned k;
    if (u < big) {
        o.piece = (int)(u / (unsigned)a.nb_big);
        k = u % (unsigned)a.nb_big;
    } else {
        o.piece = a.extra + (int)((u - big) / (unsigned)a.nb_small);
        k = (u - big) % (unsigned)a.nb_small;
    }
    o.row = (int)k * kBlock;
    o.rows = min(a.base + (o.piece < a.extra ? 1 : 0) - o.row, kBlock);
    o.first = o.piece * a.base + min(o.piece, a.extra) + o.row;
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

// G is also divided by the largest weight's significand, in [1, 2).  Where all tokens weigh
// the same (a mean), (softmax - 1) weight, the largest entry of a row, else
// rounds in the same direction for every unforeseen target, by up to half a unit in
// the last place: as much as the gradients' own rounding, and the same for all.
__device__ __forceinline__ float g_unit(const XentArgs &a) {
    const float m = __uint_as_float(*a.w_max);
    return m > 0.0f ? ldexpf(m, -ilogbf(m)) : 1.0f;
}
// What undoes both.
template <int DT>
__device__ __forceinline__ float g_undo(const XentArgs &a) {
    return ldexpf(g_unit(a), -g_exponent<DT>(a));
}

enum XentMode { XENT_STATS, XENT_G, XENT_DHIDDEN, XENT_DWEIGHT, XENT_STATS_SUMS, XENT_G_SUMS };  // (_SUMS: see kStepsPerSum)
template <int MODE>
struct Mode {
    static constexpr bool sums = MODE == XENT_STATS_SUMS || MODE == XENT_G_SUMS;
    static constexpr bool stats = MODE == XENT_STATS || MODE == XENT_STATS_SUMS, g = MODE == XENT_G || MODE == XENT_G_SUMS, logits = stats || g;
    // whether a row of the operand is a row of K (MN-major); rows of a box; boxes of a stage
    static constexpr bool a_mn = MODE == XENT_DWEIGHT, b_mn = MODE == XENT_DHIDDEN || MODE == XENT_DWEIGHT;
    static constexpr int a_box = a_mn ? 64 : 128, b_box = b_mn ? 64 : 128;
    static constexpr int a_boxes = 128 / a_box, b_boxes = 128 / b_box;
};

// One tile of a pair of CTAs: its place, and its range along K.
struct XentItem {
    int row;     // first row of the tile (token, row of the window's blocks, or 0)
    int col;     // first column (of dim, or 0)
    int n;       // columns that the product covers, a multiple of 32
    int block;   // block of the window (not XENT_DHIDDEN)
    int split;
    int k0, k1;  // XENT_DHIDDEN: blocks of the window; else steps of 64
};

__host__ __device__ inline int tiles_of(long long n) { return (int)((n + kTile - 1) / kTile); }
__device__ __forceinline__ int round32(int n) { return n >= kTile ? kTile : (n + 31) / 32 * 32; }

// Tiles in an order in which those that run at one time share operands:
// columns of 8 tiles, so that 76 pairs work on about 8 x 9 tiles.
template <int MODE>
__device__ __forceinline__ XentItem xent_item(const XentArgs &a, int b0, int nb, int i) {
    XentItem o;
    o.split = 0;
    o.block = 0;
    o.col = 0;
    o.k0 = 0;
    const unsigned tb = (unsigned)tiles_of(a.tokens), db = (unsigned)tiles_of(a.dim);
    const unsigned rows = MODE == XENT_DWEIGHT ? (unsigned)nb : tb;
    const unsigned cols = MODE == XENT_DHIDDEN ? db * (unsigned)a.splits : MODE == XENT_DWEIGHT ? db : (unsigned)nb;
    const unsigned g = (unsigned)i / (8 * cols), in = (unsigned)i - g * 8 * cols;
    const unsigned width = min(rows - g * 8, 8u), c = in / width;
    const int r = (int)(g * 8 + in - c * width);
    o.row = r * kTile;
    if (Mode<MODE>::logits) {
        o.block = (int)c;
        o.n = round32(block_of(a, b0 + (int)c).rows);
        o.k1 = (int)((a.dim + 63) / 64);
    } else if (MODE == XENT_DHIDDEN) {
        o.split = (int)(c / db);
        o.col = (int)(c % db) * kTile;
        o.n = round32((int)a.dim - o.col);
        o.k0 = (int)((long long)nb * o.split / a.splits);
        o.k1 = (int)((long long)nb * (o.split + 1) / a.splits);
    } else {
        o.block = r;
        o.col = (int)c * kTile;
        o.n = round32((int)a.dim - o.col);
        o.k1 = (int)((a.tokens + 63) / 64);
    }
    return o;
}
template <int MODE>
__host__ __device__ inline int xent_items(const XentArgs &a, int nb) {
    const int tb = tiles_of(a.tokens), db = tiles_of(a.dim);
    return MODE == XENT_DHIDDEN ? tb * db * a.splits : MODE == XENT_DWEIGHT ? nb * db : tb * nb;
}

// Calls f for every step of 64 along K: f(step within the block or the
// range, block of the window, the block).  Stops when f returns false.
template <int MODE, typename F>
__device__ __forceinline__ bool xent_steps(const XentArgs &a, int b0, const XentItem &it, F &&f) {
    if constexpr (MODE == XENT_DHIDDEN) {
        for (int k = it.k0; k < it.k1; k++) {
            const BlockOf b = block_of(a, b0 + k);
            for (int s = 0; s * 64 < b.rows; s++)
                if (!f(s, k, b)) return false;
        }
    } else {
        const BlockOf b = block_of(a, b0 + it.block);
        for (int s = it.k0; s < it.k1; s++)
            if (!f(s, it.block, b)) return false;
    }
    return true;
}

// Good to (2 + |x|) 2^-23: ex2.approx to 2 units in the last place, the rounding of its argument
// to |x| 2^-24 and a little for the constant.  A large |x| has a weight of exp(-|x|) in the sums
// of exponentials, and in G, which is rounded to 8 or 11 bits, no relative error of its size shows.
__device__ __forceinline__ float exp_of(float x) {
    float r;
    asm("ex2.approx.f32 %0, %1;" : "=f"(r) : "f"(x * 1.4426950408889634f));
    return r;
}
// Eight values times a power of two, rounded.
template <int DT>
__device__ __forceinline__ uint4 narrow8_scaled(const float *v, float scale) {
    float f[8];
#pragma unroll
    for (int e = 0; e < 8; e++) f[e] = v[e] * scale;
    return narrow8<DT>(f);
}

// The tensor cores add to a 32-bit accumulator by truncation: an instruction loses some
// 1.5 x 2^-23 of it, always towards zero.  Over the whole of dim the logits came out low by some
// 1e-6 of their size at dim 2048 (a rounding sum: 4e-7), and where all products have one sign
// by 1e-4 at dim 16384, so that exp(z - lse) with logits near 9000 was off by a factor of 0.4.  So
// both passes that make logits, for a dim above that of one sum, end their accumulators
// every 16 steps (1024 of dim) and add them up in registers: 5e-7.  It costs 8 to 10 % of
// a long forward pass (2048 tokens by 50021 x 2048 fp16 314 us against 282, 8192 by 65536 x 4096
// bf16 2.54 ms against 2.33), 3 to 4 % with gradients.  A dim of one sum keeps the plain form
// and its time.  Products whose results are rounded to 16 bits do without.
constexpr int kStepsPerSum = 16;

// What an epilogue thread keeps of a tile: one row of it.
struct XentRow {
    int row;          // of tokens (or of the block, XENT_DWEIGHT)
    bool live;        // the row exists
    int cols;         // columns of its half that exist
    int target;       // column of its target in its half, or one out of range
    float w, lse;     // logits for G
    float max, sum;   // logits for the statistics
    char *out;        // where the row's half begins
    float *part;      // XENT_DHIDDEN: the sums so far
};

template <int MODE, int DT>
__device__ __forceinline__ XentRow xent_row(const XentArgs &a, int b0, const XentItem &it, int row, int half) {
    XentRow r;
    r.row = row;
    r.out = nullptr;
    r.part = nullptr;
    if constexpr (MODE == XENT_DHIDDEN) {
        r.live = row < a.tokens;
        r.cols = (int)a.dim - it.col - half;
        r.out = static_cast<char *>(a.dhidden) + (row * a.dhidden_stride + it.col + half) * 2;
        r.part = a.dh_part + ((long long)it.split * a.tokens + row) * a.dim + it.col + half;
    } else if constexpr (MODE == XENT_DWEIGHT) {
        const BlockOf b = block_of(a, b0 + it.block);
        r.row = row - it.row;
        r.live = r.row < b.rows;
        r.cols = (int)a.dim - it.col - half;
        r.out = rank_ptr(a.dw, a.p, b.piece) + ((long long)(b.row + r.row) * a.dweight_stride + it.col + half) * 2;
    } else {
        const BlockOf b = block_of(a, b0 + it.block);
        r.live = row < a.tokens;
        r.cols = b.rows - half;
        const long long y = r.live ? load_index(a.targets, a.index_bytes, row) - b.first - half : -1;
        r.target = y >= 0 && y < r.cols ? (int)y : -1;
        r.max = -INFINITY;
        r.sum = 0.0f;
        if constexpr (Mode<MODE>::g) {
            r.w = r.live ? ldexpf(a.row_weight[row] / g_unit(a), g_exponent<DT>(a)) : 0.0f;
            r.lse = r.live ? a.lse_ws[row] : 0.0f;
            r.out = static_cast<char *>(a.g) + (((long long)row * a.window + it.block) * kBlock + half) * 2;
        }
    }
    return r;
}

// Columns c0 .. c0 + 31 of the row's half.
template <int MODE, int DT>
__device__ __forceinline__ void xent_columns(const XentArgs &a, XentRow &r, int c0, float undo, bool first, bool direct, float (&v)[32]) {
    if (!r.live) return;
    const int cols = r.cols - c0;
    if constexpr (Mode<MODE>::stats) {
        if (cols <= 0) return;
        if (cols < 32) {
#pragma unroll
            for (int c = 0; c < 32; c++) v[c] = c < cols ? v[c] : -INFINITY;
        }
        const int y = r.target - c0;
        if (y >= 0 && y < 32) {
            float z = 0.0f;
#pragma unroll
            for (int c = 0; c < 32; c++)  // (in this form v stays in registers)
                asm("{\n\t.reg .pred P;\n\tsetp.eq.s32 P, %1, %2;\n\tselp.f32 %0, %3, %0, P;\n\t}" : "+f"(z) : "r"(y), "r"(c), "f"(v[c]));
            a.z_target[r.row] = z;
        }
        float m = r.max;
#pragma unroll
        for (int c = 0; c < 32; c++) m = fmaxf(m, v[c]);
        // nothing but -inf (or NaN, which the sum then shows)
        const float ref = m == -INFINITY ? 0.0f : m;
        float s = r.sum * exp_of(r.max - ref);
#pragma unroll
        for (int c = 0; c < 32; c++) s += exp_of(v[c] - ref);
        r.max = m;
        r.sum = s;
    } else if constexpr (Mode<MODE>::g) {
        const int y = r.target - c0;
#pragma unroll
        for (int c = 0; c < 32; c++) {
            const float p = exp_of(v[c] - r.lse) - (c == y ? 1.0f : 0.0f);
            v[c] = c < cols && r.w != 0.0f ? p * r.w : 0.0f;
        }
#pragma unroll
        for (int c = 0; c < 32; c += 16) {
            const uint4 x = narrow8<DT>(v + c), y4 = narrow8<DT>(v + c + 8);
            const uint32_t q[8] = {x.x, x.y, x.z, x.w, y4.x, y4.y, y4.z, y4.w};
            store_32b(r.out + (c0 + c) * 2, q);
        }
    } else if constexpr (MODE == XENT_DHIDDEN) {
#pragma unroll
        for (int c = 0; c < 32; c += 8) {
            if (c >= cols) continue;
            float *part = r.part + c0 + c;
            if (!first) {
                uint32_t q[8];
                load_32b(part, q);
#pragma unroll
                for (int e = 0; e < 8; e++) v[c + e] += __uint_as_float(q[e]);
            }
            if (direct) {
                *reinterpret_cast<uint4 *>(r.out + (c0 + c) * 2) = narrow8_scaled<DT>(v + c, undo);
            } else {
                uint32_t q[8];
#pragma unroll
                for (int e = 0; e < 8; e++) q[e] = __float_as_uint(v[c + e]);
                store_32b(part, q);
            }
        }
    } else {
#pragma unroll
        for (int c = 0; c < 32; c += 8)
            if (c < cols) *reinterpret_cast<uint4 *>(r.out + (c0 + c) * 2) = narrow8_scaled<DT>(v + c, undo);
    }
}

// Adds sums of exponentials, each relative to its maximum.
__device__ __forceinline__ void add_exp(float &m, float &s, float om, float os) {
    if (os == 0.0f) return;  // nothing there
    const float top = fmaxf(m, om);
    // (a block of -inf or NaN alone has a sum of its own to keep)
    s = top == -INFINITY ? s + os : s * exp_of(m - top) + os * exp_of(om - top);
    m = top;
}

// Persistent: a pair of CTAs takes tiles i, i + pairs, ...  Warps 0 to 7: epilogue,
// 8: loads, 9 (of the pair's first CTA): products.  The epilogue reads its half
// row 32 columns at a time: the code of all 128 at once is four times as long, and
// its instruction fetches showed in calls of a few tiles.
// At most 152 registers: three warps of this kernel then leave each quarter of an SM
// room for a warp of 32, so that a CTA of the join can wait there for the end.
template <int MODE, int DT>
__global__ void __cluster_dims__(2, 1, 1) __maxnreg__(152)
    xent_tile_kernel(const __grid_constant__ XentArgs a, const __grid_constant__ XentMaps maps, int b0, int nb) {
    extern __shared__ unsigned char dyn[];
    __shared__ TcShared sh;
    const uint32_t stages = (smem_u32(dyn) + 1023u) & ~1023u;
    const uint32_t rank = cluster_rank();
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    if (threadIdx.x < 2) tc_prefetch_map(threadIdx.x ? &maps.w[0] : &maps.one);
    tc_begin(&sh);
    pdl_wait();
    pdl_launch_dependents();
    if (Mode<MODE>::stats && blockIdx.x == 0 && threadIdx.x == 0) *a.w_max = 0u;
    const int items = xent_items<MODE>(a, nb), pairs = gridDim.x / 2, first = blockIdx.x / 2;
    constexpr bool a_mn = Mode<MODE>::a_mn, b_mn = Mode<MODE>::b_mn;
    constexpr int kABoxes = Mode<MODE>::a_boxes, kLoaders = kABoxes + Mode<MODE>::b_boxes;
    if (warp == kTcEpilogueWarps && lane < kLoaders) {
        // a lane a box, first those of A
        constexpr unsigned kLanes = (1u << kLoaders) - 1;
        const bool is_a = lane < kABoxes;
        const int part = is_a ? lane * Mode<MODE>::a_box : (lane - kABoxes) * Mode<MODE>::b_box;  // rows (columns) into the operand
        unsigned step = 0;
        uint32_t st = 0, phase = 0;
        for (int i = first; i < items && !__any_sync(kLanes, *(volatile int *)&sh.failed); i += pairs) {
            const XentItem it = xent_item<MODE>(a, b0, nb, i);
            xent_steps<MODE>(a, b0, it, [&](int s, int k, const BlockOf &b) {
                // (a new barrier's preceding phase counts as complete: the first turn does not wait)
                if (!__all_sync(kLanes, tc_wait(&sh, a.limits, &sh.empty[st], phase ^ 1, 0))) return false;
                // a CTA whose rows of A all lie past the last loads none of them: its
                // rows of the accumulator are never read
                auto a_rows = [&](int r) { return MODE == XENT_DWEIGHT || it.row + r * 128 < a.tokens; };
                if (rank == 0 && lane == 0)
                    mbar_expect_tx(&sh.full[st], 32768u + 16384u * (1u + a_rows(1)));
                const uint32_t bar = peer_addr(smem_u32(&sh.full[st]), 0);
                const uint32_t to = stages + st * kTcStageBytes + (is_a ? 0 : 16384) + part * 128;
                const CUtensorMap *map = is_a ? &maps.one : &maps.w[MODE == XENT_DWEIGHT ? 0 : b.piece];
                const int row = it.row + (int)rank * 128 + part, col = it.col + (int)rank * it.n / 2 + part;
                int x, y;
                if (MODE == XENT_DHIDDEN) x = is_a ? k * kBlock + s * 64 : col, y = is_a ? row : b.row + s * 64;
                else if (MODE == XENT_DWEIGHT) x = is_a ? row : col, y = s * 64;
                else x = s * 64, y = is_a ? row : b.row + col;
                if (!is_a || a_rows((int)rank)) tc_load_box(map, to, bar, x, y);
                step++;
                if (++st == kTcStages) st = 0, phase ^= 1;
                return true;
            });
        }
        // neither CTA may leave while the pair's loads, products or arrivals are under way,
        // nor give its tensor memory back, even after a wait that ran out: products in flight
        // belong to the last stages, whose `empty` they arrive at in both CTAs
        for (unsigned k = step > kTcStages ? step - kTcStages : 0; k < step && lane == 0; k++) {
            const int st = (int)(k % kTcStages);
            if (rank == 0 && !mbar_drain(&sh.full[st], (k / kTcStages) & 1)) break;
            if (!mbar_drain(&sh.empty[st], (k / kTcStages) & 1)) break;
        }
    } else if (warp == kTcEpilogueWarps + 1 && lane == 0 && rank == 0) {
        const uint64_t operand_a = tc_operand(stages, a_mn ? 8192 : 16, 1024), operand_b = tc_operand(stages + 16384, b_mn ? 8192 : 16, 1024);
        // the next stage and its phase; accumulators begun.  (This thread issues a step of 64
        // every 512 cycles or so: what it computes between two steps is time lost.)
        uint32_t st = 0, phase = 0, sums = 0;
        for (int i = first; i < items; i += pairs) {
            const XentItem it = xent_item<MODE>(a, b0, nb, i);
            const uint32_t idesc = tc_instruction(DT == DT_BF16, a_mn, b_mn, (uint32_t)it.n);
            uint32_t d = 0;
            int left = 0;  // steps that the present accumulator takes yet
            bool more = false;
            const bool ok = xent_steps<MODE>(a, b0, it, [&](int, int, const BlockOf &) {
                if (left == 0) {
                    if (more) tc_commit(&sh.acc_full[(sums - 1) & 1]);
                    if (sums >= 2 && !tc_wait(&sh, a.limits, &sh.acc_empty[sums & 1], (sums / 2 - 1) & 1, 2)) return false;
                    tc_fence_after();
                    d = sh.tmem + (sums & 1) * kTile;
                    sums++;
                    left = Mode<MODE>::sums ? kStepsPerSum : 0x7FFFFFFF;
                    more = false;
                }
                if (!tc_wait(&sh, a.limits, &sh.full[st], phase, 3)) return false;
                tc_fence_after();
                // descriptors count addresses in units of 16 bytes
                const uint64_t da = operand_a + st * (kTcStageBytes / 16), db = operand_b + st * (kTcStageBytes / 16);
#pragma unroll
                for (int k = 0; k < 4; k++) {
                    tc_mma(d, da + k * (a_mn ? 128 : 2), db + k * (b_mn ? 128 : 2), idesc, more);
                    more = true;
                }
                tc_commit(&sh.empty[st]);
                if (++st == kTcStages) st = 0, phase ^= 1;
                left--;
                return true;
            });
            if (!ok) break;
            tc_commit(&sh.acc_full[(sums - 1) & 1]);
        }
    } else if (warp < kTcEpilogueWarps) {
        const int quarter = warp % 4;
        const float undo = MODE == XENT_DHIDDEN || MODE == XENT_DWEIGHT ? g_undo<DT>(a) : 1.0f;
        const bool first_window = b0 == 0, direct = a.direct && b0 + nb == a.n_blocks;
        unsigned sums = 0;  // accumulators read
        auto ready = [&] {
            const bool ok = __all_sync(0xFFFFFFFFu, tc_wait(&sh, a.limits, &sh.acc_full[sums & 1], (sums / 2) & 1, 4));
            tc_fence_after();
            return ok;
        };
        auto release = [&] {
            tc_fence_before();
            __syncwarp();
            if (lane == 0) tc_arrive_cluster(peer_addr(smem_u32(&sh.acc_empty[sums & 1]), 0));
            sums++;
        };
        bool ok = true;
        for (int i = first; i < items; i += pairs) {
            const XentItem it = xent_item<MODE>(a, b0, nb, i);
            const int half = warp / 4 * 128, row = it.row + (int)rank * 128 + quarter * 32 + lane;
            XentRow r = xent_row<MODE, DT>(a, b0, it, row, half);
            auto at = [&](int c) { return sh.tmem + ((uint32_t)quarter << 21) + (sums & 1) * kTile + half + c; };
            if (Mode<MODE>::sums) {
                // all sums but the last into registers, and these onto the last
                float z[128];
#pragma unroll
                for (int c = 0; c < 128; c++) z[c] = 0.0f;
#pragma unroll 1
                for (int k = kStepsPerSum; k < it.k1; k += kStepsPerSum) {
                    if (!(ok = ready())) break;
#pragma unroll
                    for (int q = 0; q < 128; q += 8) {
                        float v[8];
                        tc_read8(at(q), v);
                        tc_read_wait();
#pragma unroll
                        for (int c = 0; c < 8; c++) z[q + c] += v[c];
                    }
                    release();
                }
                if (!ok || !(ok = ready())) break;
#pragma unroll
                for (int q = 0; q < 128; q += 8) {
                    float v[8];
                    tc_read8(at(q), v);
                    tc_read_wait();
#pragma unroll
                    for (int c = 0; c < 8; c++) v[c] += z[q + c];
                    tc_write8(at(q), v);
                }
                tc_write_wait();
            } else if (!(ok = ready())) {
                break;
            }
#pragma unroll 1
            for (int c0 = 0; c0 < 128; c0 += 32) {
                float v[32];
                tc_read32(at(c0), v);
                tc_read_wait();
                xent_columns<MODE, DT>(a, r, c0, undo, first_window, direct, v);
            }
            release();
            if constexpr (Mode<MODE>::stats)
                if (r.live) a.stats[(2ll * (b0 + it.block) + half / 128) * a.tokens + row] = make_float2(r.max, r.sum);
        }
    }
    __syncwarp();
    tc_end(&sh);
}

// Joins the blocks of some tokens, a warp a token, to lse and loss; with gradients also their
// weights and hidden states, cleared where a token is left out (0 x NaN is not 0
// in dweights' sum).  Without gradients a CTA is small enough to stand beside one of
// the tile kernel and wait there for its end: 256 tokens by 32768 x 2048 took 37 us
// so and 48 us with 8 tokens a CTA; with gradients 8 tokens, whose loads are in flight
// together, took 262 us of a whole call against 281 (1024 by 32000 x 1024; the call takes 230 now).
template <bool GRAD>
constexpr int kJoinTokens = GRAD ? 8 : 4;
template <int DT, bool GRAD>
__global__ void __launch_bounds__(32 * kJoinTokens<GRAD>, GRAD ? 1 : 16) xent_join_kernel(const __grid_constant__ XentArgs a) {
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

// dhidden from the splits' sums.
template <int DT>
__global__ void __launch_bounds__(256) xent_dhidden_join_kernel(const __grid_constant__ XentArgs a) {
    pdl_wait();
    pdl_launch_dependents();
    const float undo = g_undo<DT>(a);
    const long long vecs = a.dim / 8, n = a.tokens * vecs;
    for (long long i = (long long)blockIdx.x * blockDim.x + threadIdx.x; i < n; i += (long long)gridDim.x * blockDim.x) {
        const long long t = n < 0x7FFFFFFF ? (long long)((uint32_t)i / (uint32_t)vecs) : i / vecs, d = (i - t * vecs) * 8;
        const float *part = a.dh_part + t * a.dim + d;
        const long long pitch = a.tokens * a.dim;
        float v[8] = {};
        for (int k0 = 0; k0 < a.splits; k0 += 4) {
            uint32_t q[4][8];  // loads in flight together
#pragma unroll
            for (int k = 0; k < 4; k++) load_32b(part + min(k0 + k, a.splits - 1) * pitch, q[k]);
#pragma unroll
            for (int k = 0; k < 4; k++)
                if (k0 + k < a.splits)
#pragma unroll
                    for (int e = 0; e < 8; e++) v[e] += __uint_as_float(q[k][e]);
        }
        *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(a.dhidden) + t * a.dhidden_stride + d) = narrow8_scaled<DT>(v, undo);
    }
}

namespace {

constexpr size_t kWindowBytes = (size_t)256 << 20;  // of G
constexpr size_t kPairs = 76;                       // pairs of SMs on a GB300: sizes the workspace, not the grid

// cuTensorMapEncodeTiled, from the driver that the runtime has loaded.
using EncodeTiled = decltype(&cuTensorMapEncodeTiled);
EncodeTiled encode_tiled() {
    static const EncodeTiled fn = [] {
        void *p = nullptr;
        cudaDriverEntryPointQueryResult found;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &found) != cudaSuccess ||
            found != cudaDriverEntryPointSuccess) {
            cudaGetLastError();
            p = nullptr;
        }
        return (EncodeTiled)p;
    }();
    return fn;
}

// A map of a rows x cols matrix of 16-bit elements, boxes of box_rows x 64; what lies
// beyond the matrix reads as zero.
bool make_map(CUtensorMap *m, int dtype, const void *ptr, long long rows, long long cols, long long stride, int box_rows) {
    const EncodeTiled encode = encode_tiled();
    if (!encode) return false;
    if (rows == 1) stride = cols;  // (no distance to a next row: any value is accepted)
    const cuuint64_t dims[2] = {(cuuint64_t)cols, (cuuint64_t)rows}, strides[1] = {(cuuint64_t)stride * 2};
    const cuuint32_t box[2] = {64, (cuuint32_t)box_rows}, steps[2] = {1, 1};
    return encode(m, dtype == DT_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 2,
                  const_cast<void *>(ptr), dims, strides, box, steps, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                  CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int MODE, int DT>
cudaError_t launch_tiles(const rar_ctx *h, const XentArgs &k, const XentMaps &maps, int b0, int nb, cudaStream_t stream) {
    auto kern = xent_tile_kernel<MODE, DT>;
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kTcSmem);
    if (e != cudaSuccess) return e;
    const int pairs = std::min(xent_items<MODE>(k, nb), h->sm_count / 2);
    return launch_pdl(kern, dim3((unsigned)(2 * pairs)), dim3(kTcThreads), kTcSmem, stream, k, maps, b0, nb);
}

void plan_blocks(size_t vocab, int p, XentArgs *k) {
    k->base = (int)(vocab / p);
    k->extra = (int)(vocab % p);
    k->nb_big = (k->base + 1 + kBlock - 1) / kBlock;
    k->nb_small = (k->base + kBlock - 1) / kBlock;
    k->n_blocks = k->extra * k->nb_big + (p - k->extra) * k->nb_small;
}

size_t plan(void *base, size_t tokens, size_t dim, size_t vocab, int p, bool grad, XentArgs *k) {
    WorkspacePlan w(base);
    plan_blocks(vocab, p, k);
    const size_t n_blocks = (size_t)k->n_blocks;
    k->stats = w.take<float2>(2 * n_blocks * tokens);
    k->z_target = w.take<float>(tokens);
    k->w_max = w.take<unsigned>(1);
    k->window = 0;
    if (grad) {
        k->lse_ws = w.take<float>(tokens);
        k->row_weight = w.take<float>(tokens);
        k->hidden_used = w.take<uint16_t>(tokens * dim);
        size_t window = kWindowBytes / (sizeof(uint16_t) * kBlock * std::max<size_t>(tokens, 1));
        window = std::min(std::max<size_t>(window, 1), n_blocks);
        k->window = (int)window;
        k->g = w.take<uint16_t>(tokens * window * kBlock);
        // few tiles: dhidden's sum over the window is split until there are
        // about two tiles a pair of SMs
        const size_t tiles = ((tokens + kTile - 1) / kTile) * ((dim + kTile - 1) / kTile);
        const size_t splits = std::min(std::max<size_t>(2 * kPairs / std::max<size_t>(tiles, 1), 1), window);
        k->splits = (int)splits;
        k->direct = splits == 1;
        k->dh_part = w.take<float>(window < n_blocks || splits > 1 ? splits * tokens * dim : 0);
    }
    return w.used;
}

bool sizes_ok(size_t tokens, size_t dim, size_t vocab, int p) {
    return p >= 1 && p <= kInlineP && dim >= 1 && vocab >= 1 && vocab <= 0x7FFFFF00u &&
           dim % 8 == 0 && dim <= 0x7FFFFF00u && tokens <= 0x7FFFFF00u &&
           // tiles and steps are counted in 32 bits
           (tokens / kTile + 1) * (vocab / kBlock + p + 1) < 0x7FFFFFFFu && (dim / kTile + 1) * (vocab / kBlock + p + 1) < 0x7FFFFFFFu &&
           (tokens / kTile + 1) * (dim / kTile + 1) < 0x3FFFFFFFu;
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

    k.limits = {h->status, op_timeout_ns(h), op_muted_rank(h)};

    XentMaps logits, dh, dw;  // of the products that use them
    bool mapped = true;
    if (k.tokens) {
        mapped = make_map(&logits.one, a->dtype, k.hidden, k.tokens, k.dim, k.hidden_stride, 128);
        for (int r = 0; r < k.p && mapped; r++) {
            const long long rows = k.base + (r < k.extra ? 1 : 0);
            const int short_of = r == k.limits.mute ? 1 : 0;  // a box without its last row completes no stage
            if (rows) mapped = make_map(&logits.w[r], a->dtype, k.w.inl[r], rows, k.dim, k.weight_stride, 128 - short_of);
            if (rows && mapped && k.dhidden) mapped = make_map(&dh.w[r], a->dtype, k.w.inl[r], rows, k.dim, k.weight_stride, 64 - short_of);
        }
        const long long pitch = (long long)k.window * kBlock;
        if (k.dhidden) mapped = mapped && make_map(&dh.one, a->dtype, k.g, k.tokens, pitch, pitch, 128);
        if (k.want_dw)
            mapped = mapped && make_map(&dw.one, a->dtype, k.g, k.tokens, pitch, pitch, 64) &&
                     make_map(&dw.w[0], a->dtype, k.hidden_used, k.tokens, k.dim, k.dim, 64);
    }
    if (!mapped) return fail(h, RAR_ECUDA, "rar_vocab_xent: the driver refused a tensor map");

    auto run = [&](auto dt) {
        constexpr int DT = decltype(dt)::value;
        cudaError_t e = cudaSuccess;
        if (!k.tokens) {  // no tokens: the pieces' gradients are zeros
            for (int r = 0; r < k.p && e == cudaSuccess; r++) {
                const size_t rows = (size_t)(k.base + (r < k.extra ? 1 : 0));
                if (rows) e = cudaMemset2DAsync(k.dw.inl[r], (size_t)k.dweight_stride * 2, 0, (size_t)k.dim * 2, rows, stream);
            }
            return e;
        }
        const bool sums = k.dim > 64 * kStepsPerSum;
        e = sums ? launch_tiles<XENT_STATS_SUMS, DT>(h, k, logits, 0, k.n_blocks, stream)
                 : launch_tiles<XENT_STATS, DT>(h, k, logits, 0, k.n_blocks, stream);
        const int join = grad ? kJoinTokens<true> : kJoinTokens<false>;
        if (e == cudaSuccess)
            e = launch_pdl(grad ? xent_join_kernel<DT, true> : xent_join_kernel<DT, false>, dim3((unsigned)((k.tokens + join - 1) / join)), dim3(32 * join), 0, stream, k);
        if (!grad) return e;
        for (int b0 = 0; b0 < k.n_blocks && e == cudaSuccess; b0 += k.window) {
            const int nb = std::min(k.window, k.n_blocks - b0);
            e = sums ? launch_tiles<XENT_G_SUMS, DT>(h, k, logits, b0, nb, stream) : launch_tiles<XENT_G, DT>(h, k, logits, b0, nb, stream);
            if (e == cudaSuccess && k.dhidden) {
                XentArgs kw = k;
                kw.splits = std::min(k.splits, nb);
                e = launch_tiles<XENT_DHIDDEN, DT>(h, kw, dh, b0, nb, stream);
            }
            if (e == cudaSuccess && k.want_dw) e = launch_tiles<XENT_DWEIGHT, DT>(h, k, dw, b0, nb, stream);
        }
        if (e == cudaSuccess && k.dhidden && k.splits > 1) {
            const long long n = k.tokens * (k.dim / 8);
            const unsigned grid = (unsigned)std::min<long long>((n + 255) / 256, h->sm_count * 8);
            e = launch_pdl(xent_dhidden_join_kernel<DT>, dim3(grid), dim3(256), 0, stream, k);
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

// vocab_tiles.cuh -- the matrix products between hidden states and a vocabulary
// in p pieces, as tiles of a pair of CTAs on the tensor cores (tc_gemm.cuh): logits
// and what their epilogues make of them (statistics, the logits' gradient G), and
// the products of G with the pieces and with the hidden states.  Used by
// vocab_xent.cu and vocab_logprobs.cu.
//
// The vocabulary is walked in blocks of kBlock rows, none of which crosses a piece.
#pragma once

#include <algorithm>

#include "op_host.h"
#include "tc_gemm.cuh"

namespace rar {

constexpr int kBlock = 256;  // vocabulary rows of a block: a tile's columns
constexpr int kTile = 256;   // rows and columns of a tile

struct VocabArgs {
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
    // log probabilities
    float scale;               // of the logits (cross entropy: 1)
    const float *dlogprob, *dentropy, *lse_in, *entropy_in;
    // blocks
    int base, extra;       // chunk_bounds(vocab, p)
    int nb_big, nb_small;  // blocks of a piece of base + 1 / base rows
    int n_blocks;
    // workspace
    float2 *stats;        // [2 n_blocks][tokens]: a half block's max, sum of exp(z - max)
    float *z_target;      // [tokens]
    float *lse_ws;        // [tokens]
    float *row_weight;    // [tokens] token_weight (log probabilities: dlogprob), 0 where left out
    float *row_entropy;   // [tokens] dentropy, 0 where left out
    unsigned *w_max;      // bits of the largest finite |token_weight|, or bound on a token's G
    void *hidden_used;    // [tokens][dim]: hidden, zeros where left out
    void *g;              // [tokens][window * kBlock]
    float *dh_part;       // [splits][tokens][dim]
    int window;           // blocks of a window
    int splits;           // of dhidden's sum over a window
    long long pair;       // not 0: row t + pair of G is what rounding left of row t, for rows of `pair` tokens
    bool direct;          // one split: the last window writes dhidden itself
    // log probabilities: sums and alternatives of each row of tiles' pairs, by half a block's columns
    int width;                    // rows of tiles that are worked on at a time
    int pairs;                    // of the launch
    int stages;                   // of the ring
    int top;
    float4 *sums;                 // [2 slots][tokens]: max, S, U (see LogitSums)
    unsigned long long *lists;    // [2 slots][top][tokens]: keys, in no order
    uint32_t *bars;               // [tokens]: the largest least logit (as in a key) of a full list so far, or NULL
    WaitLimits limits;
};

// Tensor maps of a launch: `one` is the operand that is one matrix (hidden or G),
// `w` the pieces of W, or hidden as TILES_DWEIGHT's second operand.  Boxes are 64
// elements of 128 rows where K runs along the rows, else of 64.
struct VocabMaps {
    CUtensorMap one, w[kInlineP];
};

struct BlockOf {
    int piece;
    int row;    // first row in the piece
    int rows;   // 1 .. kBlock
    int first;  // its index in the vocabulary
};
__device__ __forceinline__ BlockOf block_of(const VocabArgs &a, int b) {
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
__device__ __forceinline__ int g_exponent(const VocabArgs &a) {
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
__device__ __forceinline__ float g_unit(const VocabArgs &a) {
    const float m = __uint_as_float(*a.w_max);
    return m > 0.0f ? ldexpf(m, -ilogbf(m)) : 1.0f;
}
// Both, of a token's weights.  (The power of two is a normal number, so the product is rounded as
// ldexp's result.)
struct GScale {
    float unit, power;
    __device__ __forceinline__ float scaled(float w) const { return w / unit * power; }
};
template <int DT>
__device__ __forceinline__ GScale g_scale(const VocabArgs &a) {
    return {g_unit(a), ldexpf(1.0f, g_exponent<DT>(a))};
}
// What undoes both, and brings in the logits' scale.
template <int DT>
__device__ __forceinline__ float g_undo(const VocabArgs &a) {
    return ldexpf(g_unit(a) * a.scale, -g_exponent<DT>(a));
}

// What a tile is: statistics of logits (for the cross entropy), G of the cross entropy, the
// products with G, sums and alternatives of logits (for log probabilities), G of log
// probabilities.  (_SUMS: see kStepsPerSum)
enum TileMode {
    TILES_STATS, TILES_G, TILES_DHIDDEN, TILES_DWEIGHT, TILES_STATS_SUMS, TILES_G_SUMS,
    TILES_LOGPROB, TILES_LOGPROB_SUMS, TILES_LOGPROB_G, TILES_LOGPROB_G_SUMS
};
template <int MODE>
struct Mode {
    static constexpr bool sums = MODE == TILES_STATS_SUMS || MODE == TILES_G_SUMS || MODE == TILES_LOGPROB_SUMS || MODE == TILES_LOGPROB_G_SUMS;
    static constexpr bool stats = MODE == TILES_STATS || MODE == TILES_STATS_SUMS;
    // a pair stays with one row of tiles while it walks the vocabulary, and keeps sums and alternatives meanwhile
    static constexpr bool resident = MODE == TILES_LOGPROB || MODE == TILES_LOGPROB_SUMS, logprob = MODE == TILES_LOGPROB_G || MODE == TILES_LOGPROB_G_SUMS;
    static constexpr bool g = MODE == TILES_G || MODE == TILES_G_SUMS || logprob, logits = stats || g || resident;
    // whether a row of the operand is a row of K (MN-major); rows of a box; boxes of a stage
    static constexpr bool a_mn = MODE == TILES_DWEIGHT, b_mn = MODE == TILES_DHIDDEN || MODE == TILES_DWEIGHT;
    static constexpr int a_box = a_mn ? 64 : 128, b_box = b_mn ? 64 : 128;
    static constexpr int a_boxes = 128 / a_box, b_boxes = 128 / b_box;
};

// One tile of a pair of CTAs: its place, and its range along K.
struct TileItem {
    int row;     // first row of the tile (token, row of the window's blocks, or 0)
    int col;     // first column (of dim, or 0)
    int n;       // columns that the product covers, a multiple of 32
    int block;   // block of the window (not TILES_DHIDDEN)
    int split;
    int k0, k1;  // TILES_DHIDDEN: blocks of the window; else steps of 64
    int slot;          // resident: the pair's place among those of its row of tiles
    bool begins, ends; // resident: its first tile of this row, its last
};

__host__ __device__ inline int tiles_of(long long n) { return (int)((n + kTile - 1) / kTile); }
__device__ __forceinline__ int round32(int n) { return n >= kTile ? kTile : (n + 31) / 32 * 32; }

// Tiles in an order in which those that run at one time share operands:
// columns of 8 tiles, so that 76 pairs work on about 8 x 9 tiles.
template <int MODE>
__device__ __forceinline__ TileItem tile_item(const VocabArgs &a, int b0, int nb, int i) {
    TileItem o;
    o.split = 0;
    o.block = 0;
    o.col = 0;
    o.k0 = 0;
    const unsigned tb = (unsigned)tiles_of(a.tokens), db = (unsigned)tiles_of(a.dim);
    const unsigned rows = MODE == TILES_DWEIGHT ? (unsigned)nb : tb;
    const unsigned cols = MODE == TILES_DHIDDEN ? db * (unsigned)a.splits : MODE == TILES_DWEIGHT ? db : (unsigned)nb;
    const unsigned g = (unsigned)i / (8 * cols), in = (unsigned)i - g * 8 * cols;
    const unsigned width = min(rows - g * 8, 8u), c = in / width;
    const int r = (int)(g * 8 + in - c * width);
    o.row = r * kTile;
    if (Mode<MODE>::logits) {
        o.block = (int)c;
        o.n = round32(block_of(a, b0 + (int)c).rows);
        o.k1 = (int)((a.dim + 63) / 64);
    } else if (MODE == TILES_DHIDDEN) {
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
__host__ __device__ inline int tile_items(const VocabArgs &a, int nb) {
    const int tb = tiles_of(a.tokens), db = tiles_of(a.dim);
    return MODE == TILES_DHIDDEN ? tb * db * a.splits : MODE == TILES_DWEIGHT ? nb * db : tb * nb;
}

// Pairs that work on each of `w` rows of tiles at a time.
__host__ __device__ inline int pairs_a_row(int pairs, int w) { return pairs / w; }
// Calls f for the tiles of this pair until it returns false.
template <int MODE, typename F>
__device__ __forceinline__ void tile_walk(const VocabArgs &a, int b0, int nb, F &&f) {
    const int pairs = gridDim.x / 2, first = blockIdx.x / 2;
    if constexpr (!Mode<MODE>::resident) {
        const int items = tile_items<MODE>(a, nb);
        for (int i = first; i < items; i += pairs)
            if (!f(tile_item<MODE>(a, b0, nb, i))) return;
    } else {
        const int tb = tiles_of(a.tokens);
        TileItem o{};
        o.k1 = (int)((a.dim + 63) / 64);
        int next = 0;
        for (int r0 = 0; r0 < tb; r0 += a.width) {
            const int w = min(a.width, tb - r0), share = pairs_a_row(pairs, w), slot = first / w, turn = next % share;
            next = (turn + nb) % share;  // the blocks that are left over go to other pairs the next time
            if (slot >= share) continue;
            o.row = (r0 + first % w) * kTile;
            o.slot = slot + turn < share ? slot + turn : slot + turn - share;
            o.begins = true;
            for (int b = o.slot; b < nb; b += share) {
                o.block = b;
                o.n = round32(block_of(a, b0 + b).rows);
                o.ends = b + share >= nb;
                if (!f(o)) return;
                o.begins = false;
            }
        }
    }
}

// Calls f for every step of 64 along K: f(step within the block or the
// range, block of the window, the block).  Stops when f returns false.
template <int MODE, typename F>
__device__ __forceinline__ bool tile_steps(const VocabArgs &a, int b0, const TileItem &it, F &&f) {
    if constexpr (MODE == TILES_DHIDDEN) {
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
// a long forward pass (2048 tokens by 50021 x 2048 fp16 314 us against 282 when it came in, 285 now; 8192 by
// 65536 x 4096 bf16 2.54 ms against 2.33), 3 to 4 % with gradients.  A dim of one sum keeps the plain form
// and its time.  Products whose results are rounded to 16 bits do without.
constexpr int kStepsPerSum = 16;

// Values in the order of their logits, equal ones from the lowest token on: the larger key first.
// 0 is no value; NaN and -inf have none.
__device__ __forceinline__ unsigned long long top_key(float z, uint32_t token) {
    const uint32_t b = __float_as_uint(z + 0.0f);  // (no -0)
    return (unsigned long long)(b & 0x80000000u ? ~b : b | 0x80000000u) << 32 | (uint32_t)~token;
}
__device__ __forceinline__ float top_value(unsigned long long key) {
    const uint32_t b = (uint32_t)(key >> 32);
    return __uint_as_float(b & 0x80000000u ? b ^ 0x80000000u : ~b);
}
__device__ __forceinline__ uint32_t top_token(unsigned long long key) { return ~(uint32_t)key; }

// exp(scale x) for k = scale log2(e); good to (2 + |scale x|) 2^-23 (see exp_of).
__device__ __forceinline__ float exp_scaled(float x, float k) {
    float r;
    asm("ex2.approx.f32 %0, %1;" : "=f"(r) : "f"(x * k));
    return r;
}

// max, S and U of some logits, S and U relative to the maximum.
struct LogitSums {
    float max = -INFINITY, s = 0.0f, u = 0.0f;
    // moves the maximum up to `top`
    __device__ __forceinline__ void raise(float top, float k) {
        const float d = fmaxf(max - top, -1e30f), f = exp_scaled(d, k);  // (from -inf: s and u are 0)
        u = f * fmaf(d, s, u);
        s *= f;
        max = top;
    }
    // z[n], of which those that are not there are -inf
    template <int N>
    __device__ __forceinline__ void add(const float (&z)[N], float k) {
        float most = z[0];
#pragma unroll
        for (int i = 1; i < N; i++) most = fmaxf(most, z[i]);
        add(z, k, most);
    }
    // the same where their maximum is known
    template <int N>
    __device__ __forceinline__ void add(const float (&z)[N], float k, float most) {
        const float top = fmaxf(max, most);
        if (top > max) raise(top, k);
        const float ref = top == -INFINITY ? 0.0f : top;  // nothing but -inf, or NaN, which s then shows
        // two logits an instruction, and two sums
        float s2[2] = {s, 0.0f}, u2[2] = {u, 0.0f};
#pragma unroll
        for (int i = 0; i < N; i += 2) {
            float d[2] = {z[i], z[i + 1]}, x[2], e[2];
            asm("{\n\t.reg .b64 a, b;\n\tmov.b64 a, {%0, %1};\n\tmov.b64 b, {%4, %4};\n\tadd.rn.f32x2 a, a, b;\n\tmov.b64 {%0, %1}, a;\n\t"
                "mov.b64 b, {%5, %5};\n\tmul.rn.f32x2 a, a, b;\n\tmov.b64 {%2, %3}, a;\n\t}"
                : "+f"(d[0]), "+f"(d[1]), "=f"(x[0]), "=f"(x[1])
                : "f"(-ref), "f"(k));
#pragma unroll
            for (int j = 0; j < 2; j++) {
                asm("ex2.approx.f32 %0, %1;" : "=f"(e[j]) : "f"(x[j]));
                d[j] = fmaxf(d[j], -1e30f);  // (-inf: 0 to be added)
            }
            asm("{\n\t.reg .b64 a, b, c;\n\tmov.b64 a, {%4, %5};\n\tmov.b64 c, {%0, %1};\n\tadd.rn.f32x2 c, c, a;\n\tmov.b64 {%0, %1}, c;\n\t"
                "mov.b64 b, {%6, %7};\n\tmov.b64 c, {%2, %3};\n\tfma.rn.f32x2 c, a, b, c;\n\tmov.b64 {%2, %3}, c;\n\t}"
                : "+f"(s2[0]), "+f"(s2[1]), "+f"(u2[0]), "+f"(u2[1])
                : "f"(e[0]), "f"(e[1]), "f"(d[0]), "f"(d[1]));
        }
        s = s2[0] + s2[1];
        u = u2[0] + u2[1];
    }
    __device__ __forceinline__ void join(float om, float os, float ou, float k) {
        if (os == 0.0f) return;  // nothing there
        LogitSums o{om, os, ou};
        const float top = fmaxf(max, om);
        if (top != -INFINITY) {
            raise(top, k);
            o.raise(top, k);
        }
        s += o.s;
        u += o.u;
    }
    // over all lanes, with the same bits in each: first to one maximum, then the sums
    __device__ __forceinline__ void join_lanes(float k) {
        float top = max;
#pragma unroll
        for (int d = 16; d; d /= 2) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, d));
        if (top != -INFINITY) raise(top, k);
#pragma unroll
        for (int d = 16; d; d /= 2) {
            s += __shfl_xor_sync(0xFFFFFFFFu, s, d);
            u += __shfl_xor_sync(0xFFFFFFFFu, u, d);
        }
    }
};

// Maxima of groups of 4 columns (-infinity where all four are NaN: a group without a logit bounds nothing).
__device__ __forceinline__ void group_maxima(const float (&v)[32], float (&m)[8]) {
#pragma unroll
    for (int i = 0; i < 8; i++) m[i] = fmaxf(fmaxf(fmaxf(v[4 * i], v[4 * i + 1]), fmaxf(v[4 * i + 2], v[4 * i + 3])), -INFINITY);
}
// In falling order (Batcher's odd-even merges: runs of P into runs of 2 P, by steps of K = P, P / 2, .. 1).
// (Template arguments: with loop variables in their place x would lie in memory.)
template <int P = 1, int K = P>
__device__ __forceinline__ void sort_falling(float (&x)[32]) {
#pragma unroll
    for (int n = 0; n < 32; n++) {
        constexpr int kFirst = K % P;
        const bool leads = n >= kFirst && (n - kFirst) % (2 * K) < K && n + K < 32 && n / (2 * P) == (n + K) / (2 * P);
        if (leads) {
            const float hi = fmaxf(x[n], x[n + K < 32 ? n + K : n]);
            x[n + K < 32 ? n + K : n] = fminf(x[n], x[n + K < 32 ? n + K : n]);
            x[n] = hi;
        }
    }
    if constexpr (K > 1) sort_falling<P, K / 2>(x);
    else if constexpr (P < 16) sort_falling<2 * P>(x);
}

// The `top` largest keys that a thread has seen, in shared memory: place i of thread t at
// [i][t], so that a warp's accesses meet no bank twice.  Each thread first notes the columns
// that may belong into its list; when one has noted many, and at the end of a tile, all insert theirs
// side by side, so that a step of a warp serves all of its rows (column by column, with a step for each
// column that any of 32 rows wants, there would be several times as many).  A new key takes
// the place of the least one; which is the least then is known from the 8 places around and the other
// groups' least, in registers.  In a row's first tile the bound is the `top`-th largest of the maxima of 32
// groups of columns.  (2048 tokens by 50021 x 2048 fp16 back to back: 320 us with 8 alternatives; alone 276 us
// without, 301 with 1, 332 with 8 and some 420 with 32; with the least of as many groups' maxima for a bound 78 us
// more with 32, with a look at all places for each key twice the time.)
struct TileTop {
    static constexpr int kNoted = 24, kRow = 32 * kTcEpilogueWarps, kGroups = RAR_LOGPROBS_MAX_TOP / 8;
    static constexpr int kNotedBytes = kNoted * kRow * 5;
    uint32_t noted, column, list;       // shared-memory addresses: logits and columns noted, keys
    uint32_t next;                      // where the next logit is noted
    unsigned long long group[kGroups];  // least keys of 8 places each
    unsigned long long least;           // of all: 0 until the list is full
    uint32_t at;                        // its place, in bits 0 to 7; that of group g in bits 8 + 3 g and on
    __device__ __forceinline__ TileTop(uint32_t addr)
        : noted(addr + threadIdx.x * 4), column(addr + kNoted * kRow * 4 + threadIdx.x), list(addr + kNotedBytes + threadIdx.x * 8), next(noted) {}
    static __device__ __forceinline__ unsigned long long load(uint32_t addr) {
        unsigned long long x;
        asm volatile("ld.shared.u64 %0, [%1];" : "=l"(x) : "r"(addr));
        return x;
    }
    static __device__ __forceinline__ void store(uint32_t addr, unsigned long long x) { asm volatile("st.shared.u64 [%0], %1;" ::"r"(addr), "l"(x) : "memory"); }
    // places beyond `top` hold what is never the least
    __device__ __forceinline__ void clear(int top) {
        const int places = (top + 7) / 8 * 8;
        for (int i = 0; i < places; i++) store(list + i * kRow * 8, i < top ? 0ull : ~0ull);
#pragma unroll
        for (int g = 0; g < kGroups; g++) group[g] = g * 8 < top ? 0ull : ~0ull;
        least = 0;
        at = 0;
    }
    __device__ __forceinline__ unsigned long long get(int i) const { return load(list + i * kRow * 8); }
    __device__ __forceinline__ void insert(unsigned long long x) {
        if (x <= least) return;
        const uint32_t place = at & 0xFFu, g = place / 8;
        store(list + place * kRow * 8, x);
        unsigned long long y[8];
#pragma unroll
        for (int i = 0; i < 8; i++) y[i] = load(list + (g * 8 + i) * kRow * 8);
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; i++) {
            w[i] = y[2 * i + 1] < y[2 * i] ? 2 * i + 1 : 2 * i;
            y[i] = y[2 * i + 1] < y[2 * i] ? y[2 * i + 1] : y[2 * i];
        }
        w[0] = y[1] < y[0] ? w[1] : w[0], y[0] = y[1] < y[0] ? y[1] : y[0];
        w[2] = y[3] < y[2] ? w[3] : w[2], y[2] = y[3] < y[2] ? y[3] : y[2];
        w[0] = y[2] < y[0] ? w[2] : w[0], y[0] = y[2] < y[0] ? y[2] : y[0];
        at = (at & ~(7u << (8 + 3 * g)) & ~0xFFu) | w[0] << (8 + 3 * g);
        uint32_t worst = 0;
#pragma unroll
        for (int i = 0; i < kGroups; i++) {
            group[i] = g == i ? y[0] : group[i];
            if (i == 0 || group[i] < least) least = group[i], worst = i;
        }
        at |= worst * 8 + (at >> (8 + 3 * worst) & 7u);
    }
    // The first tile of a row: maxima of its groups of columns c0 .. c0 + 31, before the list is there, and the
    // `top`-th largest of them all, which so many logits are not below.
    // (They lie where this thread's logits are noted, and the last ones in its list's first places: no
    // other thread's, which may be at another row.)
    __device__ __forceinline__ uint32_t maximum_at(int i) const {
        return i < kNoted ? noted + i * kRow * 4 : list + (i - kNoted) / 2 * kRow * 8 + (i - kNoted) % 2 * 4;
    }
    static_assert(kNoted % 8 == 0 && kNoted + 16 >= 32, "8 places of a list take what the noted ones leave");
    __device__ __forceinline__ void keep_maxima(const float (&m)[8], int c0) {
#pragma unroll
        for (int i = 0; i < 8; i++) asm volatile("st.shared.f32 [%0], %1;" ::"r"(maximum_at(c0 / 4 + i)), "f"(m[i]) : "memory");
    }
    __device__ __forceinline__ float bound_of_maxima(int top) const {
        float x[32], b = -INFINITY;
#pragma unroll
        for (int i = 0; i < 32; i++) asm volatile("ld.shared.f32 %0, [%1];" : "=f"(x[i]) : "r"(maximum_at(i)));
        sort_falling(x);
#pragma unroll
        for (int i = 0; i < 32; i++)  // (in this form x stays in registers)
            asm("{\n\t.reg .pred P;\n\tsetp.eq.s32 P, %1, %2;\n\tselp.f32 %0, %3, %0, P;\n\t}" : "+f"(b) : "r"(top - 1), "r"(i), "f"(x[i]));
        return b;
    }
    // what has to be passed to get into the list
    __device__ __forceinline__ float bar() const { return least ? top_value(least) : -INFINITY; }
    // columns c0 .. c0 + 31 of a row whose first is `first`, of which those up to `bound` are not wanted (infinity: none is)
    __device__ __forceinline__ void add(const float (&v)[32], float bound, int c0, uint32_t first) {
#pragma unroll
        for (int h = 0; h < 32; h += 16) {
            const float over = fmaxf(bar(), bound);
            uint32_t where = column + (next - noted) / 4;
#pragma unroll
            for (int c = h; c < h + 16; c++)
                asm volatile("{\n\t.reg .pred P;\n\tsetp.gt.f32 P, %2, %3;\n\t@P st.shared.f32 [%0], %2;\n\t@P st.shared.u8 [%1], %6;\n\t"
                             "@P add.u32 %0, %0, %4;\n\t@P add.u32 %1, %1, %5;\n\t}"
                             : "+r"(next), "+r"(where)
                             : "f"(v[c]), "f"(over), "n"(kRow * 4), "n"(kRow), "r"(c0 + c)
                             : "memory");
            if (__any_sync(0xFFFFFFFFu, next > noted + (kNoted - 16) * kRow * 4)) insert_noted(first);
        }
    }
    __device__ __forceinline__ void insert_noted(uint32_t first) {
        const int n = (int)(next - noted) / (kRow * 4), steps = __reduce_max_sync(0xFFFFFFFFu, n);
#pragma unroll 1
        for (int i = 0; i < steps; i++)
            if (i < n) {
                float x;
                uint32_t c;
                asm volatile("ld.shared.f32 %0, [%1];" : "=f"(x) : "r"(noted + i * kRow * 4));
                asm volatile("ld.shared.u8 %0, [%1];" : "=r"(c) : "r"(column + i * kRow));
                insert(top_key(x, first + c));
            }
        next = noted;
    }
};

// What an epilogue thread keeps of a tile: one row of it.
struct TileRow {
    int row;          // of tokens (or of the block, TILES_DWEIGHT)
    bool live;        // the row exists
    int cols;         // columns of its half that exist
    int target;       // column of its target in its half, or one out of range
    float w, lse;     // logits for G
    float w_log;      // G of log probabilities: p (w + w_log log p) + w_target at the target
    float w_target;
    bool used;        // the token has a part in the gradients
    bool rest;        // what rounding leaves of another row of G (see VocabArgs::pair)
    float max, sum;   // logits for the statistics
    int first;        // the vocabulary's row of the half's first column
    char *out;        // where the row's half begins
    float *part;      // TILES_DHIDDEN: the sums so far
};

template <int MODE, int DT>
__device__ __forceinline__ TileRow tile_row(const VocabArgs &a, const GScale &g, int b0, const TileItem &it, int row, int half) {
    TileRow r;
    r.row = row;
    r.out = nullptr;
    r.part = nullptr;
    if constexpr (MODE == TILES_DHIDDEN) {
        r.live = row < a.tokens;
        r.cols = (int)a.dim - it.col - half;
        r.out = static_cast<char *>(a.dhidden) + (row * a.dhidden_stride + it.col + half) * 2;
        r.part = a.dh_part + ((long long)it.split * a.tokens + row) * a.dim + it.col + half;
    } else if constexpr (MODE == TILES_DWEIGHT) {
        const BlockOf b = block_of(a, b0 + it.block);
        r.row = row - it.row;
        r.live = r.row < b.rows;
        r.cols = (int)a.dim - it.col - half;
        r.out = rank_ptr(a.dw, a.p, b.piece) + ((long long)(b.row + r.row) * a.dweight_stride + it.col + half) * 2;
    } else {
        const BlockOf b = block_of(a, b0 + it.block);
        r.live = row < a.tokens;
        r.rest = false;
        if constexpr (Mode<MODE>::logprob)
            if (a.pair && row >= a.pair) r.rest = true, row -= (int)a.pair;
        r.cols = b.rows - half;
        const long long y = r.live ? load_index(a.targets, a.index_bytes, row) - b.first - half : -1;
        r.target = y >= 0 && y < r.cols ? (int)y : -1;
        r.max = -INFINITY;
        r.sum = 0.0f;
        r.first = b.first + half;
        if constexpr (Mode<MODE>::logprob) {
            const float da = r.live ? g.scaled(a.row_weight[row]) : 0.0f, db = r.live ? g.scaled(a.row_entropy[row]) : 0.0f;
            r.used = da != 0.0f || db != 0.0f;
            r.w = -da - (db != 0.0f ? db * a.entropy_in[row] : 0.0f);
            r.w_log = -db;
            r.w_target = da;
            r.lse = r.used ? a.lse_in[row] : 0.0f;
        } else if constexpr (Mode<MODE>::g) {
            r.w = r.live ? g.scaled(a.row_weight[row]) : 0.0f;
            r.lse = r.live ? a.lse_ws[row] : 0.0f;
        }
        if constexpr (Mode<MODE>::g) r.out = static_cast<char *>(a.g) + (((long long)r.row * a.window + it.block) * kBlock + half) * 2;
    }
    return r;
}

// Columns beyond the block's last.
__device__ __forceinline__ void mask_columns(float (&v)[32], int cols) {
    if (cols >= 32) return;
#pragma unroll
    for (int c = 0; c < 32; c++) v[c] = c < cols ? v[c] : -INFINITY;
}
__device__ __forceinline__ void keep_target(const VocabArgs &a, const TileRow &r, int c0, const float (&v)[32]) {
    const int y = r.target - c0;
    if (y < 0 || y >= 32) return;
    float z = 0.0f;
#pragma unroll
    for (int c = 0; c < 32; c++)  // (in this form v stays in registers)
        asm("{\n\t.reg .pred P;\n\tsetp.eq.s32 P, %1, %2;\n\tselp.f32 %0, %3, %0, P;\n\t}" : "+f"(z) : "r"(y), "r"(c), "f"(v[c]));
    a.z_target[r.row] = z;
}

// Columns c0 .. c0 + 31 of the row's half.
template <int MODE, int DT>
__device__ __forceinline__ void tile_columns(const VocabArgs &a, TileRow &r, int c0, float undo, bool first, bool direct, float (&v)[32]) {
    if (!r.live) return;
    const int cols = r.cols - c0;
    if constexpr (Mode<MODE>::stats) {
        if (cols <= 0) return;
        mask_columns(v, cols);
        keep_target(a, r, c0, v);
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
            if constexpr (Mode<MODE>::logprob) {
                // (every step for every column: one that is made on a condition becomes a branch.  Below -128 p is
                // 0 in 32 bits, and so is p log p: for a logit of -infinity, too, where 0 x infinity would be NaN.
                // p has the log probability as it is, so that NaN stays NaN.)
                const float logp = fmaf(v[c], a.scale, -r.lse), w = fmaf(r.w_log, fmaxf(logp, -128.0f), r.w), p = exp_of(logp);
                const float x = fmaf(p, w, c == y ? r.w_target : 0.0f);
                v[c] = c < cols && r.used ? x : 0.0f;
            } else {
                const float p = exp_of(v[c] - r.lse) - (c == y ? 1.0f : 0.0f);
                v[c] = c < cols && r.w != 0.0f ? p * r.w : 0.0f;
            }
        }
        if constexpr (Mode<MODE>::logprob)
            if (r.rest)
#pragma unroll
                for (int c = 0; c < 32; c++) v[c] -= widen<DT>(narrow<DT>(v[c]));
#pragma unroll
        for (int c = 0; c < 32; c += 16) {
            const uint4 x = narrow8<DT>(v + c), y4 = narrow8<DT>(v + c + 8);
            const uint32_t q[8] = {x.x, x.y, x.z, x.w, y4.x, y4.y, y4.z, y4.w};
            store_32b(r.out + (c0 + c) * 2, q);
        }
    } else if constexpr (MODE == TILES_DHIDDEN) {
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
// room for a warp of 32, so that a CTA of the join can wait there for the end.  (Where the logits come as sums of 1024,
// whose 128 registers live beside an epilogue's own, log probabilities spill 224 bytes a thread so, their G 56.)
template <int MODE, int DT>
__global__ void __cluster_dims__(2, 1, 1) __maxnreg__(152)
    vocab_tile_kernel(const __grid_constant__ VocabArgs a, const __grid_constant__ VocabMaps maps, int b0, int nb) {
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
    const uint32_t ring = Mode<MODE>::resident ? (uint32_t)a.stages : kTcStages;
    constexpr bool a_mn = Mode<MODE>::a_mn, b_mn = Mode<MODE>::b_mn;
    constexpr int kABoxes = Mode<MODE>::a_boxes, kLoaders = kABoxes + Mode<MODE>::b_boxes;
    if (warp == kTcEpilogueWarps && lane < kLoaders) {
        // a lane a box, first those of A
        constexpr unsigned kLanes = (1u << kLoaders) - 1;
        const bool is_a = lane < kABoxes;
        const int part = is_a ? lane * Mode<MODE>::a_box : (lane - kABoxes) * Mode<MODE>::b_box;  // rows (columns) into the operand
        unsigned step = 0;
        uint32_t st = 0, phase = 0;
        tile_walk<MODE>(a, b0, nb, [&](const TileItem &it) {
            if (__any_sync(kLanes, *(volatile int *)&sh.failed)) return false;
            tile_steps<MODE>(a, b0, it, [&](int s, int k, const BlockOf &b) {
                // (a new barrier's preceding phase counts as complete: the first turn does not wait)
                if (!__all_sync(kLanes, tc_wait(&sh, a.limits, &sh.empty[st], phase ^ 1, 0))) return false;
                // a CTA whose rows of A all lie past the last loads none of them: its
                // rows of the accumulator are never read
                auto a_rows = [&](int r) { return MODE == TILES_DWEIGHT || it.row + r * 128 < a.tokens; };
                if (rank == 0 && lane == 0)
                    mbar_expect_tx(&sh.full[st], 32768u + 16384u * (1u + a_rows(1)));
                const uint32_t bar = peer_addr(smem_u32(&sh.full[st]), 0);
                const uint32_t to = stages + st * kTcStageBytes + (is_a ? 0 : 16384) + part * 128;
                const CUtensorMap *map = is_a ? &maps.one : &maps.w[MODE == TILES_DWEIGHT ? 0 : b.piece];
                const int row = it.row + (int)rank * 128 + part, col = it.col + (int)rank * it.n / 2 + part;
                int x, y;
                if (MODE == TILES_DHIDDEN) x = is_a ? k * kBlock + s * 64 : col, y = is_a ? row : b.row + s * 64;
                else if (MODE == TILES_DWEIGHT) x = is_a ? row : col, y = s * 64;
                else x = s * 64, y = is_a ? row : b.row + col;
                if (!is_a || a_rows((int)rank)) tc_load_box(map, to, bar, x, y);
                step++;
                if (++st == ring) st = 0, phase ^= 1;
                return true;
            });
            return true;
        });
        // neither CTA may leave while the pair's loads, products or arrivals are under way,
        // nor give its tensor memory back, even after a wait that ran out: products in flight
        // belong to the last stages, whose `empty` they arrive at in both CTAs
        for (unsigned k = step > ring ? step - ring : 0; k < step && lane == 0; k++) {
            const int st = (int)(k % ring);
            if (rank == 0 && !mbar_drain(&sh.full[st], (k / ring) & 1)) break;
            if (!mbar_drain(&sh.empty[st], (k / ring) & 1)) break;
        }
    } else if (warp == kTcEpilogueWarps + 1 && lane == 0 && rank == 0) {
        const uint64_t operand_a = tc_operand(stages, a_mn ? 8192 : 16, 1024), operand_b = tc_operand(stages + 16384, b_mn ? 8192 : 16, 1024);
        // the next stage and its phase; accumulators begun.  (This thread issues a step of 64
        // every 512 cycles or so: what it computes between two steps is time lost.)
        uint32_t st = 0, phase = 0, sums = 0;
        tile_walk<MODE>(a, b0, nb, [&](const TileItem &it) {
            const uint32_t idesc = tc_instruction(DT == DT_BF16, a_mn, b_mn, (uint32_t)it.n);
            uint32_t d = 0;
            int left = 0;  // steps that the present accumulator takes yet
            bool more = false;
            const bool ok = tile_steps<MODE>(a, b0, it, [&](int, int, const BlockOf &) {
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
                if (++st == ring) st = 0, phase ^= 1;
                left--;
                return true;
            });
            if (ok) tc_commit(&sh.acc_full[(sums - 1) & 1]);
            return ok;
        });
    } else if (warp < kTcEpilogueWarps) {
        const int quarter = warp % 4;
        const float undo = MODE == TILES_DHIDDEN || MODE == TILES_DWEIGHT ? g_undo<DT>(a) : 1.0f;
        GScale g;
        if constexpr (Mode<MODE>::g) g = g_scale<DT>(a);
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
        [[maybe_unused]] LogitSums own;
        [[maybe_unused]] TileTop top(stages + ring * kTcStageBytes);
        tile_walk<MODE>(a, b0, nb, [&](const TileItem &it) {
            bool ok = true;
            const int half = warp / 4 * 128, row = it.row + (int)rank * 128 + quarter * 32 + lane;
            TileRow r = tile_row<MODE, DT>(a, g, b0, it, row, half);
            [[maybe_unused]] uint32_t seen = 0;
            if constexpr (Mode<MODE>::resident)
                if (a.bars && r.live) seen = *(volatile const uint32_t *)(a.bars + row);
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
                if (!ok || !ready()) return false;
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
            } else if (!ready()) {
                return false;
            }
            [[maybe_unused]] float most = -INFINITY;
            if constexpr (Mode<MODE>::resident) {
                if (it.begins) own = LogitSums();
                if (it.begins && r.cols < 128 && a.top > 1) {  // (columns that the block does not have)
                    const float none[8] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY, -INFINITY, -INFINITY, -INFINITY, -INFINITY};
                    for (int c0 = 0; c0 < 128; c0 += 32) top.keep_maxima(none, c0);
                }
            }
#pragma unroll 1
            for (int c0 = 0; c0 < 128; c0 += 32) {
                float v[32];
                tc_read32(at(c0), v);
                tc_read_wait();
                if constexpr (Mode<MODE>::resident) {
                    if (r.cols - c0 <= 0) break;  // (the same for the whole warp)
                    mask_columns(v, r.cols - c0);
                    keep_target(a, r, c0, v);
                    float m[8], here = -INFINITY;
                    group_maxima(v, m);
#pragma unroll
                    for (int i = 0; i < 8; i++) here = fmaxf(here, m[i]);
                    own.add(v, a.scale * 1.4426950408889634f, here);
                    most = fmaxf(most, here);
                    if (it.begins && a.top > 1) top.keep_maxima(m, c0);
                } else {
                    tile_columns<MODE, DT>(a, r, c0, undo, first_window, direct, v);
                }
            }
            if constexpr (Mode<MODE>::resident) {
                // A second look, where a row of the warp has a column for its list.  What lies below
                // `top` logits of this tile, or of those that another pair has, is not wanted; what equals the least
                // of them may have the lower token.  (When a bar is seen decides what is noted, not what comes out.)
                float bound = -INFINITY;
                if (a.top && it.begins) {
                    bound = a.top == 1 ? most : top.bound_of_maxima(a.top);
                    top.clear(a.top);
                    if (a.bars && r.live && bound > -INFINITY) {
                        const uint32_t bar = (uint32_t)(top_key(bound, 0) >> 32);
                        if (bar > seen) atomicMax(a.bars + row, bar);
                        seen = *(volatile const uint32_t *)(a.bars + row);
                    }
                    bound = nextafterf(bound, -INFINITY);
                }
                // (a bar of 0 has the key of -0 below it, which is no less)
                if (seen) bound = fmaxf(bound, top_value((unsigned long long)(seen - (seen == 0x80000000u ? 2 : 1)) << 32));
                if (!r.live) bound = INFINITY;
                if (a.top && __any_sync(0xFFFFFFFFu, most > fmaxf(top.bar(), bound))) {
                    const unsigned long long least = top.least;
#pragma unroll 1
                    for (int c0 = 0; c0 < 128; c0 += 32) {
                        if (r.cols - c0 <= 0) break;
                        float v[32];
                        tc_read32(at(c0), v);
                        tc_read_wait();
                        mask_columns(v, r.cols - c0);
                        top.add(v, bound, c0, (uint32_t)r.first);
                    }
                    top.insert_noted((uint32_t)r.first);
                    if (a.bars && r.live && top.least > least && (uint32_t)(top.least >> 32) > seen) atomicMax(a.bars + row, (uint32_t)(top.least >> 32));
                }
            }
            release();
            if constexpr (Mode<MODE>::stats)
                if (r.live) a.stats[(2ll * (b0 + it.block) + half / 128) * a.tokens + row] = make_float2(r.max, r.sum);
            if constexpr (Mode<MODE>::resident)
                if (it.ends && r.live) {
                    const long long list = 2ll * it.slot + half / 128;
                    a.sums[list * a.tokens + row] = make_float4(own.max, own.s, own.u, 0.0f);
                    for (int i = 0; i < a.top; i++) a.lists[(list * a.top + i) * a.tokens + row] = top.get(i);
                }
            return true;
        });
    }
    __syncwarp();
    tc_end(&sh);
}

// dhidden from the splits' sums, and the paired rows'.
template <int DT>
__global__ void __launch_bounds__(256) vocab_dhidden_join_kernel(const __grid_constant__ VocabArgs a) {
    pdl_wait();
    pdl_launch_dependents();
    const float undo = g_undo<DT>(a);
    const long long vecs = a.dim / 8, n = (a.pair ? a.pair : a.tokens) * vecs, pitch = a.tokens * a.dim, half = a.pair * a.dim;
    const int parts = a.pair ? 2 * a.splits : a.splits;  // (those of a pair one after the other)
    for (long long i = (long long)blockIdx.x * blockDim.x + threadIdx.x; i < n; i += (long long)gridDim.x * blockDim.x) {
        const long long t = n < 0x7FFFFFFF ? (long long)((uint32_t)i / (uint32_t)vecs) : i / vecs, d = (i - t * vecs) * 8;
        const float *part = a.dh_part + t * a.dim + d;
        float v[8] = {};
        for (int k0 = 0; k0 < parts; k0 += 4) {
            uint32_t q[4][8];  // loads in flight together
#pragma unroll
            for (int k = 0; k < 4; k++) {
                const int j = min(k0 + k, parts - 1);
                load_32b(part + (a.pair ? (j / 2) * pitch + (j % 2) * half : j * pitch), q[k]);
            }
#pragma unroll
            for (int k = 0; k < 4; k++)
                if (k0 + k < parts)
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

// Shared memory of the alternatives' lists.
constexpr int list_bytes(int top) { return top ? (top + 7) / 8 * 8 * TileTop::kRow * 8 + TileTop::kNotedBytes : 0; }
// Stages that fit beside them (2048 tokens by 50021 x 2048 fp16 take the same time with 4 to 7).
constexpr int stages_beside(int top) { return (kTcSmem - 1024 - list_bytes(top)) / kTcStageBytes; }
static_assert(stages_beside(RAR_LOGPROBS_MAX_TOP) >= 4 && stages_beside(0) == kTcStages, "the lists leave four stages");

template <int MODE, int DT>
cudaError_t launch_tiles(const rar_ctx *h, const VocabArgs &k, const VocabMaps &maps, int b0, int nb, cudaStream_t stream) {
    auto kern = vocab_tile_kernel<MODE, DT>;
    const int pairs = Mode<MODE>::resident ? k.pairs : std::min(tile_items<MODE>(k, nb), h->sm_count / 2);
    const int smem = Mode<MODE>::resident ? k.stages * kTcStageBytes + 1024 + list_bytes(k.top) : kTcSmem;
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kTcSmem);
    if (e != cudaSuccess) return e;
    return launch_pdl(kern, dim3((unsigned)(2 * pairs)), dim3(kTcThreads), (size_t)smem, stream, k, maps, b0, nb);
}

void plan_blocks(size_t vocab, int p, VocabArgs *k) {
    k->base = (int)(vocab / p);
    k->extra = (int)(vocab % p);
    k->nb_big = (k->base + 1 + kBlock - 1) / kBlock;
    k->nb_small = (k->base + kBlock - 1) / kBlock;
    k->n_blocks = k->extra * k->nb_big + (p - k->extra) * k->nb_small;
}

// The gradients' share of a workspace: G for a window of blocks, and dhidden's sums.  tokens: rows of G.
// rounds: tiles a pair of SMs that dhidden's sum is split into.
void plan_grad(WorkspacePlan &w, size_t tokens, size_t dim, size_t rounds, VocabArgs *k) {
    const size_t n_blocks = (size_t)k->n_blocks;
    k->hidden_used = w.take<uint16_t>(tokens * dim);
    size_t window = kWindowBytes / (sizeof(uint16_t) * kBlock * std::max<size_t>(tokens, 1));
    window = std::min(std::max<size_t>(window, 1), n_blocks);
    k->window = (int)window;
    k->g = w.take<uint16_t>(tokens * window * kBlock);
    // few tiles: dhidden's sum over the window is split until there are
    // about so many
    const size_t tiles = ((tokens + kTile - 1) / kTile) * ((dim + kTile - 1) / kTile);
    const size_t splits = std::min(std::max<size_t>(rounds * kPairs / std::max<size_t>(tiles, 1), 1), window);
    k->splits = (int)splits;
    k->direct = splits == 1 && !k->pair;
    k->dh_part = w.take<float>(window < n_blocks || !k->direct ? splits * tokens * dim : 0);
}

// The maps of a call: of the logits' products, dhidden's and dweights'.
struct CallMaps {
    VocabMaps logits, dh, dw;
};
bool make_maps(int dtype, const VocabArgs &k, CallMaps *m) {
    bool mapped = make_map(&m->logits.one, dtype, k.hidden, k.tokens, k.dim, k.hidden_stride, 128);
    for (int r = 0; r < k.p && mapped; r++) {
        const long long rows = k.base + (r < k.extra ? 1 : 0);
        const int short_of = r == k.limits.mute ? 1 : 0;  // a box without its last row completes no stage
        if (rows) mapped = make_map(&m->logits.w[r], dtype, k.w.inl[r], rows, k.dim, k.weight_stride, 128 - short_of);
        if (rows && mapped && k.dhidden) mapped = make_map(&m->dh.w[r], dtype, k.w.inl[r], rows, k.dim, k.weight_stride, 64 - short_of);
    }
    const long long pitch = (long long)k.window * kBlock;
    if (k.dhidden) mapped = mapped && make_map(&m->dh.one, dtype, k.g, k.tokens, pitch, pitch, 128);
    if (k.want_dw)
        mapped = mapped && make_map(&m->dw.one, dtype, k.g, k.tokens, pitch, pitch, 64) &&
                 make_map(&m->dw.w[0], dtype, k.hidden_used, k.tokens, k.dim, k.dim, 64);
    return mapped;
}

// Zeros in the pieces' gradients: those of no tokens.
cudaError_t clear_dweights(const VocabArgs &k, cudaStream_t stream) {
    cudaError_t e = cudaSuccess;
    for (int r = 0; r < k.p && e == cudaSuccess; r++) {
        const size_t rows = (size_t)(k.base + (r < k.extra ? 1 : 0));
        if (rows) e = cudaMemset2DAsync(k.dw.inl[r], (size_t)k.dweight_stride * 2, 0, (size_t)k.dim * 2, rows, stream);
    }
    return e;
}

// Both gradients, a window of blocks at a time.  G: how its tiles are made.
template <int G, int DT>
cudaError_t launch_gradients(const rar_ctx *h, const VocabArgs &k, const CallMaps &m, cudaStream_t stream) {
    cudaError_t e = cudaSuccess;
    for (int b0 = 0; b0 < k.n_blocks && e == cudaSuccess; b0 += k.window) {
        const int nb = std::min(k.window, k.n_blocks - b0);
        e = launch_tiles<G, DT>(h, k, m.logits, b0, nb, stream);
        if (e == cudaSuccess && k.dhidden) {
            VocabArgs kw = k;
            kw.splits = std::min(k.splits, nb);
            e = launch_tiles<TILES_DHIDDEN, DT>(h, kw, m.dh, b0, nb, stream);
        }
        if (e == cudaSuccess && k.want_dw) e = launch_tiles<TILES_DWEIGHT, DT>(h, k, m.dw, b0, nb, stream);
    }
    if (e == cudaSuccess && k.dhidden && !k.direct) {
        const long long n = (k.pair ? k.pair : k.tokens) * (k.dim / 8);
        const unsigned grid = (unsigned)std::min<long long>((n + 255) / 256, h->sm_count * 8);
        e = launch_pdl(vocab_dhidden_join_kernel<DT>, dim3(grid), dim3(256), 0, stream, k);
    }
    return e;
}

bool sizes_ok(size_t tokens, size_t dim, size_t vocab, int p) {
    return p >= 1 && p <= kInlineP && dim >= 1 && vocab >= 1 && vocab <= 0x7FFFFF00u &&
           dim % 8 == 0 && dim <= 0x7FFFFF00u && tokens <= 0x7FFFFF00u &&
           // tiles and steps are counted in 32 bits
           (tokens / kTile + 1) * (vocab / kBlock + p + 1) < 0x7FFFFFFFu && (dim / kTile + 1) * (vocab / kBlock + p + 1) < 0x7FFFFFFFu &&
           (tokens / kTile + 1) * (dim / kTile + 1) < 0x3FFFFFFFu;
}

}  // namespace
}  // namespace rar

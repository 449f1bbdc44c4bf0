// vocab_logprobs.cu -- log probabilities of given tokens, entropy and the most likely
// alternatives over a vocabulary in p pieces, from the hidden states
// (rar_vocab_logprobs), and their gradients (rar_vocab_logprobs_grad).
//
//   z = hidden W^T,  l = scale z,  m = max z,  S = sum exp(scale (z - m)),  U = sum exp(scale (z - m)) (z - m)
//   lse = scale m + log S,  logprob = scale (z[target] - m) - log S,  entropy = log S - scale U / S
//
// (in this form nothing large cancels: S is at least 1 and U at most 0).  The gradient
// for z, from those of the log probability, a, and of the entropy, b:
//
//   G = scale (a onehot(target) - p (a + b (log p + entropy))),  p = exp(l - lse)
//   dhidden = G W,  dweights = G^T hidden
//
// which takes lse and the entropy as the forward pass gave them, so that the logits are
// made once: 6 tokens x vocab x dim operations in all.
//
// Two forms of the forward pass, by what bounds it:
//   up to 128 tokens (stream_fits), memory: the pieces are streamed once (vocab_stream.cuh), the logits go
//     through L2 to a cluster of CTAs a token.  16 tokens by 65536 x 4096 bf16: 85 us for 537 MB (6.3 TB/s), 99 us
//     with the selection of 5 alternatives; 1 by 32768 x 2048: 26 us, 34 with 20.  By tiles 64 tokens by 32768 x
//     2048 took 75 us with 8 alternatives, here 54 with 5; 128 by 4096 x 50021, whose accumulators leave room for one
//     tile of rows at a time, took longer here than by tiles (160 us for the logits alone; by tiles 65 to 128 tokens by
//     65536 x 4096 take 112 in all), so that is left to them.
//   above, the tensor cores: tiles whose epilogues keep sums and alternatives (vocab_tiles.cuh), joined by token.  8192
//     by 65536 x 4096 bf16 2.46 ms (1.79 PFLOP/s at the power limit), 2048 by 50021 x 2048 fp16 276 us, with 8
//     alternatives 320: then the epilogues of a row's first tiles, whose lists fill, outlast the products.
// Gradients: 8192 by 65536 x 4096 bf16 7.7 ms (1.72 PFLOP/s at the power limit); 333 by 10007 x 520 fp16 59 us, the latency
// of six launches.
#include <cmath>

#include "vocab_stream.cuh"

namespace rar {

// The largest keys seen by a warp, one a lane in falling order; `least` is the one at `top`.
// (Short code, and called, not repeated: these kernels run for a few microseconds, in which
// instructions that are fetched for the first time show.)
struct TopList {
    unsigned long long key = 0, least = 0;
};
// runs of n keys in a bitonic order, into falling order (rising ones where lane & n)
__device__ __forceinline__ unsigned long long top_fall(unsigned long long x, int n) {
    const int lane = threadIdx.x % 32;
#pragma unroll 1
    for (int d = n / 2; d; d /= 2) {
        const unsigned long long y = __shfl_xor_sync(0xFFFFFFFFu, x, d);
        const bool first = ((lane & d) == 0) == ((lane & n) == 0);
        x = first == (x > y) ? x : y;
    }
    return x;
}
// in falling order (Batcher's bitonic sort)
__device__ __noinline__ unsigned long long top_sorted(unsigned long long x) {
#pragma unroll 1
    for (int n = 2; n <= 32; n *= 2) x = top_fall(x, n);
    return x;
}
// The 32 largest of two lists: of two falling runs, one turned round, the larger ones of each
// place, which are in a bitonic order.
__device__ __noinline__ unsigned long long top_merged(unsigned long long key, unsigned long long other) {
    const unsigned long long x = __shfl_sync(0xFFFFFFFFu, other, 31 - threadIdx.x % 32);
    return top_fall(key > x ? key : x, 32);
}
// takes the lanes' keys; 0 where a lane has none
__device__ __noinline__ TopList top_add(TopList list, unsigned long long x, int top) {
    const int lane = threadIdx.x % 32;
    unsigned more = __ballot_sync(0xFFFFFFFFu, x > list.least);
    if (__popc(more) > 6) {  // sorted and merged, 20 steps: as much as inserting six
        x = top_sorted(x);
        list.key = __any_sync(0xFFFFFFFFu, list.key) ? top_merged(list.key, x) : x;
        list.least = __shfl_sync(0xFFFFFFFFu, list.key, top - 1);
        return list;
    }
#pragma unroll 1
    for (; more; more &= more - 1) {
        const unsigned long long y = __shfl_sync(0xFFFFFFFFu, x, __ffs(more) - 1);
        if (y <= list.least) continue;
        const int at = __popc(__ballot_sync(0xFFFFFFFFu, list.key > y));
        const unsigned long long before = __shfl_up_sync(0xFFFFFFFFu, list.key, 1);
        list.key = lane < at ? list.key : lane == at ? y : before;
        list.least = __shfl_sync(0xFFFFFFFFu, list.key, top - 1);
    }
    return list;
}
// The lanes' values, no NaN among them, in falling order (as top_sorted).
__device__ __noinline__ float falling(float x) {
    const int lane = threadIdx.x % 32;
#pragma unroll 1
    for (int n = 2; n <= 32; n *= 2)
#pragma unroll 1
        for (int d = n / 2; d; d /= 2) {
            const float y = __shfl_xor_sync(0xFFFFFFFFu, x, d);
            x = ((lane & d) == 0) == ((lane & n) == 0) ? fmaxf(x, y) : fminf(x, y);
        }
    return x;
}
// takes the keys noted in shared memory
__device__ __noinline__ TopList top_add_noted(TopList list, const unsigned long long *noted, int n, int top) {
    __syncwarp();
#pragma unroll 1
    for (int i0 = 0; i0 < n; i0 += 32) {
        const int i = i0 + threadIdx.x % 32;
        list = top_add(list, i < n ? noted[i] : 0ull, top);
    }
    __syncwarp();
    return list;
}

// Where a call's results go.
struct LogprobOut {
    long long vocab;
    float scale;
    int top;
    const void *targets;
    int index_bytes;
    float *logprob, *entropy, *lse;
    float *top_logprob;
    long long *top_token;
};
// Those of one token, by a warp with the same sums in every lane.
__device__ __forceinline__ void write_token(const LogprobOut &o, long long t, const LogitSums &sums, float z_target, unsigned long long key) {
    const int lane = threadIdx.x % 32;
    const float log_s = logf(sums.s);
    if (lane == 0) {
        const long long y = load_index(o.targets, o.index_bytes, t);
        if (o.logprob) o.logprob[t] = y >= 0 && y < o.vocab ? fmaf(o.scale, z_target - sums.max, -log_s) : 0.0f;
        if (o.entropy) o.entropy[t] = log_s - o.scale * __fdiv_rn(sums.u, sums.s);
        if (o.lse) o.lse[t] = fmaf(o.scale, sums.max, log_s);
    }
    if (lane < o.top) {
        if (top_token(key) >= o.vocab) key = 0;  // (after a wait that ran out nothing is certain but this)
        o.top_token[t * o.top + lane] = key ? (long long)top_token(key) : -1ll;
        o.top_logprob[t * o.top + lane] = key ? fmaf(o.scale, top_value(key) - sums.max, -log_s) : -INFINITY;
    }
}

struct SelectArgs {
    LogprobOut out;
    const float *logits;  // [tokens][pitch], 16-byte aligned rows
    long long pitch;
};

// Warps of a CTA, CTAs of a token at most.
constexpr int kSelectWarps = 4, kSelectCluster = 8, kSelectNoted = 256;

// Everything about a token from its logits, for few tokens: a cluster of CTAs a token, each with a range
// of the vocabulary, whose warps keep sums and a list of their own.  AHEAD: 16-byte loads that a lane has in flight.  A
// round of these loads costs a sort whatever it brings, so there is one round where 16 loads suffice for the
// range: a whole call for 16 tokens by 65536 x 4096 bf16 with 5 alternatives took 101 us so, 107 in rounds of 4
// with 8 warps.  Where fewer do, fewer: the others' instructions are executed, too.
template <int AHEAD>
__global__ void __launch_bounds__(32 * kSelectWarps) logprob_select_kernel(const __grid_constant__ SelectArgs a) {
    __shared__ unsigned long long lists[kSelectWarps][32], noted[kSelectWarps][kSelectNoted];
    __shared__ float3 sums[kSelectWarps];
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, top = a.out.top;
    const uint32_t rank = cluster_rank(), ctas = gridDim.x;
    const long long t = blockIdx.y;
    const float k = a.out.scale * 1.4426950408889634f;
    pdl_wait();
    pdl_launch_dependents();
    const float *row = a.logits + t * a.pitch;
    const uint32_t vocab = (uint32_t)a.out.vocab, vecs = (vocab + 3) / 4;
    const uint32_t v0 = (uint32_t)((unsigned long long)vecs * rank / ctas), v1 = (uint32_t)((unsigned long long)vecs * (rank + 1) / ctas);
    LogitSums own;
    TopList list;
    for (uint32_t v = v0 + warp * 32; v < v1; v += 32 * kSelectWarps * AHEAD) {
        float z[4 * AHEAD];
        const uint32_t at = v + lane;
#pragma unroll
        for (int u = 0; u < AHEAD; u++) {  // loads in flight together
            float4 q = make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);
            if (at + u * 32 * kSelectWarps < v1) q = __ldcg(reinterpret_cast<const float4 *>(row) + at + u * 32 * kSelectWarps);
            z[4 * u] = q.x, z[4 * u + 1] = q.y, z[4 * u + 2] = q.z, z[4 * u + 3] = q.w;
        }
        auto token = [&](int i) { return (at + (i / 4) * 32 * kSelectWarps) * 4 + i % 4; };
#pragma unroll
        for (int i = 0; i < 4 * AHEAD; i++)
            if (token(i) >= vocab) z[i] = -INFINITY;  // (behind the row's last)
        own.add(z, k);
        if (!top) continue;
        // each lane's best: of these in falling order, what is below the one at `top` is not among the `top` largest
        float best = z[0];
#pragma unroll
        for (int i = 1; i < 4 * AHEAD; i++) best = fmaxf(best, z[i]);
        const float full = list.least ? top_value(list.least) : -INFINITY;
        if (!__any_sync(0xFFFFFFFFu, best >= full)) continue;
        const float bar = list.least ? full : __shfl_sync(0xFFFFFFFFu, falling(fmaxf(best, -INFINITY)), top - 1);
        int n = 0;  // noted so far
#pragma unroll
        for (int i = 0; i < 4 * AHEAD; i++) {
            const bool wanted = z[i] >= bar && z[i] > -INFINITY;
            const unsigned who = __ballot_sync(0xFFFFFFFFu, wanted);
            if (wanted) noted[warp][n + __popc(who & ((1u << lane) - 1))] = top_key(z[i], token(i));
            n += __popc(who);
            if (i % 4 == 3 && n > kSelectNoted - 4 * 32) {  // (seldom: far fewer are above the bar, unless they rise along the row)
                list = top_add_noted(list, noted[warp], n, top);
                n = 0;
            }
        }
        list = top_add_noted(list, noted[warp], n, top);
    }
    own.join_lanes(k);
    lists[warp][lane] = list.key;
    if (lane == 0) sums[warp] = make_float3(own.max, own.s, own.u);
    // the CTA's, and then the cluster's, in warp 0 of its first CTA
    auto join = [&](int n) {
        for (int d = 1; d < n; d *= 2) {
            __syncthreads();
            if (top && warp % (2 * d) == 0 && warp + d < n) {
                list.key = top_merged(list.key, lists[warp + d][lane]);
                lists[warp][lane] = list.key;
            }
        }
        __syncthreads();
        if (warp == 0) {
            own = LogitSums();
            if (lane < n) own.join(sums[lane].x, sums[lane].y, sums[lane].z, k);
            own.join_lanes(k);
        }
    };
    join(kSelectWarps);
    if (ctas > 1) {
        if (warp == 0 && lane == 0) sums[0] = make_float3(own.max, own.s, own.u);
        cluster_sync_all();
        list.key = 0;
        own = LogitSums();
        for (int c = warp; c < (int)ctas && rank == 0; c += kSelectWarps) {
            const uint32_t at = peer_addr(smem_u32(&lists[0][lane]), (uint32_t)c), st = peer_addr(smem_u32(&sums[0]), (uint32_t)c);
            unsigned long long x;
            float m, e, u;
            asm volatile("ld.shared::cluster.u64 %0, [%1];" : "=l"(x) : "r"(at) : "memory");
            asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(m) : "r"(st) : "memory");
            asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(e) : "r"(st + 4) : "memory");
            asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(u) : "r"(st + 8) : "memory");
            list.key = c == warp ? x : top_merged(list.key, x);
            own.join(m, e, u, k);
        }
        cluster_sync_all();  // all of it is read: the others may end, and this one may write
        if (rank) return;
        lists[warp][lane] = list.key;
        if (lane == 0) sums[warp] = make_float3(own.max, own.s, own.u);
        join(min((int)ctas, kSelectWarps));
    }
    if (warp == 0) {
        const long long y = load_index(a.out.targets, a.out.index_bytes, t);
        write_token(a.out, t, own, y >= 0 && y < a.out.vocab ? __ldcg(row + y) : 0.0f, list.key);
    }
}

// Results from the pairs' sums and alternatives.  SHARED: by a CTA of warps a token, for few tokens
// (which have the longer lists), else by a warp a token.
constexpr int kJoinWarps = 4, kJoinAhead = 10;
template <bool SHARED>
__global__ void __launch_bounds__(32 * kJoinWarps) logprob_join_kernel(const __grid_constant__ VocabArgs a, const __grid_constant__ LogprobOut o) {
    constexpr int kWarps = SHARED ? kJoinWarps : 1;
    __shared__ unsigned long long found[kJoinWarps][32], noted[kJoinWarps][32 * kJoinAhead];
    pdl_wait();
    pdl_launch_dependents();
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32, part = SHARED ? warp : 0;
    const long long t = SHARED ? (long long)blockIdx.x : (long long)blockIdx.x * kJoinWarps + warp;
    if (t >= a.tokens) return;
    const float k = a.scale * 1.4426950408889634f;
    const int tb = tiles_of(a.tokens), r0 = (int)(t / kTile) / a.width * a.width;
    const int lists = 2 * min(pairs_a_row(a.pairs, min(a.width, tb - r0)), a.n_blocks);
    LogitSums own;
    float z = 0.0f;
    if (part == 0) {
        const long long y = load_index(o.targets, o.index_bytes, t);
        z = y >= 0 && y < a.vocab ? a.z_target[t] : 0.0f;
        for (int i = lane; i < lists; i += 32) {
            const float4 q = __ldcg(a.sums + (long long)i * a.tokens + t);
            own.join(q.x, q.y, q.z, k);
        }
    }
    TopList list;
    const int n = lists * a.top;
    for (int i0 = part * 32; i0 < n; i0 += 32 * kWarps * kJoinAhead) {
        unsigned long long x[kJoinAhead], best = 0;
#pragma unroll
        for (int u = 0; u < kJoinAhead; u++) {  // loads in flight together
            const int i = i0 + u * 32 * kWarps + lane;
            x[u] = i < n ? __ldcg(a.lists + (long long)i * a.tokens + t) : 0ull;
        }
#pragma unroll
        for (int u = 0; u < kJoinAhead; u++) best = x[u] > best ? x[u] : best;
        if (!__any_sync(0xFFFFFFFFu, best > list.least)) continue;
        // (see logprob_select_kernel)
        const unsigned long long bound = list.least ? list.least : __shfl_sync(0xFFFFFFFFu, top_sorted(best), a.top - 1);
        int m = 0;  // noted so far
#pragma unroll
        for (int u = 0; u < kJoinAhead; u++) {
            const bool wanted = x[u] >= bound && x[u];
            const unsigned who = __ballot_sync(0xFFFFFFFFu, wanted);
            if (wanted) noted[warp][m + __popc(who & ((1u << lane) - 1))] = x[u];
            m += __popc(who);
        }
        list = top_add_noted(list, noted[warp], m, a.top);
    }
    if (SHARED && a.top) {
        found[warp][lane] = list.key;
        __syncthreads();
        if (warp == 0)
            for (int w = 1; w < kWarps; w++) list.key = top_merged(list.key, found[w][lane]);
    }
    if (part) return;
    own.join_lanes(k);
    write_token(o, t, own, z, list.key);
}

// Of each token: its weights in G (none where its target is left out), the largest bound on an
// entry of its row of G, and its hidden state, cleared where it has no part in the gradients
// (0 x NaN is not 0 in dweights' sum).  A warp a token.
constexpr int kPrepareTokens = 8;
__global__ void __launch_bounds__(32 * kPrepareTokens) logprob_prepare_kernel(const __grid_constant__ VocabArgs a) {
    pdl_wait();
    pdl_launch_dependents();
    const int lane = threadIdx.x % 32;
    const long long t = (long long)blockIdx.x * kPrepareTokens + threadIdx.x / 32;
    if (t >= (a.pair ? a.pair : a.tokens)) return;
    const long long y = load_index(a.targets, a.index_bytes, t);
    const bool counts = y >= 0 && y < a.vocab;
    const float da = counts && a.dlogprob ? a.dlogprob[t] : 0.0f, db = counts && a.dentropy ? a.dentropy[t] : 0.0f;
    const bool used = da != 0.0f || db != 0.0f;
    if (lane == 0) {
        a.row_weight[t] = da;
        a.row_entropy[t] = db;
        // |G| <= |a| + |b| max(p |log p|, p entropy)
        const float most = fabsf(da) + (db != 0.0f ? fabsf(db) * fmaxf(1.0f, fabsf(a.entropy_in[t])) : 0.0f);
        if (isfinite(most)) atomicMax(a.w_max, __float_as_uint(most));
    }
    const int vecs = (int)(a.dim / 8);
    const uint4 *from = reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(a.hidden) + t * a.hidden_stride);
    uint4 *to = reinterpret_cast<uint4 *>(static_cast<uint16_t *>(a.hidden_used) + t * a.dim);
    for (int i0 = lane; i0 < vecs; i0 += 32 * 4) {
        uint4 q[4];  // loads in flight together
#pragma unroll
        for (int u = 0; u < 4; u++) q[u] = used ? __ldg(from + min(i0 + u * 32, vecs - 1)) : make_uint4(0, 0, 0, 0);
#pragma unroll
        for (int u = 0; u < 4; u++)
            if (i0 + u * 32 < vecs) {
                to[i0 + u * 32] = q[u];
                if (a.pair) to[a.pair * vecs + i0 + u * 32] = q[u];
            }
    }
}

namespace {

// Tokens for which a CTA joins a token's lists: 256 tokens of one row of tiles have up to 152 lists, 2048
// of 8 rows 38.
constexpr long long kSharedJoin = 1024;
// Tokens of a pass over the pieces: bounds the workspace.
constexpr size_t kPassTokens = 16384;

// Rows of tiles that are worked on at a time: the most that cost little more rounds of tiles than the best
// number (in the last round of a single group of rows a block too few costs as much as one; over several groups
// that evens out).  Each group reads all pieces once and begins its lists anew, so 5 % more rounds are worth fewer
// groups, and 10 % a single one: 2048 tokens by 50021 x 2048 fp16 with 8 alternatives take 325 us with 8 rows in
// 23 rounds, 341 with 6 in 22, 334 with 5 and 331 with 4 in 21; 600 by 50021 x 1024 66 us without any by 3 rows, 76
// row by row; 8192 by 65536 x 4096 bf16 2.28 ms with 5 rows, which is the choice, and with 4 (109 and 108 rounds), 2.30
// with 6 or 8 (113).  (Alternatives have no say: with and without them the sums are the same.)
int choose_width(int tb, int nb, int pairs) {
    auto rounds = [&](int w) {
        const int groups = tb / w, rest = tb % w;
        const double n = groups * (double)nb / pairs_a_row(pairs, w) + (rest ? (double)nb / pairs_a_row(pairs, rest) : 0.0);
        return groups + (rest != 0) == 1 ? std::ceil(n) : n;
    };
    double least = rounds(1);
    for (int w = 2; w <= std::min(tb, 8); w++) least = std::min(least, rounds(w));
    int w = std::min(tb, 8);
    while (rounds(w) > least * (tb <= 8 ? 1.1 : 1.05)) w--;
    return w;
}

size_t plan(void *base, size_t tokens, size_t dim, size_t vocab, int p, int top, VocabArgs *k, float **logits) {
    WorkspacePlan w(base);
    plan_blocks(vocab, p, k);
    *logits = nullptr;
    if (stream_fits(tokens, dim)) {
        *logits = w.take<float>(tokens * stream_pitch(vocab));
        return w.used;
    }
    const size_t pass = std::min(tokens, kPassTokens);
    k->window = (int)pass;
    if (tokens) {
        // (a last pass of fewer tokens has a width of its own, and up to all pairs on a row)
        const int tb = tiles_of((long long)pass), width = choose_width(tb, k->n_blocks, (int)kPairs), rest = tb % width;
        const bool even = tokens % pass == 0;
        const int share = even ? pairs_a_row((int)kPairs, rest ? rest : width) : (int)kPairs;
        const size_t lists = 2 * (size_t)std::min(std::max(share, pairs_a_row((int)kPairs, width)), k->n_blocks);
        k->z_target = w.take<float>(pass);
        k->sums = w.take<float4>(lists * pass);
        k->lists = w.take<unsigned long long>(lists * pass * (size_t)top);
        k->bars = w.take<uint32_t>(top ? pass : 0);
    }
    return w.used;
}
// G is held as two 16-bit rows a token, the second what rounding left of the first, and the products take both, for few
// tokens.  A gradient of few tokens is a sum of few products, in which G's rounding shows as much as the
// gradient's own or, where one entry decides it, up to 2.6 times as much; over many it adds 1.4 times.  A piece has only
// the tokens that aim at it to decide it, so there up to 256 a piece count as few, while the work is little: the second
// rows take 1.2 times the time for 1569 tokens by 854 x 480 (56 and 69 us), 1.5 times for 2048 by 4096 x 1024 (71 and
// 105 us), which goes without.
bool paired(size_t tokens, size_t dim, size_t vocab, int p) {
    return tokens <= 512 || (tokens <= 256 * (size_t)p && (double)tokens * (double)dim * (double)vocab <= 0x1p32);
}
size_t plan_gradients(void *base, size_t tokens, size_t dim, size_t vocab, int p, VocabArgs *k) {
    WorkspacePlan w(base);
    plan_blocks(vocab, p, k);
    k->w_max = w.take<unsigned>(1);
    k->row_weight = w.take<float>(tokens);
    k->row_entropy = w.take<float>(tokens);
    k->pair = paired(tokens, dim, vocab, p) ? (long long)tokens : 0;
    // (one round: 333 tokens by 10007 x 520 63 us, 66 with two, 71 with three)
    plan_grad(w, k->pair ? 2 * tokens : tokens, dim, 1, k);
    return w.used;
}

// What both calls have: sizes, hidden states, pieces, targets.
template <typename Args>
int check_inputs(OpCheck &c, const Args *a) {
    if (!a) return c.bad("args is NULL");
    int rc = c.dtype(a->dtype, false);
    if (rc != RAR_OK) return rc;
    if (a->p < 1 || a->p > kInlineP) return c.bad("p must be in [1, 64]");
    if (a->dim < 1 || a->vocab < 1) return c.bad("dim and vocab must be at least 1");
    if (a->dim % 8) return c.bad("dim must be a multiple of 8");
    if (a->index_bytes != 4 && a->index_bytes != 8) return c.bad("index_bytes must be 4 or 8");
    if (!(a->logit_scale > 0.0f && a->logit_scale <= 0x1p126f)) return c.bad("logit_scale must be positive and at most 2^126");
    if (!sizes_ok(a->tokens, a->dim, a->vocab, a->p)) return c.bad("the sizes are too large");
    MatrixSpan s;
    if ((rc = c.matrix("hidden", a->hidden, a->tokens, a->dim, a->hidden_stride, 2, 16, &s)) != RAR_OK) return rc;
    c.input(s);
    if (!a->weights) return c.bad("weights is NULL");
    for (int r = 0; r < a->p; r++) {
        const size_t rows = a->vocab / a->p + ((size_t)r < a->vocab % a->p ? 1 : 0);
        if ((rc = c.matrix("a weight piece", a->weights[r], rows, a->dim, a->weight_stride, 2, 16, &s)) != RAR_OK) return rc;
        c.input(s);
    }
    const size_t ib = (size_t)a->index_bytes;
    if ((rc = c.matrix("targets", a->targets, 1, a->tokens, 0, ib, ib, &s)) != RAR_OK) return rc;
    c.input(s);
    return RAR_OK;
}
template <typename Args>
void set_inputs(rar_ctx *h, const Args *a, VocabArgs *k) {
    for (int r = 0; r < a->p; r++) k->w.inl[r] = const_cast<void *>(a->weights[r]);
    k->p = a->p;
    k->tokens = (long long)a->tokens;
    k->dim = (long long)a->dim;
    k->vocab = (long long)a->vocab;
    k->hidden_stride = (long long)(a->hidden_stride ? a->hidden_stride : a->dim);
    k->weight_stride = (long long)(a->weight_stride ? a->weight_stride : a->dim);
    k->hidden = a->hidden;
    k->targets = a->targets;
    k->index_bytes = a->index_bytes;
    k->scale = a->logit_scale;
    k->limits = {h->status, op_timeout_ns(h), op_muted_rank(h)};
}
struct Vec { const char *name; const void *ptr; size_t n, eb; };

cudaError_t launch_select(const rar_ctx *h, const SelectArgs &s, int tokens, cudaStream_t stream) {
    // CTAs a token: until there are two an SM, but at least 2048 logits each (with 1024, 90 tokens by 4000 x 512 took 27 us,
    // now 24)
    unsigned ctas = 1;
    while (ctas < kSelectCluster && tokens * (int)ctas < 2 * h->sm_count && s.out.vocab / (2 * ctas) >= 2048) ctas *= 2;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(ctas, (unsigned)tokens);
    cfg.blockDim = dim3(32 * kSelectWarps);
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = ctas;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    const long long range = ((s.out.vocab + 3) / 4 + ctas - 1) / ctas, loads = (range + 32 * kSelectWarps - 1) / (32 * kSelectWarps);
    return cudaLaunchKernelEx(&cfg, loads <= 2 ? logprob_select_kernel<2> : loads <= 4 ? logprob_select_kernel<4> : loads <= 8 ? logprob_select_kernel<8>
                                                                                                        : logprob_select_kernel<16>, s);
}

int vocab_logprobs(rar_ctx *h, const rar_vocab_logprobs_args *a, cudaStream_t stream) {
    OpCheck c(h, "rar_vocab_logprobs");
    int rc = check_inputs(c, a);
    if (rc != RAR_OK) return rc;
    if (a->top < 0 || a->top > RAR_LOGPROBS_MAX_TOP || (size_t)a->top > a->vocab) return c.bad("top must be in [0, RAR_LOGPROBS_MAX_TOP] and at most vocab");
    MatrixSpan s;
    const size_t n = a->tokens, listed = n * (size_t)a->top;
    for (const Vec &v : {Vec{"logprob", a->logprob, n, 4}, Vec{"entropy", a->entropy, n, 4}, Vec{"lse", a->lse, n, 4}})
        if (v.ptr) {
            if ((rc = c.matrix(v.name, v.ptr, 1, v.n, 0, v.eb, v.eb, &s)) != RAR_OK) return rc;
            c.output(s);
        }
    for (const Vec &v : {Vec{"top_logprob", a->top_logprob, listed, 4}, Vec{"top_token", a->top_token, listed, 8}}) {  // (top 0: nothing)
        if ((rc = c.matrix(v.name, v.ptr, 1, v.n, 0, v.eb, v.eb, &s)) != RAR_OK) return rc;
        c.output(s);
    }
    VocabArgs k{};
    float *logits;
    const size_t need = plan(nullptr, a->tokens, a->dim, a->vocab, a->p, a->top, &k, &logits);
    if ((rc = c.workspace(a->workspace, a->workspace_bytes, need)) != RAR_OK) return rc;
    if ((rc = c.overlaps([](const MatrixSpan &, const MatrixSpan &) { return false; })) != RAR_OK) return rc;
    if (a->tokens == 0) return RAR_OK;

    DeviceGuard dg(h->device);
    if (dg.err != cudaSuccess) return cuda_fail(h, dg.err, "selecting the device");
    plan(a->workspace, a->tokens, a->dim, a->vocab, a->p, a->top, &k, &logits);
    set_inputs(h, a, &k);
    note_op_call(h, a->p, stream);

    if (stream_fits(n, a->dim)) {
        StreamArgs st{};
        VocabMaps maps;
        stream_shape(&st, (int)n, k.dim, k.base, k.extra, k.p, h->sm_count);
        st.logits = logits;
        st.pitch = (long long)stream_pitch(a->vocab);
        st.limits = k.limits;
        if (!stream_maps(a->dtype, k, st, &maps)) return fail(h, RAR_ECUDA, "rar_vocab_logprobs: the driver refused a tensor map");
        const SelectArgs sel{{k.vocab, k.scale, a->top, k.targets, k.index_bytes, a->logprob, a->entropy, a->lse, a->top_logprob, a->top_token}, logits, st.pitch};
        cudaError_t e = a->dtype == RAR_BFLOAT16 ? launch_stream<DT_BF16>(h, st, maps, stream) : launch_stream<DT_F16>(h, st, maps, stream);
        if (e == cudaSuccess) e = launch_select(h, sel, (int)n, stream);
        return e == cudaSuccess ? RAR_OK : cuda_fail(h, e, "launching the log probabilities");
    }
    CallMaps m;
    if (!make_maps(a->dtype, k, &m)) return fail(h, RAR_ECUDA, "rar_vocab_logprobs: the driver refused a tensor map");
    auto run = [&](auto dt) {
        constexpr int DT = decltype(dt)::value;
        cudaError_t e = cudaSuccess;
        for (long long t0 = 0; t0 < (long long)n && e == cudaSuccess; t0 += k.window) {
            VocabArgs part = k;
            part.tokens = std::min((long long)n - t0, (long long)k.window);
            part.hidden = static_cast<const uint16_t *>(k.hidden) + t0 * k.hidden_stride;
            part.targets = static_cast<const char *>(k.targets) + t0 * k.index_bytes;
            part.top = a->top;
            part.stages = stages_beside(a->top);
            const int tb = tiles_of(part.tokens);
            part.width = choose_width(tb, k.n_blocks, (int)kPairs);
            part.pairs = std::min(std::min(h->sm_count / 2, (int)kPairs), std::min(tb, part.width) * k.n_blocks);
            // (a pair with one tile of a row has little to learn from the others, who are at theirs: 98 us against 104 for
            // 333 tokens by 10007 x 520 with 32 alternatives, none with 8)
            const bool share = a->top && k.n_blocks > pairs_a_row(part.pairs, std::min(part.width, tb));
            if (!share) part.bars = nullptr;
            else if ((e = cudaMemsetAsync(part.bars, 0, sizeof(uint32_t) * (size_t)part.tokens, stream)) != cudaSuccess) return e;
            if (t0 && !make_map(&m.logits.one, a->dtype, part.hidden, part.tokens, k.dim, k.hidden_stride, 128)) return cudaErrorInvalidValue;
            e = k.dim > 64 * kStepsPerSum ? launch_tiles<TILES_LOGPROB_SUMS, DT>(h, part, m.logits, 0, k.n_blocks, stream)
                                          : launch_tiles<TILES_LOGPROB, DT>(h, part, m.logits, 0, k.n_blocks, stream);
            auto at = [&](float *v) { return v ? v + t0 : nullptr; };
            LogprobOut o{k.vocab, k.scale, a->top, part.targets, k.index_bytes, at(a->logprob), at(a->entropy), at(a->lse), nullptr, nullptr};
            if (a->top) o.top_logprob = a->top_logprob + t0 * a->top, o.top_token = a->top_token + t0 * a->top;
            if (e == cudaSuccess)
                e = part.tokens <= kSharedJoin
                        ? launch_pdl(logprob_join_kernel<true>, dim3((unsigned)part.tokens), dim3(32 * kJoinWarps), 0, stream, part, o)
                        : launch_pdl(logprob_join_kernel<false>, dim3((unsigned)((part.tokens + kJoinWarps - 1) / kJoinWarps)), dim3(32 * kJoinWarps), 0, stream, part, o);
        }
        return e;
    };
    const cudaError_t ce = a->dtype == RAR_BFLOAT16 ? run(IntC<DT_BF16>{}) : run(IntC<DT_F16>{});
    return ce == cudaSuccess ? RAR_OK : cuda_fail(h, ce, "launching the log probabilities");
}

int vocab_logprobs_grad(rar_ctx *h, const rar_vocab_logprobs_grad_args *a, cudaStream_t stream) {
    OpCheck c(h, "rar_vocab_logprobs_grad");
    int rc = check_inputs(c, a);
    if (rc != RAR_OK) return rc;
    MatrixSpan s;
    const size_t n = a->tokens;
    if (n && !a->dlogprob && !a->dentropy) return c.bad("dlogprob and dentropy are NULL");
    const Vec ins[] = {{"lse", a->lse, n, 1}, {"dlogprob", a->dlogprob, n, a->dlogprob != nullptr}, {"dentropy", a->dentropy, n, a->dentropy != nullptr},
                       {"entropy", a->entropy, n, a->dentropy != nullptr}};
    for (const Vec &v : ins)
        if (v.eb) {  // (needed)
            if ((rc = c.matrix(v.name, v.ptr, 1, v.n, 0, 4, 4, &s)) != RAR_OK) return rc;
            c.input(s);
        }
    if (!a->dhidden && !a->dweights) return c.bad("dhidden and dweights are NULL");
    if (a->dhidden) {
        if ((rc = c.matrix("dhidden", a->dhidden, n, a->dim, a->dhidden_stride, 2, 16, &s)) != RAR_OK) return rc;
        c.output(s);
    }
    for (int r = 0; r < a->p && a->dweights; r++) {
        const size_t rows = a->vocab / a->p + ((size_t)r < a->vocab % a->p ? 1 : 0);
        if ((rc = c.matrix("a dweight piece", a->dweights[r], rows, a->dim, a->dweight_stride, 2, 16, &s)) != RAR_OK) return rc;
        c.output(s);
    }
    VocabArgs k{};
    const size_t need = plan_gradients(nullptr, n, a->dim, a->vocab, a->p, &k);
    if ((rc = c.workspace(a->workspace, a->workspace_bytes, need)) != RAR_OK) return rc;
    if ((rc = c.overlaps([](const MatrixSpan &, const MatrixSpan &) { return false; })) != RAR_OK) return rc;
    if (n == 0 && !a->dweights) return RAR_OK;

    DeviceGuard dg(h->device);
    if (dg.err != cudaSuccess) return cuda_fail(h, dg.err, "selecting the device");
    plan_gradients(a->workspace, n, a->dim, a->vocab, a->p, &k);
    set_inputs(h, a, &k);
    for (int r = 0; r < a->p; r++) k.dw.inl[r] = a->dweights ? a->dweights[r] : nullptr;
    k.dhidden_stride = (long long)(a->dhidden_stride ? a->dhidden_stride : a->dim);
    k.dweight_stride = (long long)(a->dweight_stride ? a->dweight_stride : a->dim);
    k.dhidden = a->dhidden;
    k.want_dw = a->dweights != nullptr;
    k.lse_in = a->lse;
    k.entropy_in = a->entropy;
    k.dlogprob = a->dlogprob;
    k.dentropy = a->dentropy;
    note_op_call(h, a->p, stream);

    // the products' rows are those of G, and of the hidden states that have a part in it
    if (k.pair) k.tokens = 2 * k.pair;
    VocabArgs rows = k;
    rows.hidden = k.hidden_used;
    rows.hidden_stride = k.dim;
    CallMaps m;
    if (k.tokens && !make_maps(a->dtype, rows, &m)) return fail(h, RAR_ECUDA, "rar_vocab_logprobs_grad: the driver refused a tensor map");
    auto run = [&](auto dt) {
        constexpr int DT = decltype(dt)::value;
        if (!k.tokens) return clear_dweights(k, stream);
        cudaError_t e = cudaMemsetAsync(k.w_max, 0, sizeof(*k.w_max), stream);
        if (e == cudaSuccess)
            e = launch_pdl(logprob_prepare_kernel, dim3((unsigned)((n + kPrepareTokens - 1) / kPrepareTokens)), dim3(32 * kPrepareTokens), 0, stream, k);
        if (e != cudaSuccess) return e;
        return k.dim > 64 * kStepsPerSum ? launch_gradients<TILES_LOGPROB_G_SUMS, DT>(h, k, m, stream) : launch_gradients<TILES_LOGPROB_G, DT>(h, k, m, stream);
    };
    const cudaError_t ce = a->dtype == RAR_BFLOAT16 ? run(IntC<DT_BF16>{}) : run(IntC<DT_F16>{});
    return ce == cudaSuccess ? RAR_OK : cuda_fail(h, ce, "launching the log probabilities' gradients");
}

}  // namespace
}  // namespace rar

extern "C" {

size_t rar_vocab_logprobs_workspace(size_t tokens, size_t dim, size_t vocab, int p, int top) {
    if (!rar::sizes_ok(tokens, dim, vocab, p) || top < 0 || top > RAR_LOGPROBS_MAX_TOP) return 0;
    rar::VocabArgs k{};
    float *logits;
    return rar::plan(nullptr, tokens, dim, vocab, p, top, &k, &logits);
}

int rar_vocab_logprobs(rar_handle h, const rar_vocab_logprobs_args *a, void *stream) {
    return rar::guarded(h, [&] {
        if (!h) return rar::fail(nullptr, RAR_EINVAL, "handle is NULL");
        return rar::vocab_logprobs(h, a, (cudaStream_t)stream);
    });
}

size_t rar_vocab_logprobs_grad_workspace(size_t tokens, size_t dim, size_t vocab, int p) {
    if (!rar::sizes_ok(tokens, dim, vocab, p)) return 0;
    rar::VocabArgs k{};
    return rar::plan_gradients(nullptr, tokens, dim, vocab, p, &k);
}

int rar_vocab_logprobs_grad(rar_handle h, const rar_vocab_logprobs_grad_args *a, void *stream) {
    return rar::guarded(h, [&] {
        if (!h) return rar::fail(nullptr, RAR_EINVAL, "handle is NULL");
        return rar::vocab_logprobs_grad(h, a, (cudaStream_t)stream);
    });
}

}  // extern "C"

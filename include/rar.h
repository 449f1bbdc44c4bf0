/*
 * rar.h -- ring all-reduce over p virtual ranks held in one GPU's memory.
 *
 * The operation ("Ring All-Reduce, in depth", section "The schedule"):
 * p ranks, each with an n-element buffer cut into p chunks by chunk_bounds
 * (section "An implementation": the first n mod p chunks are one element
 * longer).  Reduce-scatter runs p - 1 steps; at step s rank r sends chunk
 * (r - s) mod p to rank r + 1, which combines it into its own copy, so that
 * afterwards rank r holds the complete reduction of chunk (r + 1) mod p.
 * All-gather runs p - 1 more steps; at step s rank r sends chunk
 * (r + 1 - s) mod p and the receiver overwrites its copy.  Every rank ends
 * with the elementwise reduction ("AllReduce 与 Ring 通信算法详解", section
 * "AllReduce 语义": sum, average or maximum).
 *
 * Arithmetic follows the ring's hop order exactly: element i of chunk c
 * becomes x_c[i] (+) x_(c+1)[i] (+) ... (+) x_(c+p-1)[i] (indices mod p),
 * each (+) rounded to the buffer's dtype ("Derive the cost of a ring
 * all-reduce", last probe: the reduction runs in the buffer's dtype), so the
 * result is bit-identical to the schedule run on real ranks.  avg is that
 * sum times 1/p (rounded to binary32), applied once by the chunk's owner and
 * rounded once to binary32, then to a 16-bit dtype.  max keeps the running
 * value unless the receiver's element is strictly greater.
 *
 * All p rank buffers live in the GPU's HBM; the library moves no data
 * between GPUs.  Engines (rar_options.engine):
 *   RAR_ENGINE_FUSED       one kernel reads every rank's element once, folds
 *                          in hop order and stores the result to every rank
 *                          (2 p n element moves); on the per-thread path with
 *                          p > 8, a second small launch folds the vectors that
 *                          lie across an unaligned chunk start;
 *   RAR_ENGINE_RING        persistent executor: CTA groups play the ranks and
 *                          run the schedule step by step, slice-pipelined,
 *                          handing slices to the right neighbour through
 *                          acquire/release flags (5 (p - 1) n element moves),
 *                          or, for small buffers, through tagged words in a
 *                          mailbox (rar_options.protocol);
 *   RAR_ENGINE_RING_BIDIR  as RING, with the buffer's second half run by a
 *                          ring in the opposite direction ("Bidirectional
 *                          rings" in "Ring All-Reduce, in depth", section
 *                          "What real libraries add");
 *   RAR_ENGINE_FUSED_TREE  one kernel, tree order over the rank index (adjacent
 *                          pairs level by level); not bit-identical to the
 *                          ring, float sums within 4 p 2^-24 sum|x| of exact.
 *   RAR_ENGINE_TREE        persistent executor of the tree all-reduce schedule
 *                          ("Derive the cost of a ring all-reduce": reduce up a
 *                          binary tree, broadcast down, 2 ceil(log2 p) steps);
 *                          same arithmetic as RAR_ENGINE_FUSED_TREE; full
 *                          all-reduce with sum, max or avg; the same two
 *                          hand-offs as RAR_ENGINE_RING.
 *
 * Conventions for every call:
 *   - Return value: RAR_OK or a rar_status_code; rar_last_error(h) gives a
 *     message.  Argument errors are reported synchronously and launch
 *     nothing.  Device-side errors (a ring wait that timed out) surface
 *     through rar_status().
 *   - Buffers: `bufs` is a host array of p device pointers, each to n
 *     contiguous elements on the handle's device, pairwise non-overlapping.
 *     The caller owns them; the operation is in place.  The array itself is
 *     read during the call only.  All pointers 16-byte aligned select the
 *     128-bit path; otherwise a per-element path runs (same results).
 *   - Streams: work is enqueued on `stream` (a cudaStream_t; NULL = the
 *     legacy default stream) and the call returns without waiting.  One call
 *     in flight per handle: calls on one stream are ordered; calls on several
 *     streams with one handle must be ordered by the caller.
 *   - Ring and tree engines run one cooperative launch of up to every
 *     co-resident CTA of the device; the GPU runs all CTAs of a launch
 *     together, and every wait inside is bounded (rar_options.timeout_ns),
 *     so a launch that cannot make progress ends with RAR_ETIMEOUT rather
 *     than hanging.
 *   - CUDA graphs: rar_allreduce, rar_reduce_scatter and rar_all_gather may
 *     be recorded with stream capture and replayed any number of times; the
 *     ring and tree executors keep their epoch in device memory, so every
 *     replay is a fresh launch.  Create the handle outside the capture.
 *   - Trivial calls: p == 1 or n == 0 return RAR_OK and launch nothing (the
 *     torch ring in "An implementation" returns its tensor when p == 1);
 *     with n == 0 the rank pointers may be NULL.
 */
#ifndef RAR_H
#define RAR_H

#include <stddef.h>

#ifdef __cplusplus
extern "C" {
#endif

#define RAR_VERSION 1
#define RAR_MAX_P 1024

typedef struct rar_ctx *rar_handle;

typedef enum { RAR_INT32 = 0, RAR_FLOAT32 = 1, RAR_BFLOAT16 = 2, RAR_FLOAT16 = 3 } rar_dtype;
typedef enum {
    RAR_SUM = 0,
    RAR_MAX = 1,
    RAR_AVG = 2,        /* ring-order sum, then x 1/p at the chunk's owner */
    RAR_AVG_PREDIV = 3  /* every rank's element x 1/p (rounded to the dtype) as it
                           enters the ring, then the ring-order sum: a 16-bit sum over
                           many ranks cannot overflow ("Ring All-Reduce, in depth",
                           "Failure modes": pre-divide) */
} rar_op;
typedef enum {
    RAR_ENGINE_FUSED = 0,
    RAR_ENGINE_RING = 1,
    RAR_ENGINE_RING_BIDIR = 2,
    RAR_ENGINE_FUSED_TREE = 3,
    RAR_ENGINE_TREE = 4
} rar_engine;

typedef enum {
    RAR_OK = 0,
    RAR_EINVAL = 1,        /* bad argument (null, p out of range, overlap, wrong device) */
    RAR_EUNSUPPORTED = 2,  /* valid but not offered (avg on int32, grid not co-resident) */
    RAR_ENOMEM = 3,        /* scratch allocation failed in rar_init */
    RAR_ECUDA = 4,         /* a CUDA runtime call failed; message in rar_last_error */
    RAR_ETIMEOUT = 5,      /* a bounded wait ran past timeout_ns (from rar_status) */
    RAR_EABORTED = 6       /* the call was abandoned after another CTA timed out */
} rar_status_code;

typedef enum { RAR_FAULT_NONE = 0, RAR_FAULT_MUTE = 1, RAR_FAULT_DELAY = 2 } rar_fault_mode;

/* Options; an all-zero struct means "defaults". */
typedef struct {
    int engine;                    /* rar_engine */
    int channels;                  /* ring engines: CTAs per rank, 0 = chosen from the SM count */
    int slice_elems;               /* ring engines: elements per pipelined slice, 0 = auto */
    int block_threads;             /* threads per CTA (multiple of 32, <= 1024), 0 = auto */
    unsigned long long timeout_ns; /* bound on every wait of the ring and tree engines, of
                                      the fused engine's streaming path (a bulk load
                                      that does not arrive) and of the model operators;
                                      0 = 2 s; nonzero values
                                      below 1 ms (1000000) are refused with RAR_EINVAL.
                                      A wait that runs out ends the call with
                                      RAR_ETIMEOUT (rar_status); the streaming path
                                      still waits for every bulk load it issued before
                                      its CTAs finish, whatever this bound */
    int skip_pointer_check;        /* nonzero: skip the per-call device-pointer query */
    int fault_mode;                /* rar_fault_mode (tests): ring and tree engines; and
                                      RAR_FAULT_MUTE on the fused streaming path, where
                                      the loads of rank fault_rank are never issued, as
                                      if that rank had died, and in the same way in
                                      rar_add_rmsnorm and its gradient, for many rows,
                                      rar_vocab_xent, rar_vocab_logprobs and its gradient
                                      (fault_rank: a piece) */
    int fault_rank;                /* rank the fault applies to (rar_add_rmsnorm_grad: 0 dout,
                                      1 sum, 2 dsum) */
    unsigned fault_delay_ns;       /* RAR_FAULT_DELAY: pause before each slice */
    int fused_path;                /* RAR_ENGINE_FUSED data path, same results on both:
                                      0 auto; 1 per-thread 128-bit loads of all p
                                      ranks and streaming stores; 2 rank-sequential
                                      streaming: bulk copies (TMA) of one rank tile
                                      at a time in hop order into shared memory,
                                      running values in registers, bulk stores of
                                      the result (full all-reduce, 16-byte aligned
                                      ranks; slice_elems = tile elements per rank,
                                      channels = pipeline stages, 0 = auto) */
    int hier_group;                /* 0 (or 1 or p): the flat ring.  g with 1 < g < p, g | p:
                                      the hierarchical 2D schedule over p / g nodes of g
                                      consecutive ranks ("Ring All-Reduce, in depth",
                                      "Hierarchy"): reduce-scatter inside each node,
                                      all-reduce of each 1/g shard across the nodes, all-gather
                                      inside each node.  Full all-reduce only; RAR_ENGINE_RING
                                      runs it as three ring launches, RAR_ENGINE_FUSED folds in
                                      its order on the per-thread path */
    int protocol;                  /* RAR_ENGINE_RING and RAR_ENGINE_TREE hand-off, same
                                      results on both:
                                      0 auto (low latency for small buffers);
                                      1 progress words: a slice is published by a
                                      release store, and the receiver reads it in place
                                      in the sender's buffer;
                                      2 low latency: every 32-bit word travels with a
                                      tag in one 64-bit store through a mailbox in the
                                      handle's scratch.  Ring: full all-reduce on the flat
                                      ring, while p * 2 (p - 1) chunk-sized slots fit in
                                      RAR_LL_MAILBOX_BYTES; tree: while
                                      p * (ceil(log2 p) + 1) buffer-sized slots fit */
    int slice_block;               /* ring and tree executors with progress words.  Ring:
                                      each channel takes its slices in blocks of this many and
                                      runs a block through every step before the next, so that
                                      the reader finds a fresh slice still in L2 (0 = auto: 1;
                                      a value at least the slices per step gives the
                                      step-by-step order).  Tree: slices per CTA of the
                                      least-loaded ranks in one group of the wavefront (0 =
                                      auto: 1 or 2).  Results do not depend on it. */
    int trace;                     /* nonzero: the ring executor (flat and bidirectional)
                                      and the tree executor, with progress words, record per
                                      rank and schedule step the time spent waiting for the
                                      neighbour and the time spent on its slices (rar_trace).
                                      rar_init / rar_set_options allocate the record, 2 x
                                      RAR_MAX_P x RAR_TRACE_MAX_STEPS words (32 MB) */
} rar_options;

/* Schedule steps a trace holds per rank (2 (RAR_MAX_P - 1)). */
#define RAR_TRACE_MAX_STEPS 2046

/* Bytes of the low-latency mailbox each handle allocates in rar_init. */
#define RAR_LL_MAILBOX_BYTES (64u << 20)

/* Create a handle on `device`; allocates the ring and tree engines' progress
 * words, counters and status word there (about 33 MB) and the low-latency mailbox
 * (RAR_LL_MAILBOX_BYTES).  opt may be NULL.
 * Errors: RAR_EINVAL (out NULL, bad device or option), RAR_ENOMEM,
 * RAR_ECUDA. */
int rar_init(rar_handle *out, int device, const rar_options *opt);

/* Replace the handle's options between calls (same validation as rar_init). */
int rar_set_options(rar_handle h, const rar_options *opt);

/* In-place all-reduce of p rank buffers of n elements (the whole schedule:
 * reduce-scatter then all-gather).
 * Errors: RAR_EINVAL (null handle/array/pointer, p < 1 or p > RAR_MAX_P,
 * unknown dtype or op, n * element size overflows, overlapping buffers,
 * pointers not device memory of the handle's device), RAR_EUNSUPPORTED
 * (avg or avg_prediv on int32; ring engine grid cannot be co-resident), RAR_ECUDA. */
int rar_allreduce(rar_handle h, void *const *bufs, int p, size_t n, int dtype, int op,
                  void *stream);

/* The reduce-scatter half alone ("Ring All-Reduce, in depth", section
 * "Trade-offs": the two halves are also used separately).  Afterwards rank r
 * holds the complete reduction of chunk (r + 1) mod p in that chunk's place
 * in its buffer (avg already scaled); its other chunks hold partial values
 * (fused engines: unchanged inputs; ring engines: the schedule's partials).
 * RAR_ENGINE_RING_BIDIR: the first half's chunk (r + 1) and the second
 * half's chunk (r - 1), both by chunk_bounds of that half.
 * Same arguments and errors as rar_allreduce. */
int rar_reduce_scatter(rar_handle h, void *const *bufs, int p, size_t n, int dtype, int op,
                       void *stream);

/* The all-gather half alone: rank r's chunk (r + 1) mod p is copied to every
 * other rank (RAR_ENGINE_RING_BIDIR: by the same split as in
 * rar_reduce_scatter).  After rar_reduce_scatter this completes the
 * all-reduce.  No arithmetic; dtype only sets the element size.
 * Same arguments and errors as rar_allreduce (op is not taken). */
int rar_all_gather(rar_handle h, void *const *bufs, int p, size_t n, int dtype, void *stream);

/* In-place all-reduce of the index range [lo, hi) of p rank buffers of
 * n_total elements each: bufs[r] points at element lo of rank r's buffer
 * (hi - lo elements behind it, owned by the caller).  Chunks are cut from
 * n_total by chunk_bounds, and every element is reduced in its chunk's order,
 * so the range ends up exactly as rar_allreduce over the whole buffers leaves
 * it, bit for bit, with the handle's engine.  The pages have no such call;
 * it rests on each result element depending only on the inputs at its index
 * and on its chunk: disjoint ranges can be reduced by separate calls (on
 * separate streams, or on the GPUs that hold them) without any exchange.
 * Send counts (rar_send_counts) are the elements moved for this range; over
 * ranges that cover [0, n_total) they add up to the whole call's counts.
 * Errors: as rar_allreduce; RAR_EINVAL unless lo <= hi <= n_total.
 * lo == hi is a no-op. */
int rar_allreduce_range(rar_handle h, void *const *bufs, int p, size_t n_total, size_t lo, size_t hi, int dtype,
                        int op, void *stream);

/* All-reduce of host-resident rank buffers, with the handle's engine.
 *   host_bufs  host array of p host pointers, n elements each; the result
 *              replaces the inputs
 *   dev_bufs   host array of p device pointers (n elements each, owned by
 *              the caller), or NULL; used only for pageable host memory
 * If every host buffer is page-locked and mapped for the handle's device
 * (cudaHostAlloc, or torch's pin_memory), the kernel reads the inputs and
 * writes the results over the host link itself, in one pass, and dev_bufs is
 * not touched.  Otherwise the buffers are staged, in stream order: each host
 * buffer is copied into dev_bufs[r], those are all-reduced (as
 * rar_allreduce), and the results are copied back (these copies wait for the
 * host when the memory is pageable).  The library allocates nothing.
 * Errors: as rar_allreduce; RAR_EINVAL if host_bufs or an entry is NULL, or
 * the memory is pageable and dev_bufs is NULL. */
int rar_allreduce_host(rar_handle h, void *const *host_bufs, void *const *dev_bufs, int p, size_t n, int dtype,
                       int op, void *stream);

/* All-reduce for callers that may not allocate device memory: callers whose
 * device memory belongs to another allocator (a framework's caching
 * allocator, a pre-planned arena with a fixed budget), and callers that
 * cannot pay for cudaMalloc/cudaFree at call time (both can block; cudaFree
 * synchronises the device).  The source pages have no counterpart: this is
 * the ring executor (RAR_ENGINE_RING with progress words) without a handle,
 * with its scratch -- progress words, receive counters, the status and the
 * abort word -- in one fixed-size device array inside the library (about
 * 80 KB, resident on every GPU that loads the library until exit).  Its
 * tuning is fixed: 256 threads per CTA, every co-resident CTA up to 1024 in
 * all, 128 KB slices (the handle's ring uses 512 threads and slices of up to
 * 128 KB); the results are the same bits as rar_allreduce's with
 * RAR_ENGINE_RING.
 * Arguments and results are as rar_allreduce's, on the current device.
 * Limits: p <= 64 and p * channels <= 1024 CTAs; larger p returns
 * RAR_EINVAL with a message from rar_last_error(NULL).
 * The first call on a device, with that device current, sets the array up
 * (clears it once, synchronously; so does the first call after
 * cudaDeviceReset, which reloads the array); make that first call before
 * any stream capture.  Every call uses the same array: calls that overlap
 * on the GPU (two streams, two threads) race and must be ordered by the
 * caller.
 * A ring wait that runs out (2 s) ends the kernel early and leaves the
 * buffers partly reduced; without a handle this entry point cannot report
 * it, so callers who need that status use rar_allreduce.
 * Errors: as rar_allreduce, reported through the return value and
 * rar_last_error(NULL). */
int rar_allreduce_noalloc(void *const *bufs, int p, size_t n, int dtype, int op, void *stream);

/* Synchronise the stream of the last call and return the device-side status:
 * RAR_OK, or RAR_ETIMEOUT if a bounded wait ran out since the previous report
 * (in the last call, or in a replay of a captured one); rar_last_error names
 * the rank, step and slice.  Each failure is reported once.  A timed-out call
 * leaves the buffers partly updated; the handle stays usable. */
int rar_status(rar_handle h);

/* Per-rank count of elements each rank sent in the last ring-engine call
 * (the fused engines send nothing; counts are 0).  out has p entries; p must
 * equal the last call's p.  Synchronises like rar_status.  For the full
 * all-reduce, sends_r = 2 n - |C_(r+1)| - |C_(r+2)| ("Ring All-Reduce, in
 * depth", "The schedule": 2 (p - 1)/p x n when p divides n). */
int rar_send_counts(rar_handle h, unsigned long long *out, int p);

/* Message for the handle's last error (never NULL; "" when none).  Valid
 * until the next call on the handle.  h may be NULL for rar_init errors. */
const char *rar_last_error(rar_handle h);

/* Synchronise the device, free the scratch and the handle.  NULL is a no-op. */
int rar_destroy(rar_handle h);

/* RAR_VERSION of the loaded library. */
int rar_version(void);

/* Per-rank step times of the last call, when rar_options.trace was set and
 * the call ran the ring executor (flat or bidirectional) or the tree
 * executor with progress words ("Ring All-Reduce, in depth", "Failure
 * modes": a straggler shows as the rank whose steps take longest, and its
 * right neighbour as the one that waits longest).  For rank r and schedule
 * step s (global step index: 0 .. 2 (p - 1) - 1 for the ring, 0 .. 2L - 1
 * for the tree), work_ns[r * max_steps + s] is the time the rank's CTAs spent on
 * their slices of that step (from the end of the wait to the release of the
 * slice, summed over CTAs; an injected delay counts as work), and
 * wait_ns[r * max_steps + s] the time they spent waiting for the neighbour's
 * progress word; both from the first warp of each CTA, in nanoseconds of
 * %globaltimer.  *steps receives the step count; the arrays hold
 * p * max_steps entries.  Synchronises like rar_status.
 * Errors: RAR_EINVAL (null argument, p differs from the last call's,
 * max_steps too small, or the last call was not traced). */
int rar_trace(rar_handle h, unsigned long long *work_ns, unsigned long long *wait_ns, int p, int max_steps,
              int *steps);

/* Test hook: set the handle's launch epoch counter (device memory; the next
 * ring-engine or tree launch runs with epoch + 1).  The ring engines tag
 * progress words and mailbox words with a 32-bit epoch; the launch that runs
 * with epoch 0xFFFFFFFF clears them all and restarts the count, so no stale
 * tag can match.  This call lets a test reach that launch without 2^32
 * calls.  Synchronises the device; no call may be in flight.
 * Errors: RAR_EINVAL (null handle), RAR_ECUDA. */
int rar_debug_set_epoch(rar_handle h, unsigned epoch);

/* ---------------------------------------------------------------------------
 * Operators of a tensor-parallel language model.
 *
 * Such a model meets the reduction over its p ranks in several places: the
 * residual stream joins the sum of the ranks' partial outputs and is
 * normalised (rar_add_rmsnorm); the output layer's vocabulary is cut into one
 * piece per rank, over which the softmax is reduced (rar_vocab_xent,
 * rar_vocab_logprobs); the input table is cut the same way (rar_embedding); and
 * all ranks' gradients have one norm (rar_grad_norm, rar_grad_clip).  The source
 * pages have no such calls.  Here the reduction is part of the operator, and what every rank
 * would hold afterwards is written once, since the ranks share one memory.
 *
 * Conventions of these calls, beyond those at the top of this file:
 *   - dtype is RAR_FLOAT32, RAR_BFLOAT16 or RAR_FLOAT16 where nothing else is
 *     said; RAR_INT32 is refused with RAR_EUNSUPPORTED.
 *   - Matrices are row-major with contiguous rows; *_stride is the distance
 *     between rows in elements, 0 means densely packed rows, any other value
 *     must be at least the row's length.  Addresses need the alignment of
 *     their type only, where nothing else is said.
 *   - "Piece r" of a vocabulary is rows [start_r, start_(r+1)) by
 *     chunk_bounds(vocab, p), as a matrix of its own; an empty piece may be
 *     NULL.
 *   - Indices (tokens, targets) are signed 32 or 64 bits wide (index_bytes 4 or
 *     8).  An index outside [0, vocab) marks a place that is left out.
 *   - Sums, norms and softmax statistics are held in 32 bits; a result is
 *     rounded once, where it is written.  Results do not depend on timing:
 *     the same call gives the same bits.
 *   - An output may not overlap an input or another output, except where a
 *     call names the pairs that may be the same matrix.
 *   - Argument errors are RAR_EINVAL (null handle, struct or matrix, a size,
 *     stride, dtype or pointer out of its range, a pointer that is not device
 *     memory of the handle's device) and launch nothing.  rar_status covers
 *     these calls too.  They may be captured into CUDA graphs, unless p is above
 *     64.  They allocate nothing: what they need beyond the results is the
 *     caller's workspace, 256-byte aligned, whose size a call of its own gives
 *     and whose contents mean nothing between calls.
 */

/* s = residual + x_0 + ... + x_(p-1), y = s / sqrt(mean(s^2) + eps) * weight,
 * row by row: the join of the residual stream with the ranks' partial results,
 * and the norm that the next layer begins with.  The partials are added in the
 * ring's hop order of the flat rows x dim buffer (so with RAR_FLOAT32 and
 * without residual `sum` has rar_allreduce's bits), in 32 bits throughout, then the
 * residual; y is taken from the unrounded s.
 * 8-bit output: for each row and each run of `group` columns,
 * scale = max(min(max|y|, FLT_MAX) / 448, FLT_MIN) over the values that are not
 * NaN, and code = y / scale rounded to nearest even to float8 e4m3 (finite
 * codes up to +-448, which also takes infinities; NaN stays NaN). */
typedef struct {
    const void *const *parts; /* host array of p matrices rows x dim */
    int p;                    /* 1 .. RAR_MAX_P */
    int dtype;                /* of parts, residual, weight, sum and out */
    size_t rows, dim;         /* rows 0 (nothing is done) .. 2^31 - 1; dim 1 .. RAR_NORM_MAX_DIM */
    size_t part_stride;
    const void *residual;     /* rows x dim, or NULL */
    size_t residual_stride;
    const void *weight;       /* dim, or NULL: ones */
    float eps;                /* >= 0 */
    void *sum;                /* out: s, or NULL; may be the residual or a part itself */
    size_t sum_stride;
    void *out;                /* out: y, or NULL; may be a part itself, or the residual */
    size_t out_stride;
    float *rstd;              /* out: rows values 1 / sqrt(mean(s^2) + eps), or NULL */
    void *out8;               /* out: codes, one byte each, or NULL */
    size_t out8_stride;
    float *scales;            /* out: rows x ceil(dim / group), needed with out8 */
    size_t group;             /* columns per scale; 0: the whole row; else a multiple of 32
                                 (one of dim or more: the whole row, too) */
} rar_rmsnorm_args;

#define RAR_NORM_MAX_DIM 32768

int rar_add_rmsnorm(rar_handle h, const rar_rmsnorm_args *a, void *stream);

/* Gradient of rar_add_rmsnorm, from the gradients of y (dout) and of s (dsum):
 *   dx = dsum + rstd (weight dout - s rstd^2 mean(weight dout s)),
 * which is the gradient of the residual and of every part alike, and
 *   dweight = sum over the rows of dout s rstd, added in a fixed order. */
typedef struct {
    int dtype;                /* of every matrix and of weight and dweight */
    size_t rows, dim;         /* 0 rows: dweight is zeros */
    const void *dout;         /* rows x dim */
    size_t dout_stride;
    const void *dsum;         /* rows x dim, or NULL: zeros */
    size_t dsum_stride;
    const void *sum;          /* s as rar_add_rmsnorm wrote it */
    size_t sum_stride;
    const float *rstd;
    const void *weight;       /* dim, or NULL: ones */
    void *dx;                 /* out: rows x dim, or NULL; may be dout or dsum itself */
    size_t dx_stride;
    void *dweight;            /* out: dim, or NULL */
    void *workspace;          /* needed with dweight */
    size_t workspace_bytes;
} rar_rmsnorm_grad_args;

size_t rar_add_rmsnorm_grad_workspace(size_t rows, size_t dim);
int rar_add_rmsnorm_grad(rar_handle h, const rar_rmsnorm_grad_args *a, void *stream);

/* Softmax cross entropy over a vocabulary in p pieces, from the hidden states:
 *   z = hidden W^T, lse = log sum exp(z), loss = lse - z[target],
 * and, where dhidden or dweights is given, the gradients of
 * sum over the tokens of token_weight x loss:
 *   G = (exp(z - lse) - onehot(target)) token_weight,
 *   dhidden = G W,  dweights = G^T hidden.
 * The logits are never kept: they are computed a tile at a time, once for lse and
 * once more for G, which is held in the dtype for a window of the vocabulary at a
 * time.  A token whose target is left out has loss 0 and no gradient, whatever its
 * hidden state holds; its lse is computed.
 * dtype: RAR_BFLOAT16 or RAR_FLOAT16 (RAR_FLOAT32: RAR_EUNSUPPORTED).  dim is a
 * multiple of 8, matrices are 16-byte aligned with strides that are multiples of
 * 8, p is at most 64. */
typedef struct {
    const void *hidden;          /* tokens x dim */
    size_t hidden_stride;
    const void *const *weights;  /* host array of p pieces, rows x dim */
    size_t weight_stride;        /* of every piece */
    int p;
    int dtype;
    size_t tokens, dim, vocab;   /* tokens may be 0, dim and vocab at least 1 */
    const void *targets;         /* tokens indices */
    int index_bytes;
    const float *token_weight;   /* tokens, or NULL: ones */
    float *loss;                 /* out: tokens, or NULL */
    float *lse;                  /* out: tokens, or NULL */
    void *dhidden;               /* out: tokens x dim, or NULL */
    size_t dhidden_stride;
    void *const *dweights;       /* out: host array of p pieces, or NULL */
    size_t dweight_stride;
    void *workspace;
    size_t workspace_bytes;
} rar_vocab_xent_args;

/* grad: whether dhidden or dweights will be asked for.  0 where the sizes are refused. */
size_t rar_vocab_xent_workspace(size_t tokens, size_t dim, size_t vocab, int p, int grad);
int rar_vocab_xent(rar_handle h, const rar_vocab_xent_args *a, void *stream);

/* out[t] = scale x table[tokens[t]] over a table in p pieces; zeros where a
 * token is left out. */
typedef struct {
    const void *const *tables; /* host array of p pieces, rows x dim */
    size_t table_stride;       /* of every piece */
    int p;                     /* 1 .. RAR_MAX_P */
    int dtype;
    size_t vocab, dim;         /* at least 1; dim at most 2^31 - 1 */
    const void *tokens;        /* n_tokens indices */
    int index_bytes;
    size_t n_tokens;           /* 0: nothing is done */
    float scale;
    void *out;                 /* n_tokens x dim */
    size_t out_stride;
} rar_embedding_args;

int rar_embedding(rar_handle h, const rar_embedding_args *a, void *stream);

/* Gradient of rar_embedding for the table, dtables[v] = scale x sum of dout[t]
 * over the t with tokens[t] = v.  The tokens are sorted by index and cut into chunks of
 * 16 places or more; a row's gradients are added in 32 bits, in the order of t within a
 * chunk, and the sums of a token that lies in several chunks in an order that the
 * sizes decide.  accumulate: added to what dtables holds (rows without a token stay
 * untouched); otherwise every row is written. */
typedef struct {
    const void *dout;          /* n_tokens x dim */
    size_t dout_stride;
    const void *tokens;
    int index_bytes;
    size_t n_tokens;           /* at most 2^24 */
    void *const *dtables;      /* host array of p pieces */
    size_t dtable_stride;
    int p;
    int dtype;
    size_t vocab, dim;         /* at least 1; vocab at most 2^31 - 1, dim at most 2^22 */
    float scale;
    int accumulate;
    void *workspace;
    size_t workspace_bytes;
} rar_embedding_grad_args;

size_t rar_embedding_grad_workspace(size_t n_tokens, size_t vocab, size_t dim);
int rar_embedding_grad(rar_handle h, const rar_embedding_grad_args *a, void *stream);

/* What the model answers with, from the hidden states and the pieces of
 * rar_vocab_xent: with z = hidden W^T and l = logit_scale z (1 / temperature),
 *   lse = log sum exp(l),  logprob = l[target] - lse,
 *   entropy = lse - sum exp(l - lse) l,
 * and the `top` largest logits of each token, in falling order, equal ones from
 * the lowest index on, with their log probabilities.  A token whose target is left out has
 * logprob 0; its entropy, lse and alternatives are computed.  A logit of NaN or
 * -infinity is no alternative: where fewer than `top` are left, the rest have
 * index -1 and log probability -infinity.
 * dtype, dim, alignment, strides and p as in rar_vocab_xent. */
#define RAR_LOGPROBS_MAX_TOP 32

typedef struct {
    const void *hidden;         /* tokens x dim */
    size_t hidden_stride;
    const void *const *weights; /* host array of p pieces, rows x dim */
    size_t weight_stride;       /* of every piece */
    int p;
    int dtype;
    size_t tokens, dim, vocab;  /* tokens may be 0, dim and vocab at least 1 */
    const void *targets;        /* tokens indices */
    int index_bytes;
    float logit_scale;          /* positive, at most 2^126 */
    int top;                    /* 0 .. RAR_LOGPROBS_MAX_TOP, at most vocab */
    float *logprob;             /* out: tokens, or NULL */
    float *entropy;             /* out: tokens, or NULL */
    float *lse;                 /* out: tokens, or NULL */
    float *top_logprob;         /* out: tokens x top */
    long long *top_token;       /* out: tokens x top */
    void *workspace;
    size_t workspace_bytes;
} rar_vocab_logprobs_args;

/* 0 where the sizes are refused. */
size_t rar_vocab_logprobs_workspace(size_t tokens, size_t dim, size_t vocab, int p, int top);
int rar_vocab_logprobs(rar_handle h, const rar_vocab_logprobs_args *a, void *stream);

/* Gradients of rar_vocab_logprobs, from those of logprob (a) and entropy (b):
 *   G = logit_scale (a onehot(target) - q (a + b (log q + entropy))),
 *   q = exp(l - lse),  dhidden = G W,  dweights = G^T hidden,
 * with lse and entropy as the call above gave them.  A token whose target is
 * left out, or with a = b = 0, has no part in them, whatever its hidden state holds;
 * for a target left out that holds of dentropy, too.
 * Where q is 0 (a logit of -infinity, or one that is it after scaling) q log q is 0, too.
 * G is held in the dtype for a window of the vocabulary at a time. */
typedef struct {
    const void *hidden;         /* as in rar_vocab_logprobs_args, down to logit_scale */
    size_t hidden_stride;
    const void *const *weights;
    size_t weight_stride;
    int p;
    int dtype;
    size_t tokens, dim, vocab;
    const void *targets;
    int index_bytes;
    float logit_scale;
    const float *lse;           /* tokens */
    const float *entropy;       /* tokens; needed with dentropy */
    const float *dlogprob;      /* tokens, or NULL: zeros */
    const float *dentropy;      /* tokens, or NULL: zeros; one of the two is needed */
    void *dhidden;              /* out: tokens x dim, or NULL */
    size_t dhidden_stride;
    void *const *dweights;      /* out: host array of p pieces, or NULL */
    size_t dweight_stride;
    void *workspace;
    size_t workspace_bytes;
} rar_vocab_logprobs_grad_args;

size_t rar_vocab_logprobs_grad_workspace(size_t tokens, size_t dim, size_t vocab, int p);
int rar_vocab_logprobs_grad(rar_handle h, const rar_vocab_logprobs_grad_args *a, void *stream);

/* A matrix in a list of tensors; a tensor without gaps, of any shape, is one of one row. */
typedef struct {
    void *data;
    int dtype;         /* RAR_FLOAT32, RAR_BFLOAT16 or RAR_FLOAT16, each its own */
    size_t rows, cols; /* 0 of either: an empty tensor */
    size_t stride;     /* between rows, in elements; 0: packed */
} rar_tensor;

/* norms[i] = sqrt(sum x^2) over tensor i, norm = sqrt(sum norms^2): the norm of all
 * ranks' gradients together.  Any values of the tensors' types are squared without
 * overflow or loss; a norm beyond binary32 is infinity.  A tensor given twice counts twice. */
typedef struct {
    const rar_tensor *tensors; /* host array */
    size_t n;                  /* may be 0 (norm 0); at most 2^24, with 2^40 elements in all */
    float *norm;               /* out: one value, or NULL */
    float *norms;              /* out: n, or NULL; one of the two is needed */
    void *workspace;
    size_t workspace_bytes;
} rar_grad_norm_args;

size_t rar_grad_norm_workspace(const rar_tensor *tensors, size_t n);
int rar_grad_norm(rar_handle h, const rar_grad_norm_args *a, void *stream);

/* x * f for every element, f = max_norm / (norm + eps) where that is below 1, else 1:
 * gradients clipped to a largest norm.  A norm that is NaN, or infinite, gives what the
 * formula gives (NaN; 0, and NaN for infinite elements): the caller may look at it first.
 * Tensors that are scaled where they lie must not overlap. */
typedef struct {
    const rar_tensor *tensors; /* host array */
    size_t n;
    const rar_tensor *out;     /* host array of the same sizes, each of its tensor's dtype or RAR_FLOAT32
                                  and its tensor itself or apart from all of them; NULL: in place */
    const float *norm;         /* device memory: as rar_grad_norm gave it */
    float max_norm, eps;       /* finite, not negative */
} rar_grad_clip_args;

int rar_grad_clip(rar_handle h, const rar_grad_clip_args *a, void *stream);

#ifdef __cplusplus
}
#endif
#endif

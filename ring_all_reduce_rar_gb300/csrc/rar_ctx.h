// rar_ctx.h -- the handle behind rar_handle and the host-side helpers that
// the entry points share (errors, current device, rank pointers).
#pragma once

#include <cstring>
#include <string>

#include "rar_internal.h"

namespace rar {
extern thread_local std::string g_init_error;  // errors before a handle exists
}

struct rar_ctx {
    int device = 0;
    rar_options opt{};
    std::string err;
    int sm_count = 0;
    // scratch owned by the handle (ring engines; table for p > kInlineP)
    unsigned long long *flags = nullptr;
    unsigned long long *recv_counts = nullptr;
    rar::RingStatus *status = nullptr;
    unsigned *abort_word = nullptr;
    unsigned *epoch_words = nullptr;  // [0] last finished launch's epoch, [1] finish counter
    void **ptr_table = nullptr;
    unsigned long long *ll_box = nullptr;  // low-latency mailbox, kLLMailboxWords
    unsigned long long *trace = nullptr;   // step trace (rar_options.trace), kTraceWords
    bool last_traced = false;              // the last call filled the trace
    int last_trace_steps = 0;
    unsigned acked_seq = 0;           // status failures already reported
    // last call, for rar_status / rar_send_counts
    bool have_last = false;
    cudaStream_t last_stream = nullptr;
    bool last_ring = false;
    int last_p = 0;
    // ring launches of the last call (the hierarchical schedule makes three)
    int last_phases = 0;
    int last_layout[3] = {0, 0, 0};
    int last_channels[3] = {0, 0, 0};
    int last_fwd_channels[3] = {0, 0, 0};
    int last_group = 0;
};

namespace rar {

inline int fail(rar_ctx *h, int code, const std::string &msg) {
    if (h) h->err = msg;
    else g_init_error = msg;
    return code;
}

inline int cuda_fail(rar_ctx *h, cudaError_t e, const char *what) {
    return fail(h, RAR_ECUDA, std::string(what) + ": " + cudaGetErrorString(e));
}

// Make `dev` current for the scope of a call and restore the caller's device.
struct DeviceGuard {
    int prev = -1;
    bool changed = false;
    cudaError_t err = cudaSuccess;
    explicit DeviceGuard(int dev) {
        err = cudaGetDevice(&prev);
        if (err == cudaSuccess && prev != dev) {
            err = cudaSetDevice(dev);
            changed = err == cudaSuccess;
        }
    }
    ~DeviceGuard() {
        if (changed) cudaSetDevice(prev);
    }
};

// Fill the pointer part of the launch arguments (table copy for large p).
inline int fill_ptrs(rar_ctx *h, RankPtrs &rp, void *const *bufs, int p, cudaStream_t stream) {
    std::memset(&rp, 0, sizeof(rp));
    if (p <= kInlineP) {
        for (int r = 0; r < p; r++) rp.inl[r] = bufs[r];
        return RAR_OK;
    }
    // pageable source: staged by the runtime before the call returns
    cudaError_t ce = cudaMemcpyAsync(h->ptr_table, bufs, sizeof(void *) * (size_t)p, cudaMemcpyHostToDevice, stream);
    if (ce != cudaSuccess) return cuda_fail(h, ce, "copying the rank pointer table");
    rp.table = h->ptr_table;
    return RAR_OK;
}

}  // namespace rar

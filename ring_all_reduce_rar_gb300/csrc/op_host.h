// op_host.h -- host side shared by the model operators' entry points
// (rar_add_rmsnorm, rar_vocab_xent, rar_embedding and their gradients):
// argument checks, the handle's record of the call, and the guard that turns
// C++ exceptions into status codes.
#pragma once

#include <cstdint>
#include <exception>
#include <new>
#include <string>
#include <vector>

#include "rar_ctx.h"

namespace rar {

// A matrix as memory: `rows` runs of `width` bytes, `pitch` bytes apart.
struct MatrixSpan {
    const char *name;
    uintptr_t base;
    size_t rows, width, pitch;
    size_t extent() const { return rows ? (rows - 1) * pitch + width : 0; }
    bool same_as(const MatrixSpan &o) const { return base == o.base && pitch == o.pitch && width == o.width; }
};

// Whether two matrices share a byte.  Two column ranges of one wider matrix
// have equal pitches and interleave without meeting; any other overlap of
// the extents counts as shared.
inline bool spans_meet(const MatrixSpan &a, const MatrixSpan &b) {
    if (!a.rows || !b.rows || !a.width || !b.width) return false;
    if (a.base >= b.base + b.extent() || b.base >= a.base + a.extent()) return false;
    if (a.pitch == b.pitch && (a.rows > 1 || b.rows > 1)) {
        const uintptr_t d = (a.base <= b.base ? b.base - a.base : a.base - b.base) % a.pitch;
        const size_t lower = a.base <= b.base ? a.width : b.width, upper = a.base <= b.base ? b.width : a.width;
        if (d >= lower && d + upper <= a.pitch) return false;
    }
    return true;
}

// Collects a call's matrices and reports the first thing that is wrong.
class OpCheck {
  public:
    OpCheck(rar_ctx *h, const char *call) : h_(h), call_(call) {}
    int bad(const std::string &what) { return fail(h_, RAR_EINVAL, std::string(call_) + ": " + what); }
    int unsupported(const std::string &what) { return fail(h_, RAR_EUNSUPPORTED, std::string(call_) + ": " + what); }

    int dtype(int dt, bool allow_f32) {
        if (dt < RAR_INT32 || dt > RAR_FLOAT16) return bad("unknown dtype");
        if (dt == RAR_INT32) return unsupported("int32 is not offered");
        if (dt == RAR_FLOAT32 && !allow_f32) return unsupported("float32 is not offered");
        return RAR_OK;
    }
    // One matrix of `rows` x `cols` elements of `eb` bytes; `align` bytes.
    int matrix(const char *name, const void *ptr, size_t rows, size_t cols, size_t stride, size_t eb, size_t align,
               MatrixSpan *out) {
        *out = {name, (uintptr_t)ptr, rows, cols * eb, cols * eb};
        if (rows == 0 || cols == 0) return RAR_OK;
        if (!ptr) return bad(std::string(name) + " is NULL");
        if ((uintptr_t)ptr % align) return bad(std::string(name) + " is not aligned to " + std::to_string(align) + " bytes");
        if (cols > kMaxElems) return bad(std::string(name) + " is too large");
        if (stride && stride < cols) return bad(std::string("the stride of ") + name + " is below its row length");
        const size_t pitch = stride ? stride : cols;
        if (pitch > kMaxElems || rows > kMaxElems / pitch) return bad(std::string(name) + " is too large");
        if (align > eb && rows > 1 && pitch * eb % align)
            return bad(std::string("the stride of ") + name + " is not a multiple of " + std::to_string(align) + " bytes");
        out->pitch = pitch * eb;
        if (!h_->opt.skip_pointer_check) {
            cudaPointerAttributes at{};
            if (cudaPointerGetAttributes(&at, ptr) != cudaSuccess) {
                cudaGetLastError();
                return bad(std::string(name) + " is not CUDA memory");
            }
            if ((at.type != cudaMemoryTypeDevice && at.type != cudaMemoryTypeManaged) || at.device != h_->device)
                return bad(std::string(name) + " is not device memory of device " + std::to_string(h_->device));
        }
        return RAR_OK;
    }
    int workspace(const void *ptr, size_t have, size_t need) {
        if (!need) return RAR_OK;
        if (have < need)
            return bad("the workspace has " + std::to_string(have) + " bytes and needs " + std::to_string(need));
        MatrixSpan s;
        int rc = matrix("workspace", ptr, 1, need, 0, 1, 256, &s);
        if (rc != RAR_OK) return rc;
        outputs_.push_back(s);
        return RAR_OK;
    }
    void input(const MatrixSpan &s) { inputs_.push_back(s); }
    void output(const MatrixSpan &s) { outputs_.push_back(s); }
    // Outputs against everything.  in_place(output, input) names the pairs
    // that may be one and the same matrix.
    template <typename F>
    int overlaps(F &&in_place) {
        for (size_t i = 0; i < outputs_.size(); i++) {
            for (size_t j = i + 1; j < outputs_.size(); j++)
                if (spans_meet(outputs_[i], outputs_[j]))
                    return bad(std::string(outputs_[i].name) + " and " + outputs_[j].name + " overlap");
            for (const MatrixSpan &in : inputs_)
                if (spans_meet(outputs_[i], in) && !(outputs_[i].same_as(in) && in_place(outputs_[i], in)))
                    return bad(std::string(outputs_[i].name) + " and " + in.name + " overlap");
        }
        return RAR_OK;
    }

  private:
    static constexpr size_t kMaxElems = (size_t)1 << 58;
    rar_ctx *h_;
    const char *call_;
    std::vector<MatrixSpan> inputs_, outputs_;
};

// The call as rar_status and rar_send_counts see it: nothing was sent.
inline void note_op_call(rar_ctx *h, int p, cudaStream_t stream) {
    h->have_last = true;
    h->last_stream = stream;
    h->last_ring = false;
    h->last_traced = false;
    h->last_p = p;
    h->last_phases = 0;
}

// Whether 16-byte accesses reach every row of a matrix.
inline bool vec16(const void *ptr, size_t rows, long long stride, size_t e) {
    return (uintptr_t)ptr % 16 == 0 && (rows <= 1 || (size_t)stride * e % 16 == 0);
}

// The handle's bound on every wait of a call.
inline unsigned long long op_timeout_ns(const rar_ctx *h) { return h->opt.timeout_ns ? h->opt.timeout_ns : 2000000000ull; }

// The rank that RAR_FAULT_MUTE names, or -1.
inline int op_muted_rank(const rar_ctx *h) { return h->opt.fault_mode == RAR_FAULT_MUTE ? h->opt.fault_rank : -1; }

// Runs an entry point's body: no C++ exception leaves the library.
template <typename F>
int guarded(rar_ctx *h, F &&body) {
    try {
        return body();
    } catch (const std::bad_alloc &) {
    } catch (const std::exception &) {
    }
    try {
        return fail(h, RAR_ENOMEM, "out of host memory");
    } catch (...) {
        return RAR_ENOMEM;
    }
}

// Carves a workspace into 256-byte aligned parts; with base NULL it only
// adds up the sizes.
struct WorkspacePlan {
    char *base;
    size_t used = 0;
    explicit WorkspacePlan(void *b) : base(static_cast<char *>(b)) {}
    template <typename T>
    T *take(size_t count) {
        const size_t at = used;
        used = (used + count * sizeof(T) + 255) / 256 * 256;
        return base ? reinterpret_cast<T *>(base + at) : nullptr;
    }
};

}  // namespace rar

// torch_ops.cpp -- the model operators of include/rar.h on torch tensors: a
// CPython module that checks the tensors, allocates the results and workspaces
// with torch's caching allocator on the stream of the call, and calls the C
// function.  (The same steps through ctypes and torch's Python functions cost 12
// to 37 us a call on the host, more than most of the kernels run.)
//
// Each function returns a tuple of its results, or the status code of the C
// call where that is not RAR_OK; tensors that do not fit raise ValueError.
#include <torch/csrc/autograd/python_variable.h>
// (python first: its header wants to be included before the others)
#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>

#include <cstdint>
#include <stdexcept>
#include <string>
#include <vector>

#include "rar.h"

namespace {

using at::Tensor;

[[noreturn]] void refuse(const std::string &what) { throw std::invalid_argument(what); }

const Tensor &tensor(const std::string &name, PyObject *o) {
    if (!THPVariable_Check(o)) refuse(name + " must be a tensor");
    return THPVariable_Unpack(o);
}

// What a call's matrices share.
struct Common {
    at::ScalarType dtype;
    int code;
    at::Device device;
    Common(const char *name, const Tensor &t) : dtype(t.scalar_type()), device(t.device()) {
        switch (dtype) {
        case at::kInt: code = RAR_INT32; break;
        case at::kFloat: code = RAR_FLOAT32; break;
        case at::kBFloat16: code = RAR_BFLOAT16; break;
        case at::kHalf: code = RAR_FLOAT16; break;
        default: refuse(std::string("unsupported dtype ") + c10::toString(dtype));
        }
        if (!device.is_cuda()) refuse(std::string(name) + " must be a CUDA tensor");
        if (t.dim() != 2) refuse(std::string(name) + " must have two dimensions");
    }
    Tensor make(at::IntArrayRef shape, at::ScalarType type) const { return at::empty(shape, at::TensorOptions().dtype(type).device(device)); }
    Tensor bytes(size_t n) const { return make({(int64_t)n}, at::kByte); }
};

// Row stride of a rows x cols matrix with contiguous rows.
size_t matrix(const std::string &name, const Tensor &t, int64_t rows, int64_t cols, const Common &c) {
    if (t.dim() != 2 || t.size(0) != rows || t.size(1) != cols || t.scalar_type() != c.dtype || t.device() != c.device)
        refuse(name + " must be a (" + std::to_string(rows) + ", " + std::to_string(cols) + ") " + c10::toString(c.dtype) + " tensor on " +
               c.device.str());
    if (cols > 1 && rows > 0 && t.stride(1) != 1) refuse(name + " must have contiguous rows");
    // (a row that expand() repeats has stride 0, which in C stands for packed rows)
    if (rows > 1 && t.stride(0) < cols) refuse("the rows of " + name + " must not overlap: an expanded matrix has to be copied first");
    return (size_t)(rows > 1 ? t.stride(0) : cols);
}
void *vec(const std::string &name, const Tensor &t, int64_t n, at::ScalarType type, const Common &c) {
    if (t.dim() != 1 || t.size(0) != n || t.scalar_type() != type || t.device() != c.device || !t.is_contiguous())
        refuse(name + " must be a contiguous vector of " + std::to_string(n) + " " + c10::toString(type) + " values on " + c.device.str());
    return t.data_ptr();
}
// n < 0: any length.  Returns the bytes of an index.
int indices(const std::string &name, const Tensor &t, int64_t n, const Common &c) {
    const bool wide = t.scalar_type() == at::kLong;
    if ((!wide && t.scalar_type() != at::kInt) || t.dim() != 1 || (n >= 0 && t.size(0) != n) || t.device() != c.device || !t.is_contiguous())
        refuse(name + " must be a contiguous vector of int32 or int64 values on " + c.device.str() +
               (n >= 0 ? ", one for each of " + std::to_string(n) + " rows" : ""));
    return wide ? 8 : 4;
}

// A list or tuple of tensors.
std::vector<const Tensor *> list(const std::string &name, PyObject *o) {
    if (!PyList_Check(o) && !PyTuple_Check(o)) refuse(name + " must be a list or tuple of tensors");
    const Py_ssize_t n = PySequence_Fast_GET_SIZE(o);
    if (n < 1) refuse(name + " must hold at least one tensor");
    std::vector<const Tensor *> v;
    v.reserve((size_t)n);
    for (Py_ssize_t i = 0; i < n; i++) v.push_back(&tensor(name, PySequence_Fast_GET_ITEM(o, i)));
    return v;
}
// Pointers of matrices with one row stride, which those of a single row do
// not decide.
struct Matrices {
    std::vector<void *> ptr;
    size_t stride = 0;
    void add(const std::string &name, const Tensor &t, int64_t rows, int64_t cols, const Common &c) {
        const size_t st = matrix(name, t, rows, cols, c);
        ptr.push_back(t.data_ptr());
        if (rows > 1 && st != stride) {
            if (stride) refuse(name + ": all of them must share their row stride");
            stride = st;
        }
    }
};
// A matrix in pieces by chunk_bounds: the first vocab mod p are one row longer.
struct Pieces : Matrices {
    int64_t vocab = 0, dim = 0, p = 0;
    Pieces(const std::string &name, const std::vector<const Tensor *> &v, const Common &c) : p((int64_t)v.size()) {
        for (const Tensor *t : v) {
            if (t->dim() != 2) refuse(name + " must have two dimensions");
            vocab += t->size(0);
        }
        dim = v[0]->size(1);
        ptr.reserve(v.size());
        for (int64_t r = 0; r < p; r++) add(name, *v[(size_t)r], vocab / p + (r < vocab % p ? 1 : 0), dim, c);
    }
};

void *stream_of(const Common &c) { return c10::cuda::getCurrentCUDAStream(c.device.index()).stream(); }

PyObject *tuple(std::initializer_list<Tensor> ts) {
    PyObject *t = PyTuple_New((Py_ssize_t)ts.size());
    if (!t) return nullptr;
    Py_ssize_t i = 0;
    for (const Tensor &x : ts) {  // an undefined tensor becomes None
        PyObject *o = THPVariable_Wrap(x);
        if (!o) {
            Py_DECREF(t);
            return nullptr;
        }
        PyTuple_SET_ITEM(t, i++, o);
    }
    return t;
}

// Runs `body`, whose exceptions become Python's.
template <typename F>
PyObject *call(Py_ssize_t have, Py_ssize_t want, F &&body) {
    if (have != want) {
        PyErr_SetString(PyExc_TypeError, "wrong number of arguments");
        return nullptr;
    }
    try {
        return body();
    } catch (const std::invalid_argument &e) {
        PyErr_SetString(PyExc_ValueError, e.what());
    } catch (const c10::OutOfMemoryError &e) {
        PyErr_SetString(PyExc_MemoryError, e.what_without_backtrace());
    } catch (const c10::Error &e) {
        PyErr_SetString(PyExc_RuntimeError, e.what_without_backtrace());
    } catch (const std::exception &e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
    }
    return nullptr;
}
rar_handle handle(PyObject *o) { return o == Py_None ? nullptr : (rar_handle)PyLong_AsVoidPtr(o); }

// (handle, parts, weight, residual, eps, group or -1, keep_out) ->
// (sum, rstd, out, out8, scales)
PyObject *add_rmsnorm(PyObject *, PyObject *const *args, Py_ssize_t nargs) {
    return call(nargs, 7, [&]() -> PyObject * {
        const auto parts = list("parts", args[1]);
        const Common c("a part", *parts[0]);
        const int64_t rows = parts[0]->size(0), dim = parts[0]->size(1);
        Matrices m;
        m.ptr.reserve(parts.size());
        for (const Tensor *t : parts) m.add("a part", *t, rows, dim, c);
        const double eps = PyFloat_AsDouble(args[4]);
        const int64_t group = PyLong_AsLongLong(args[5]);
        const bool keep = PyObject_IsTrue(args[6]) == 1;
        if (PyErr_Occurred()) return nullptr;
        if (group < -1) refuse("quant_group must be None, 0 or positive");
        rar_rmsnorm_args a{};
        a.parts = m.ptr.data();
        a.p = (int)parts.size();
        a.dtype = c.code;
        a.rows = (size_t)rows;
        a.dim = (size_t)dim;
        a.part_stride = m.stride;
        a.eps = (float)eps;
        if (args[2] != Py_None) a.weight = vec("weight", tensor("weight", args[2]), dim, c.dtype, c);
        if (args[3] != Py_None) {
            const Tensor &r = tensor("residual", args[3]);
            a.residual_stride = matrix("residual", r, rows, dim, c);
            a.residual = r.data_ptr();
        }
        Tensor sum = c.make({rows, dim}, c.dtype), rstd = c.make({rows}, at::kFloat), out, out8, scales;
        a.sum = sum.data_ptr();
        a.rstd = (float *)rstd.data_ptr();
        if (group < 0 || keep) {
            out = c.make({rows, dim}, c.dtype);
            a.out = out.data_ptr();
        }
        if (group >= 0) {
            out8 = c.make({rows, dim}, at::kFloat8_e4m3fn);
            scales = c.make({rows, group && group < dim ? (dim + group - 1) / group : 1}, at::kFloat);
            a.out8 = out8.data_ptr();
            a.scales = (float *)scales.data_ptr();
            a.group = (size_t)group;
        }
        const int rc = rar_add_rmsnorm(handle(args[0]), &a, stream_of(c));
        return rc ? PyLong_FromLong(rc) : tuple({sum, rstd, out, out8, scales});
    });
}

// (handle, dout, sum, rstd, weight, dsum) -> (dx, dweight)
PyObject *add_rmsnorm_grad(PyObject *, PyObject *const *args, Py_ssize_t nargs) {
    return call(nargs, 6, [&]() -> PyObject * {
        const Tensor &dout = tensor("dout", args[1]), &sum = tensor("sum", args[2]);
        const Common c("dout", dout);
        const int64_t rows = dout.size(0), dim = dout.size(1);
        rar_rmsnorm_grad_args a{};
        a.dtype = c.code;
        a.rows = (size_t)rows;
        a.dim = (size_t)dim;
        a.dout_stride = matrix("dout", dout, rows, dim, c);
        a.dout = dout.data_ptr();
        a.sum_stride = matrix("sum", sum, rows, dim, c);
        a.sum = sum.data_ptr();
        a.rstd = (const float *)vec("rstd", tensor("rstd", args[3]), rows, at::kFloat, c);
        if (args[4] != Py_None) a.weight = vec("weight", tensor("weight", args[4]), dim, c.dtype, c);
        if (args[5] != Py_None) {
            const Tensor &d = tensor("dsum", args[5]);
            a.dsum_stride = matrix("dsum", d, rows, dim, c);
            a.dsum = d.data_ptr();
        }
        a.workspace_bytes = rar_add_rmsnorm_grad_workspace(a.rows, a.dim);
        Tensor dx = c.make({rows, dim}, c.dtype), dweight = c.make({dim}, c.dtype), ws = c.bytes(a.workspace_bytes);
        a.dx = dx.data_ptr();
        a.dweight = dweight.data_ptr();
        a.workspace = ws.data_ptr();
        const int rc = rar_add_rmsnorm_grad(handle(args[0]), &a, stream_of(c));
        return rc ? PyLong_FromLong(rc) : tuple({dx, dweight});
    });
}

// (handle, hidden, weights, targets, token_weight, grad) -> (loss, lse,
// dhidden, list of dweights)
PyObject *vocab_xent(PyObject *, PyObject *const *args, Py_ssize_t nargs) {
    return call(nargs, 6, [&]() -> PyObject * {
        const Tensor &hidden = tensor("hidden", args[1]), &targets = tensor("targets", args[3]);
        const auto weights = list("weights", args[2]);
        const Common c("hidden", hidden);
        const Pieces w("a weight piece", weights, c);
        const int64_t tokens = hidden.size(0);
        const bool grad = PyObject_IsTrue(args[5]) == 1;
        if (PyErr_Occurred()) return nullptr;
        rar_vocab_xent_args a{};
        a.hidden_stride = matrix("hidden", hidden, tokens, w.dim, c);
        a.hidden = hidden.data_ptr();
        a.weights = w.ptr.data();
        a.weight_stride = w.stride;
        a.p = (int)w.p;
        a.dtype = c.code;
        a.tokens = (size_t)tokens;
        a.dim = (size_t)w.dim;
        a.vocab = (size_t)w.vocab;
        a.index_bytes = indices("targets", targets, tokens, c);
        a.targets = targets.data_ptr();
        if (args[4] != Py_None) a.token_weight = (const float *)vec("token_weight", tensor("token_weight", args[4]), tokens, at::kFloat, c);
        a.workspace_bytes = rar_vocab_xent_workspace(a.tokens, a.dim, a.vocab, a.p, grad);
        Tensor loss = c.make({tokens}, at::kFloat), lse = c.make({tokens}, at::kFloat), ws = c.bytes(a.workspace_bytes), dhidden;
        a.loss = (float *)loss.data_ptr();
        a.lse = (float *)lse.data_ptr();
        a.workspace = ws.data_ptr();
        std::vector<Tensor> dweights;
        std::vector<void *> dptrs;
        if (grad) {
            dhidden = c.make({tokens, w.dim}, c.dtype);
            a.dhidden = dhidden.data_ptr();
            for (const Tensor *t : weights) {
                dweights.push_back(c.make({t->size(0), w.dim}, c.dtype));
                dptrs.push_back(dweights.back().data_ptr());
            }
            a.dweights = dptrs.data();
        }
        const int rc = rar_vocab_xent(handle(args[0]), &a, stream_of(c));
        if (rc) return PyLong_FromLong(rc);
        PyObject *r = tuple({loss, lse, dhidden, Tensor()});
        if (r && grad) {
            PyObject *l = PyList_New((Py_ssize_t)dweights.size());
            for (size_t i = 0; l && i < dweights.size(); i++) PyList_SET_ITEM(l, (Py_ssize_t)i, THPVariable_Wrap(dweights[i]));
            if (!l) {
                Py_DECREF(r);
                return nullptr;
            }
            Py_DECREF(PyTuple_GET_ITEM(r, 3));
            PyTuple_SET_ITEM(r, 3, l);
        }
        return r;
    });
}

// (handle, tables, tokens, scale) -> (out,)
PyObject *embedding(PyObject *, PyObject *const *args, Py_ssize_t nargs) {
    return call(nargs, 4, [&]() -> PyObject * {
        const auto tables = list("tables", args[1]);
        const Tensor &tokens = tensor("tokens", args[2]);
        const Common c("a table piece", *tables[0]);
        const Pieces w("a table piece", tables, c);
        rar_embedding_args a{};
        a.tables = w.ptr.data();
        a.table_stride = w.stride;
        a.p = (int)w.p;
        a.dtype = c.code;
        a.vocab = (size_t)w.vocab;
        a.dim = (size_t)w.dim;
        a.index_bytes = indices("tokens", tokens, -1, c);
        a.tokens = tokens.data_ptr();
        a.n_tokens = (size_t)tokens.size(0);
        a.scale = (float)PyFloat_AsDouble(args[3]);
        if (PyErr_Occurred()) return nullptr;
        Tensor out = c.make({tokens.size(0), w.dim}, c.dtype);
        a.out = out.data_ptr();
        const int rc = rar_embedding(handle(args[0]), &a, stream_of(c));
        return rc ? PyLong_FromLong(rc) : tuple({out});
    });
}

// (handle, dout, tokens, dtables, scale, accumulate) -> ()
PyObject *embedding_grad(PyObject *, PyObject *const *args, Py_ssize_t nargs) {
    return call(nargs, 6, [&]() -> PyObject * {
        const Tensor &dout = tensor("dout", args[1]), &tokens = tensor("tokens", args[2]);
        const Common c("dout", dout);
        const Pieces w("a gradient piece", list("dtables", args[3]), c);
        rar_embedding_grad_args a{};
        a.dout_stride = matrix("dout", dout, dout.size(0), w.dim, c);
        a.dout = dout.data_ptr();
        a.index_bytes = indices("tokens", tokens, dout.size(0), c);
        a.tokens = tokens.data_ptr();
        a.n_tokens = (size_t)dout.size(0);
        a.dtables = w.ptr.data();
        a.dtable_stride = w.stride;
        a.p = (int)w.p;
        a.dtype = c.code;
        a.vocab = (size_t)w.vocab;
        a.dim = (size_t)w.dim;
        a.scale = (float)PyFloat_AsDouble(args[4]);
        a.accumulate = PyObject_IsTrue(args[5]) == 1;
        if (PyErr_Occurred()) return nullptr;
        a.workspace_bytes = rar_embedding_grad_workspace(a.n_tokens, a.vocab, a.dim);
        Tensor ws = c.bytes(a.workspace_bytes);
        a.workspace = ws.data_ptr();
        const int rc = rar_embedding_grad(handle(args[0]), &a, stream_of(c));
        return rc ? PyLong_FromLong(rc) : tuple({});
    });
}

#define RAR_FAST(name) {#name, (PyCFunction)(void (*)(void))name, METH_FASTCALL, nullptr}
PyMethodDef methods[] = {RAR_FAST(add_rmsnorm), RAR_FAST(add_rmsnorm_grad), RAR_FAST(vocab_xent), RAR_FAST(embedding),
                         RAR_FAST(embedding_grad), {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_torch_ops", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__torch_ops(void) { return PyModule_Create(&module); }

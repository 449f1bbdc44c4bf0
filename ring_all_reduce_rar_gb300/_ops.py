"""ctypes binding of the model operators in include/rar.h (rar_add_rmsnorm,
rar_vocab_xent, rar_embedding and their gradients).

Argument checks and allocation of results and workspaces only; the work runs
in the library's kernels.  Results are new tensors of the caching allocator, made
on the stream that the call runs on.  Tensors that a call takes must be ready on
that stream, as for every call of this package.
"""
from __future__ import annotations

import contextlib
import ctypes
import functools
from typing import NamedTuple, Optional

from . import _abi

_vp, _sz, _i32, _f32 = ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int, ctypes.c_float


@functools.lru_cache(maxsize=None)
def _torch():
    """torch, imported with the first call: the package itself loads without it."""
    import torch
    return torch


@functools.lru_cache(maxsize=None)
def _codes():
    torch = _torch()
    return {torch.int32: 0, torch.float32: 1, torch.bfloat16: 2, torch.float16: 3}


@functools.lru_cache(maxsize=None)
def _index_bytes():
    torch = _torch()
    return {torch.int32: 4, torch.int64: 8}


class RmsNormArgs(ctypes.Structure):
    """rar_rmsnorm_args."""
    _fields_ = [("parts", _vp), ("p", _i32), ("dtype", _i32), ("rows", _sz), ("dim", _sz), ("part_stride", _sz),
                ("residual", _vp), ("residual_stride", _sz), ("weight", _vp), ("eps", _f32), ("sum", _vp),
                ("sum_stride", _sz), ("out", _vp), ("out_stride", _sz), ("rstd", _vp), ("out8", _vp),
                ("out8_stride", _sz), ("scales", _vp), ("group", _sz)]


class RmsNormGradArgs(ctypes.Structure):
    """rar_rmsnorm_grad_args."""
    _fields_ = [("dtype", _i32), ("rows", _sz), ("dim", _sz), ("dout", _vp), ("dout_stride", _sz), ("dsum", _vp),
                ("dsum_stride", _sz), ("sum", _vp), ("sum_stride", _sz), ("rstd", _vp), ("weight", _vp), ("dx", _vp),
                ("dx_stride", _sz), ("dweight", _vp), ("workspace", _vp), ("workspace_bytes", _sz)]


class VocabXentArgs(ctypes.Structure):
    """rar_vocab_xent_args."""
    _fields_ = [("hidden", _vp), ("hidden_stride", _sz), ("weights", _vp), ("weight_stride", _sz), ("p", _i32),
                ("dtype", _i32), ("tokens", _sz), ("dim", _sz), ("vocab", _sz), ("targets", _vp), ("index_bytes", _i32),
                ("token_weight", _vp), ("loss", _vp), ("lse", _vp), ("dhidden", _vp), ("dhidden_stride", _sz),
                ("dweights", _vp), ("dweight_stride", _sz), ("workspace", _vp), ("workspace_bytes", _sz)]


class EmbeddingArgs(ctypes.Structure):
    """rar_embedding_args."""
    _fields_ = [("tables", _vp), ("table_stride", _sz), ("p", _i32), ("dtype", _i32), ("vocab", _sz), ("dim", _sz),
                ("tokens", _vp), ("index_bytes", _i32), ("n_tokens", _sz), ("scale", _f32), ("out", _vp),
                ("out_stride", _sz)]


class EmbeddingGradArgs(ctypes.Structure):
    """rar_embedding_grad_args."""
    _fields_ = [("dout", _vp), ("dout_stride", _sz), ("tokens", _vp), ("index_bytes", _i32), ("n_tokens", _sz),
                ("dtables", _vp), ("dtable_stride", _sz), ("p", _i32), ("dtype", _i32), ("vocab", _sz), ("dim", _sz),
                ("scale", _f32), ("accumulate", _i32), ("workspace", _vp), ("workspace_bytes", _sz)]


class AddRmsNorm(NamedTuple):
    """Results of add_rmsnorm; those that were not asked for are None."""
    sum: torch.Tensor
    rstd: torch.Tensor
    out: Optional[torch.Tensor]
    out8: Optional[torch.Tensor]
    scales: Optional[torch.Tensor]


class VocabXent(NamedTuple):
    """Results of vocab_xent; the gradients are None unless asked for."""
    loss: torch.Tensor
    lse: torch.Tensor
    dhidden: Optional[torch.Tensor]
    dweights: Optional[list]


def declare(lib) -> None:
    """Argument types of the operators' C functions."""
    for name, args in (("rar_add_rmsnorm", RmsNormArgs), ("rar_add_rmsnorm_grad", RmsNormGradArgs),
                       ("rar_vocab_xent", VocabXentArgs), ("rar_embedding", EmbeddingArgs),
                       ("rar_embedding_grad", EmbeddingGradArgs)):
        f = getattr(lib, name)
        f.argtypes = [_vp, ctypes.POINTER(args), _vp]
        f.restype = _i32
    for name, argtypes in (("rar_add_rmsnorm_grad_workspace", [_sz, _sz]),
                           ("rar_vocab_xent_workspace", [_sz, _sz, _sz, _i32, _i32]),
                           ("rar_embedding_grad_workspace", [_sz, _sz, _sz])):
        f = getattr(lib, name)
        f.argtypes = argtypes
        f.restype = _sz


def _matrix(name, t, rows=None, cols=None, like=None):
    """(pointer, row stride) of a 2-D CUDA tensor with contiguous rows."""
    if t.dim() != 2:
        raise ValueError(f"{name} must have two dimensions")
    shape = t.shape
    if (rows is not None and shape[0] != rows) or (cols is not None and shape[1] != cols):
        raise ValueError(f"{name} must be {rows} x {cols}, got {shape[0]} x {shape[1]}")
    if like is not None and (t.dtype != like.dtype or t.device != like.device):
        raise ValueError(f"{name} must share dtype and device with the other matrices")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    stride = t.stride()
    if shape[1] > 1 and stride[1] != 1:
        raise ValueError(f"{name} must have contiguous rows")
    return t.data_ptr(), (stride[0] if shape[0] > 1 else shape[1])


def _vector(name, t, n, dtype, device):
    if t.dim() != 1 or t.shape[0] != n or t.dtype != dtype or t.device != device or (n > 1 and t.stride(0) != 1):
        raise ValueError(f"{name} must be a contiguous vector of {n} {dtype} values on {device}")
    return t.data_ptr()


def _indices(name, t, device):
    sizes = _index_bytes()
    if t.dim() != 1 or t.dtype not in sizes or t.device != device or (t.shape[0] > 1 and t.stride(0) != 1):
        raise ValueError(f"{name} must be a contiguous vector of int32 or int64 values on {device}")
    return t.data_ptr(), sizes[t.dtype], t.shape[0]


def _code(t):
    code = _codes().get(t.dtype)
    if code is None:
        raise ValueError(f"unsupported dtype {t.dtype}")
    return code


def _pieces(name, pieces, like=None):
    """(pointer array, row stride, p, vocab, dim) of a matrix in pieces by
    chunk_bounds: the first vocab mod p pieces are one row longer."""
    p = len(pieces)
    if p < 1:
        raise ValueError(f"{name}: need at least one piece")
    first = pieces[0]
    like = first if like is None else like
    if first.dim() != 2:
        raise ValueError(f"a piece of {name} must have two dimensions")
    dim = first.shape[1]
    vocab = sum(t.shape[0] for t in pieces)
    base, extra = divmod(vocab, p)
    ptrs, stride = (_vp * p)(), 0
    for r, t in enumerate(pieces):
        rows = base + (r < extra)
        ptr, st = _matrix(f"piece {r} of {name}", t, rows, dim, like)
        ptrs[r] = ptr
        if rows > 1:
            if stride and st != stride:
                raise ValueError(f"the pieces of {name} must share their row stride")
            stride = st
    return ptrs, stride, p, vocab, dim


@contextlib.contextmanager
def _external(stream, device):
    torch = _torch()
    s = torch.cuda.ExternalStream(stream, device=device) if isinstance(stream, int) else stream
    with torch.cuda.stream(s):
        yield s.cuda_stream


def _on_stream(stream, device, body):
    """body(raw stream), with results allocated on that stream."""
    if stream is None:
        return body(_torch().cuda.current_stream(device).cuda_stream)
    with _external(stream, device) as raw:
        return body(raw)


def _workspace(nbytes, device):
    torch = _torch()
    return torch.empty(nbytes, dtype=torch.uint8, device=device) if nbytes else None


def rar_add_rmsnorm(handle, parts, weight=None, residual=None, eps=1e-6, quant_group=None, keep_out=None,
                    stream=None) -> AddRmsNorm:
    """s = residual + sum of the p parts, y = s / rms(s) * weight (see
    rar_add_rmsnorm in rar.h).  parts: p matrices rows x dim of one dtype.
    quant_group None: y is returned in the parts' dtype.  0 or a multiple of
    32: y is returned as float8_e4m3fn codes with a float32 scale per row, or
    per row and run of quant_group columns; keep_out=True keeps `out` as well."""
    torch = _torch()
    if len(parts) < 1:
        raise ValueError("need at least one part")
    x = parts[0]
    if x.dim() != 2:
        raise ValueError("a part must have two dimensions")
    rows, dim = x.shape
    p = len(parts)
    a = RmsNormArgs()
    a.p, a.dtype, a.rows, a.dim, a.eps = p, _code(x), rows, dim, eps
    ptrs = (_vp * p)()
    stride = 0
    for r, t in enumerate(parts):
        ptrs[r], st = _matrix(f"part {r}", t, rows, dim, x)
        if r and st != stride:
            raise ValueError("the parts must share their row stride")
        stride = st
    a.parts, a.part_stride = ctypes.addressof(ptrs), stride
    device = x.device
    if residual is not None:
        a.residual, a.residual_stride = _matrix("residual", residual, rows, dim, x)
    if weight is not None:
        a.weight = _vector("weight", weight, dim, x.dtype, device)
    want_out = quant_group is None or bool(keep_out)

    def body(raw):
        s = torch.empty((rows, dim), dtype=x.dtype, device=device)
        rstd = torch.empty(rows, dtype=torch.float32, device=device)
        a.sum, a.rstd = s.data_ptr(), rstd.data_ptr()
        out = out8 = scales = None
        if want_out:
            out = torch.empty((rows, dim), dtype=x.dtype, device=device)
            a.out = out.data_ptr()
        if quant_group is not None:
            groups = -(-dim // quant_group) if quant_group else 1
            out8 = torch.empty((rows, dim), dtype=torch.float8_e4m3fn, device=device)
            scales = torch.empty((rows, groups), dtype=torch.float32, device=device)
            a.out8, a.scales, a.group = out8.data_ptr(), scales.data_ptr(), quant_group
        _abi._check(handle, _abi.load_library().rar_add_rmsnorm(handle, ctypes.byref(a), raw))
        return AddRmsNorm(s, rstd, out, out8, scales)

    return _on_stream(stream, device, body)


def rar_add_rmsnorm_grad(handle, dout, sum, rstd, weight=None, dsum=None, stream=None):
    """(dx, dweight) of rar_add_rmsnorm: dx is the gradient of the residual
    and of every part alike.  sum and rstd are its results; dsum is the
    gradient of its sum, if that is used elsewhere."""
    torch = _torch()
    if dout.dim() != 2:
        raise ValueError("dout must have two dimensions")
    rows, dim = dout.shape
    device = dout.device
    a = RmsNormGradArgs()
    a.dtype, a.rows, a.dim = _code(dout), rows, dim
    a.dout, a.dout_stride = _matrix("dout", dout)
    a.sum, a.sum_stride = _matrix("sum", sum, rows, dim, dout)
    a.rstd = _vector("rstd", rstd, rows, torch.float32, device)
    if dsum is not None:
        a.dsum, a.dsum_stride = _matrix("dsum", dsum, rows, dim, dout)
    if weight is not None:
        a.weight = _vector("weight", weight, dim, dout.dtype, device)
    lib = _abi.load_library()
    need = lib.rar_add_rmsnorm_grad_workspace(rows, dim)

    def body(raw):
        dx = torch.empty((rows, dim), dtype=dout.dtype, device=device)
        dweight = torch.empty(dim, dtype=dout.dtype, device=device)
        ws = _workspace(need, device)
        a.dx, a.dweight = dx.data_ptr(), dweight.data_ptr()
        if ws is not None:
            a.workspace, a.workspace_bytes = ws.data_ptr(), need
        _abi._check(handle, lib.rar_add_rmsnorm_grad(handle, ctypes.byref(a), raw))
        return dx, dweight

    return _on_stream(stream, device, body)


def rar_vocab_xent(handle, hidden, weights, targets, token_weight=None, grad=False, stream=None) -> VocabXent:
    """Softmax cross entropy of `hidden` (tokens x dim, bfloat16 or float16)
    against a vocabulary in p pieces, without keeping the logits (see
    rar_vocab_xent in rar.h).  A target outside the vocabulary leaves its
    token out.  grad=True also returns the gradients of
    sum(token_weight * loss) for hidden and for every piece."""
    torch = _torch()
    ptrs, wstride, p, vocab, dim = _pieces("weights", weights, hidden)
    device = hidden.device
    a = VocabXentArgs()
    a.hidden, a.hidden_stride = _matrix("hidden", hidden, None, dim)
    tokens = hidden.shape[0]
    a.weights, a.weight_stride, a.p, a.dtype = ctypes.addressof(ptrs), wstride, p, _code(hidden)
    a.tokens, a.dim, a.vocab = tokens, dim, vocab
    a.targets, a.index_bytes, n = _indices("targets", targets, device)
    if n != tokens:
        raise ValueError("targets must hold one index per token")
    if token_weight is not None:
        a.token_weight = _vector("token_weight", token_weight, tokens, torch.float32, device)
    lib = _abi.load_library()
    need = lib.rar_vocab_xent_workspace(tokens, dim, vocab, p, 1 if grad else 0)

    def body(raw):
        stats = torch.empty((2, tokens), dtype=torch.float32, device=device)
        loss, lse = stats.unbind(0)
        a.loss, a.lse = loss.data_ptr(), lse.data_ptr()
        dhidden = dweights = None
        if grad:
            dhidden = torch.empty((tokens, dim), dtype=hidden.dtype, device=device)
            whole = torch.empty((vocab, dim), dtype=hidden.dtype, device=device)
            dweights = list(whole.split([t.shape[0] for t in weights]))
            dptrs = (_vp * p)(*[t.data_ptr() for t in dweights])
            a.dhidden, a.dweights = dhidden.data_ptr(), ctypes.addressof(dptrs)
        ws = _workspace(need, device)
        if ws is not None:
            a.workspace, a.workspace_bytes = ws.data_ptr(), need
        _abi._check(handle, lib.rar_vocab_xent(handle, ctypes.byref(a), raw))
        return VocabXent(loss, lse, dhidden, dweights)

    return _on_stream(stream, device, body)


def rar_embedding(handle, tables, tokens, scale=1.0, stream=None):
    """scale x rows of a table in p pieces, one for each token; zeros for a
    token outside the vocabulary (see rar_embedding in rar.h)."""
    torch = _torch()
    ptrs, stride, p, vocab, dim = _pieces("tables", tables)
    first = tables[0]
    device = first.device
    a = EmbeddingArgs()
    a.tables, a.table_stride, a.p, a.dtype = ctypes.addressof(ptrs), stride, p, _code(first)
    a.vocab, a.dim, a.scale = vocab, dim, scale
    a.tokens, a.index_bytes, a.n_tokens = _indices("tokens", tokens, device)

    def body(raw):
        out = torch.empty((tokens.shape[0], dim), dtype=first.dtype, device=device)
        a.out = out.data_ptr()
        _abi._check(handle, _abi.load_library().rar_embedding(handle, ctypes.byref(a), raw))
        return out

    return _on_stream(stream, device, body)


def rar_embedding_grad(handle, dout, tokens, dtables, scale=1.0, accumulate=False, stream=None):
    """Gradient of rar_embedding for its table, into the p pieces `dtables`:
    added to them with accumulate=True, else written whole.  Returns dtables."""
    ptrs, stride, p, vocab, dim = _pieces("dtables", dtables, dout)
    device = dout.device
    a = EmbeddingGradArgs()
    a.dout, a.dout_stride = _matrix("dout", dout, None, dim)
    a.tokens, a.index_bytes, a.n_tokens = _indices("tokens", tokens, device)
    if dout.shape[0] != tokens.shape[0]:
        raise ValueError("dout must have one row per token")
    a.dtables, a.dtable_stride, a.p, a.dtype = ctypes.addressof(ptrs), stride, p, _code(dout)
    a.vocab, a.dim, a.scale, a.accumulate = vocab, dim, scale, 1 if accumulate else 0
    lib = _abi.load_library()
    need = lib.rar_embedding_grad_workspace(tokens.shape[0], vocab, dim)

    def body(raw):
        ws = _workspace(need, device)
        if ws is not None:
            a.workspace, a.workspace_bytes = ws.data_ptr(), need
        _abi._check(handle, lib.rar_embedding_grad(handle, ctypes.byref(a), raw))
        return dtables

    return _on_stream(stream, device, body)

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
import struct
from array import array
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


def _packer(cls):
    """struct.Struct of a ctypes structure: filling one costs a tenth of
    setting its fields."""
    codes = {_vp: "P", _sz: "N", _i32: "i", _f32: "f"}
    fmt = "@" + "".join(codes[kind] for _, kind in cls._fields_)
    packer = struct.Struct(fmt + "0P")
    assert packer.size == ctypes.sizeof(cls)
    return packer.pack


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


_pack_norm, _pack_norm_grad, _pack_xent, _pack_embed, _pack_embed_grad = map(
    _packer, (RmsNormArgs, RmsNormGradArgs, VocabXentArgs, EmbeddingArgs, EmbeddingGradArgs))


def declare(lib) -> None:
    """Argument types of the operators' C functions; their structs go as packed bytes or by reference."""
    for name in ("rar_add_rmsnorm", "rar_add_rmsnorm_grad", "rar_vocab_xent", "rar_embedding", "rar_embedding_grad"):
        f = getattr(lib, name)
        f.argtypes = [_vp, _vp, _vp]
        f.restype = _i32
    for name, argtypes in (("rar_add_rmsnorm_grad_workspace", [_sz, _sz]),
                           ("rar_vocab_xent_workspace", [_sz, _sz, _sz, _i32, _i32]),
                           ("rar_embedding_grad_workspace", [_sz, _sz, _sz])):
        f = getattr(lib, name)
        f.argtypes = argtypes
        f.restype = _sz


def _stride(name, t):
    """Row stride of a matrix whose rows are contiguous."""
    if t.is_contiguous():
        return t.shape[1]
    st, (rows, cols) = t.stride(), t.shape
    if cols > 1 and st[1] != 1:
        raise ValueError(f"{name} must have contiguous rows")
    return st[0] if rows > 1 else cols


def _matrix(name, t, shape, dtype, device):
    """(pointer, row stride) of a CUDA matrix of this shape."""
    if t.shape != shape or t.dtype is not dtype or t.get_device() != device:
        raise ValueError(f"{name} must be a {tuple(shape)} {dtype} tensor on device {device}, got {tuple(t.shape)} "
                         f"{t.dtype} on {t.device}")
    return t.data_ptr(), _stride(name, t)


def _vector(name, t, n, dtype, device):
    if t.shape != (n,) or t.dtype is not dtype or t.get_device() != device or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous vector of {n} {dtype} values on device {device}")
    return t.data_ptr()


def _indices(name, t, n, device):
    size = _index_bytes().get(t.dtype)
    if size is None or t.dim() != 1 or (n is not None and t.shape[0] != n) or t.get_device() != device or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous vector of int32 or int64 values on device {device}"
                         + (f", one for each of {n} rows" if n is not None else ""))
    return t.data_ptr(), size


def _first(name, t):
    """(dtype, its code, device index) that a call's matrices share."""
    code = _codes().get(t.dtype)
    device = t.get_device()
    if code is None:
        raise ValueError(f"unsupported dtype {t.dtype}")
    if device < 0:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dim() != 2:
        raise ValueError(f"{name} must have two dimensions")
    return t.dtype, code, device


def _matrices(name, tensors, dtype, device, shapes):
    """(array of pointers, row stride) of matrices with one row stride, which
    those of a single row do not decide."""
    ptrs, stride = array("Q"), 0
    for r, t in enumerate(tensors):
        if t.shape != shapes[r] or t.dtype is not dtype or t.get_device() != device:
            raise ValueError(f"{name} {r} must be a {tuple(shapes[r])} {dtype} tensor on device {device}, got "
                             f"{tuple(t.shape)} {t.dtype} on {t.device}")
        ptrs.append(t.data_ptr())
        if t.is_contiguous():
            st = shapes[r][1]
        else:
            st = _stride(f"{name} {r}", t)
        if st != stride and shapes[r][0] > 1:
            if stride:
                raise ValueError(f"{name}s must share their row stride")
            stride = st
    return ptrs, stride


def _pieces(name, pieces, dtype, device):
    """(pointer array, row stride, p, vocab, dim) of a matrix in pieces by
    chunk_bounds: the first vocab mod p pieces are one row longer."""
    p = len(pieces)
    dim = pieces[0].shape[-1]
    vocab = 0
    for t in pieces:
        vocab += t.shape[0]
    base, extra = divmod(vocab, p)
    ptrs, stride = _matrices(name, pieces, dtype, device, [(base + 1, dim)] * extra + [(base, dim)] * (p - extra))
    return ptrs, stride, p, vocab, dim


@functools.lru_cache(maxsize=None)
def _current_stream():
    """Raw handle of a device's current stream."""
    torch = _torch()
    raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
    return raw or (lambda device: torch.cuda.current_stream(device).cuda_stream)


@contextlib.contextmanager
def _external(stream, device):
    torch = _torch()
    s = torch.cuda.ExternalStream(stream, device=device) if isinstance(stream, int) else stream
    with torch.cuda.stream(s):
        yield s.cuda_stream


def _on_stream(stream, device, body):
    """body(raw stream), with results allocated on that stream."""
    if stream is None:
        return body(_current_stream()(device))
    with _external(stream, device) as raw:
        return body(raw)


def _check(handle, rc):
    if rc:
        _abi._check(handle, rc)


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
    dtype, code, device = _first("a part", x)
    shape = x.shape
    rows, dim = shape
    p = len(parts)
    ptrs, stride = _matrices("part", parts, dtype, device, [shape] * p)
    res, res_stride = _matrix("residual", residual, shape, dtype, device) if residual is not None else (0, 0)
    w = _vector("weight", weight, dim, dtype, device) if weight is not None else 0
    group = quant_group or 0
    if group < 0:
        raise ValueError("quant_group must be None, 0 or positive")

    def body(raw):
        s = torch.empty(shape, dtype=dtype, device=x.device)
        rstd = torch.empty(rows, dtype=torch.float32, device=x.device)
        out = out8 = scales = None
        out_p = out8_p = scales_p = 0
        if quant_group is None or keep_out:
            out = torch.empty_like(s)
            out_p = out.data_ptr()
        if quant_group is not None:
            out8 = torch.empty_like(s, dtype=torch.float8_e4m3fn)
            scales = torch.empty((rows, -(-dim // group) if group else 1), dtype=torch.float32, device=x.device)
            out8_p, scales_p = out8.data_ptr(), scales.data_ptr()
        args = _pack_norm(ptrs.buffer_info()[0], p, code, rows, dim, stride, res, res_stride, w, eps, s.data_ptr(), 0,
                          out_p, 0, rstd.data_ptr(), out8_p, 0, scales_p, group)
        _check(handle, _abi.load_library().rar_add_rmsnorm(handle, args, raw))
        return AddRmsNorm(s, rstd, out, out8, scales)

    return _on_stream(stream, device, body)


def rar_add_rmsnorm_grad(handle, dout, sum, rstd, weight=None, dsum=None, stream=None):
    """(dx, dweight) of rar_add_rmsnorm: dx is the gradient of the residual
    and of every part alike.  sum and rstd are its results; dsum is the
    gradient of its sum, if that is used elsewhere."""
    torch = _torch()
    dtype, code, device = _first("dout", dout)
    shape = dout.shape
    rows, dim = shape
    x, x_stride = _matrix("sum", sum, shape, dtype, device)
    r = _vector("rstd", rstd, rows, torch.float32, device)
    ds, ds_stride = _matrix("dsum", dsum, shape, dtype, device) if dsum is not None else (0, 0)
    w = _vector("weight", weight, dim, dtype, device) if weight is not None else 0
    dout_stride = _stride("dout", dout)
    lib = _abi.load_library()
    need = lib.rar_add_rmsnorm_grad_workspace(rows, dim)

    def body(raw):
        dx = torch.empty(shape, dtype=dtype, device=dout.device)
        dweight = torch.empty(dim, dtype=dtype, device=dout.device)
        ws = torch.empty(need, dtype=torch.uint8, device=dout.device)
        args = _pack_norm_grad(code, rows, dim, dout.data_ptr(), dout_stride, ds, ds_stride, x, x_stride, r, w,
                               dx.data_ptr(), 0, dweight.data_ptr(), ws.data_ptr(), need)
        _check(handle, lib.rar_add_rmsnorm_grad(handle, args, raw))
        return dx, dweight

    return _on_stream(stream, device, body)


def rar_vocab_xent(handle, hidden, weights, targets, token_weight=None, grad=False, stream=None) -> VocabXent:
    """Softmax cross entropy of `hidden` (tokens x dim, bfloat16 or float16)
    against a vocabulary in p pieces, without keeping the logits (see
    rar_vocab_xent in rar.h).  A target outside the vocabulary leaves its
    token out.  grad=True also returns the gradients of
    sum(token_weight * loss) for hidden and for every piece."""
    torch = _torch()
    if len(weights) < 1:
        raise ValueError("need at least one piece")
    dtype, code, device = _first("hidden", hidden)
    ptrs, wstride, p, vocab, dim = _pieces("weight piece", weights, dtype, device)
    tokens = hidden.shape[0]
    hid, hid_stride = _matrix("hidden", hidden, (tokens, dim), dtype, device)
    tgt, index_bytes = _indices("targets", targets, tokens, device)
    tw = _vector("token_weight", token_weight, tokens, torch.float32, device) if token_weight is not None else 0
    lib = _abi.load_library()
    need = lib.rar_vocab_xent_workspace(tokens, dim, vocab, p, 1 if grad else 0)

    def body(raw):
        loss = torch.empty(tokens, dtype=torch.float32, device=hidden.device)
        lse = torch.empty_like(loss)
        ws = torch.empty(need, dtype=torch.uint8, device=hidden.device)
        dhidden = dweights = None
        dh_p = dw_p = 0
        if grad:
            dhidden = torch.empty((tokens, dim), dtype=dtype, device=hidden.device)
            whole = torch.empty((vocab, dim), dtype=dtype, device=hidden.device)
            dweights = list(whole.split([t.shape[0] for t in weights]))
            dptrs = array("Q", [t.data_ptr() for t in dweights])
            dh_p, dw_p = dhidden.data_ptr(), dptrs.buffer_info()[0]
        args = _pack_xent(hid, hid_stride, ptrs.buffer_info()[0], wstride, p, code, tokens, dim, vocab, tgt, index_bytes,
                          tw, loss.data_ptr(), lse.data_ptr(), dh_p, 0, dw_p, 0, ws.data_ptr(), need)
        _check(handle, lib.rar_vocab_xent(handle, args, raw))
        return VocabXent(loss, lse, dhidden, dweights)

    return _on_stream(stream, device, body)


def rar_embedding(handle, tables, tokens, scale=1.0, stream=None):
    """scale x rows of a table in p pieces, one for each token; zeros for a
    token outside the vocabulary (see rar_embedding in rar.h)."""
    torch = _torch()
    if len(tables) < 1:
        raise ValueError("need at least one piece")
    first = tables[0]
    dtype, code, device = _first("a table piece", first)
    ptrs, stride, p, vocab, dim = _pieces("table piece", tables, dtype, device)
    tok, index_bytes = _indices("tokens", tokens, None, device)
    n = tokens.shape[0]

    def body(raw):
        out = torch.empty((n, dim), dtype=dtype, device=first.device)
        args = _pack_embed(ptrs.buffer_info()[0], stride, p, code, vocab, dim, tok, index_bytes, n, scale, out.data_ptr(), 0)
        _check(handle, _abi.load_library().rar_embedding(handle, args, raw))
        return out

    return _on_stream(stream, device, body)


def rar_embedding_grad(handle, dout, tokens, dtables, scale=1.0, accumulate=False, stream=None):
    """Gradient of rar_embedding for its table, into the p pieces `dtables`:
    added to them with accumulate=True, else written whole.  Returns dtables."""
    torch = _torch()
    if len(dtables) < 1:
        raise ValueError("need at least one piece")
    dtype, code, device = _first("dout", dout)
    ptrs, stride, p, vocab, dim = _pieces("gradient piece", dtables, dtype, device)
    n = dout.shape[0]
    do, do_stride = _matrix("dout", dout, (n, dim), dtype, device)
    tok, index_bytes = _indices("tokens", tokens, n, device)
    lib = _abi.load_library()
    need = lib.rar_embedding_grad_workspace(n, vocab, dim)

    def body(raw):
        ws = torch.empty(need, dtype=torch.uint8, device=dout.device)
        args = _pack_embed_grad(do, do_stride, tok, index_bytes, n, ptrs.buffer_info()[0], stride, p, code, vocab, dim,
                                scale, 1 if accumulate else 0, ws.data_ptr(), need)
        _check(handle, lib.rar_embedding_grad(handle, args, raw))
        return dtables

    return _on_stream(stream, device, body)

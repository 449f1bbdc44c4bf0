"""Python binding of the model operators in include/rar.h (rar_add_rmsnorm,
rar_vocab_xent, rar_embedding and their gradients).

The functions check their tensors, allocate results and workspaces with
torch's caching allocator on the stream that the call runs on, and call the C
functions: that part is the compiled module _torch_ops (csrc/torch_ops.cpp),
which is built with the library; there is no other path.  Tensors that a call
takes must be ready on its stream, as for every call of this package; `stream`
is a torch stream or an integer of the tensors' device.  Matrices have
contiguous rows that do not overlap: an expanded one has to be copied first.

The ctypes structures below mirror the C ones, for callers with results of
their own: load_library().rar_add_rmsnorm(handle, ctypes.byref(args), stream).
"""
from __future__ import annotations

import ctypes
import functools
import importlib.machinery
import importlib.util
import os
from typing import NamedTuple, Optional

from . import _abi, _build

_vp, _sz, _i32, _f32 = ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int, ctypes.c_float


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


@functools.lru_cache(maxsize=None)
def _module():
    """The compiled module (torch is imported with its first use)."""
    import torch  # noqa: F401  (its libraries first)
    _abi.load_library()
    path = _build.TORCH_OPS_PATH
    if not os.path.exists(path):
        lacks = _build.binding_lacks()
        raise RuntimeError(f"{path} is missing: " + (f"it cannot be built without {lacks}" if lacks else
                           "build the library first (python -c 'import __graft_entry__ as g; g.build()')"))
    loader = importlib.machinery.ExtensionFileLoader("_torch_ops", path)
    module = importlib.util.module_from_spec(importlib.util.spec_from_loader("_torch_ops", loader))
    loader.exec_module(module)
    return module


def _run(handle, stream, function, *args):
    """function(handle, *args) with `stream`, which belongs to the device of the
    tensors (args[0], a tensor or several), as the current stream; its results."""
    if stream is None:
        r = function(handle, *args)
    else:
        import torch
        first = args[0][0] if isinstance(args[0], (list, tuple)) and args[0] else args[0]
        device = getattr(first, "device", None)
        if getattr(device, "type", None) != "cuda":
            raise ValueError("the operators take CUDA tensors")
        s = torch.cuda.ExternalStream(stream, device=device) if isinstance(stream, int) else stream
        if s.device != device:
            raise ValueError(f"the stream belongs to {s.device}, the tensors are on {device}")
        with torch.cuda.stream(s):
            r = function(handle, *args)
    if type(r) is int:
        _abi._check(handle, r)
    return r


def rar_add_rmsnorm(handle, parts, weight=None, residual=None, eps=1e-6, quant_group=None, keep_out=False,
                    stream=None) -> AddRmsNorm:
    """s = residual + sum of the p parts, y = s / rms(s) * weight (see
    rar_add_rmsnorm in rar.h).  parts: p matrices rows x dim of one dtype.
    quant_group None: y is returned in the parts' dtype.  0 or a multiple of
    32: y is returned as float8_e4m3fn codes with a float32 scale per row, or
    per row and run of quant_group columns; keep_out=True keeps `out` as well."""
    return AddRmsNorm._make(_run(handle, stream, _module().add_rmsnorm, parts, weight, residual, eps,
                                 -1 if quant_group is None else quant_group, keep_out))


def rar_add_rmsnorm_grad(handle, dout, sum, rstd, weight=None, dsum=None, stream=None):
    """(dx, dweight) of rar_add_rmsnorm: dx is the gradient of the residual
    and of every part alike.  sum and rstd are its results; dsum is the
    gradient of its sum, if that is used elsewhere."""
    return _run(handle, stream, _module().add_rmsnorm_grad, dout, sum, rstd, weight, dsum)


def rar_vocab_xent(handle, hidden, weights, targets, token_weight=None, grad=False, stream=None) -> VocabXent:
    """Softmax cross entropy of `hidden` (tokens x dim, bfloat16 or float16)
    against a vocabulary in p pieces, without keeping the logits (see
    rar_vocab_xent in rar.h).  A target outside the vocabulary leaves its
    token out.  grad=True also returns the gradients of
    sum(token_weight * loss) for hidden and for every piece."""
    return VocabXent._make(_run(handle, stream, _module().vocab_xent, hidden, weights, targets, token_weight, grad))


def rar_embedding(handle, tables, tokens, scale=1.0, stream=None):
    """scale x rows of a table in p pieces, one for each token; zeros for a
    token outside the vocabulary (see rar_embedding in rar.h)."""
    return _run(handle, stream, _module().embedding, tables, tokens, scale)[0]


def rar_embedding_grad(handle, dout, tokens, dtables, scale=1.0, accumulate=False, stream=None):
    """Gradient of rar_embedding for its table, into the p pieces `dtables`:
    added to them with accumulate=True, else written whole.  Returns dtables."""
    _run(handle, stream, _module().embedding_grad, dout, tokens, dtables, scale, accumulate)
    return dtables

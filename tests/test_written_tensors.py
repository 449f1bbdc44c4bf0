"""Tensors that a call writes where they lie, and what autograd learns of it."""
import ctypes

import pytest
import torch

import ring_all_reduce_rar_gb300 as rar
from ring_all_reduce_rar_gb300 import _ops
from tests.test_model_ops import DTYPES, gen, h, normal  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows,cols,gap", [(1, 1000003, 0), (37, 8200, 3), (3001, 65, 7), (9000, 31, 2)])
def test_clipping_in_place_is_as_apart(h, dtype, rows, cols, gap):  # noqa: F811
    """Rows that begin anywhere in a vector, the threads' accesses side by side with their neighbours'."""
    for lead in (0, 1, 3):
        flat = normal(gen(rows), rows * (cols + gap) + lead, dtype=dtype)
        x = flat[lead:].view(rows, cols + gap)[:, :cols]
        apart = torch.empty(rows, cols, dtype=dtype, device="cuda")
        norm = h.grad_clip([x], 0.7, out=[apart])
        kept = flat.clone()
        assert torch.equal(h.grad_clip([x], 0.7), norm)
        assert torch.equal(x, apart)
        kept[lead:].view(rows, cols + gap)[:, :cols] = apart
        assert torch.equal(flat, kept)
    h.check()


def test_autograd_refuses_values_that_were_scaled(h):  # noqa: F811
    """A value that a backward pass still needs is not used after it changed."""
    for write in (lambda t: h.grad_clip([t], 0.1), lambda t: h.grad_clip([torch.ones(50, device="cuda")], 0.1, out=[t]),
                  lambda t: h.grad_clip([t.view(5, 10)[:, :4]], 0.1)):
        x = torch.ones(50, device="cuda", requires_grad=True)
        kept = x * 2.0
        loss = (kept * kept).sum()
        before = kept._version
        write(kept.detach())
        assert kept._version > before
        with pytest.raises(RuntimeError, match="modified by an inplace operation"):
            loss.backward()


def test_tensors_that_are_read_keep_their_version(h):  # noqa: F811
    x, out, norm = torch.ones(50, device="cuda"), torch.empty(50, device="cuda"), torch.ones((), device="cuda")
    versions = x._version, norm._version
    h.grad_norm([x])
    h.grad_clip([x], 0.1, norm=norm, out=[out])
    assert (x._version, norm._version) == versions
    with pytest.raises(ValueError):
        h.grad_clip([x], -1.0)
    with pytest.raises(rar.RarError):
        h.grad_clip([x, x], 1.0)
    assert x._version == versions[0]
    # (tensors made for inference have no version)
    with torch.inference_mode():
        y = torch.full((50,), 2.0, device="cuda")
    h.grad_clip([y], 1.0)
    assert abs(float(torch.linalg.vector_norm(y)) - 1) < 1e-5


def test_a_table_gradient_that_is_added_to(h):  # noqa: F811
    g = gen(3)
    tables = [torch.zeros(20, 16, device="cuda") for _ in range(2)]
    before = [t._version for t in tables]
    h.embedding_grad(normal(g, 7, 16), torch.arange(7, device="cuda"), tables, accumulate=True)
    assert all(t._version > v for t, v in zip(tables, before))


@pytest.mark.parametrize("stride,out_stride", [(0, 40), (40, 0), (40, 64), (1 << 40, 40)])
def test_one_row_in_place_with_any_stride(h, stride, out_stride):  # noqa: F811
    x = normal(gen(1), 40)
    norm = torch.linalg.vector_norm(x).reshape(1)
    want = x * (0.5 / norm)
    tensors, out = (_ops.Tensor(x.data_ptr(), 1, 1, 40, s) for s in (stride, out_stride))
    a = _ops.GradClipArgs()
    a.tensors, a.n, a.out = ctypes.addressof(tensors), 1, ctypes.addressof(out)
    a.norm, a.max_norm, a.eps = norm.data_ptr(), 0.5, 0.0
    lib, stream = rar.load_library(), torch.cuda.current_stream().cuda_stream
    assert lib.rar_grad_clip(h.h, ctypes.byref(a), stream) == 0, rar.rar_last_error(h.h)
    # (the quotient and the product are rounded)
    assert bool(((x.double() - want.double()).abs() <= 4 * 2.0 ** -24 * want.double().abs()).all())
    h.check()


@pytest.mark.parametrize("residual_stride,sum_stride", [(0, 40), (40, 64), (1 << 40, 0)])
def test_a_residual_of_one_row_is_written_with_any_stride(h, residual_stride, sum_stride):  # noqa: F811
    g = gen(2)
    part, residual = normal(g, 1, 40), normal(g, 1, 40)
    want = h.add_rmsnorm([part], residual=residual).sum
    ptrs = (ctypes.c_void_p * 1)(part.data_ptr())
    a = _ops.RmsNormArgs()
    a.parts, a.p, a.dtype, a.rows, a.dim = ctypes.addressof(ptrs), 1, 1, 1, 40
    a.residual, a.residual_stride, a.sum, a.sum_stride = residual.data_ptr(), residual_stride, residual.data_ptr(), sum_stride
    lib, stream = rar.load_library(), torch.cuda.current_stream().cuda_stream
    assert lib.rar_add_rmsnorm(h.h, ctypes.byref(a), stream) == 0, rar.rar_last_error(h.h)
    assert torch.equal(residual, want)
    h.check()

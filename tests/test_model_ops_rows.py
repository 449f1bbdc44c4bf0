"""The residual norm and its gradient on many rows (rows brought ahead by bulk
copies) and on rows that begin anywhere in a 16-byte vector, against the 64-bit forms
and bounds of test_model_ops."""
import ctypes

import pytest
import torch

import ring_all_reduce_rar_gb300 as rar
from ring_all_reduce_rar_gb300 import _ops
from tests.test_model_ops import (DTYPES, check_norm, check_norm_grad, gen, h, norm_reference, normal,  # noqa: F401
                                  strided)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("p,rows,dim,group,plain", [
    (1, 2500, 1024, 128, False), (8, 2500, 1024, None, False), (3, 2501, 2048, 0, False), (8, 1300, 4096, 128, False),
    (2, 700, 8192, 96, False), (7, 1231, 4096, None, True), (16, 2500, 1024, 128, True), (5, 2433, 1536, 64, False),
    (64, 611, 1024, 0, False), (33, 1300, 1024, 32, False),
])
def test_many_rows(h, dtype, p, rows, dim, group, plain):  # noqa: F811
    g = gen(rows * 3 + p)
    parts = [normal(g, rows, dim, dtype=dtype) for _ in range(p)]
    residual = None if plain else normal(g, rows, dim, dtype=dtype, std=2.0)
    weight = None if plain else normal(g, dim, dtype=dtype)
    r = h.add_rmsnorm(parts, weight, residual=residual, eps=1e-5, quant_group=group, keep_out=True)
    check_norm(r, dtype, norm_reference(parts, residual, weight, 1e-5), group)
    again = h.add_rmsnorm(parts, weight, residual=residual, eps=1e-5, quant_group=group, keep_out=True)
    for x, y in zip(r, again):
        assert x is None or torch.equal(x.view(torch.uint8), y.view(torch.uint8))
    h.check()


@pytest.mark.parametrize("p,rows,dim", [(7, 2500, 1024), (3, 1231, 2052), (11, 700, 4100)])
def test_many_rows_have_the_rings_order(h, p, rows, dim):  # noqa: F811
    """Chunk boundaries inside rows, and inside vectors."""
    g = gen(p)
    parts = [normal(g, rows, dim) for _ in range(p)]
    r = h.add_rmsnorm(parts)
    copies = [t.clone() for t in parts]
    h.allreduce(copies)
    assert torch.equal(r.sum, copies[0])


@pytest.mark.parametrize("dtype", DTYPES)
def test_many_rows_in_place_and_strided(h, dtype):  # noqa: F811
    g = gen(77)
    p, rows, dim = 4, 1400, 2048
    parts = [strided(normal(g, rows, dim, dtype=dtype), 16) for _ in range(p)]
    residual = strided(normal(g, rows, dim, dtype=dtype), 32)
    expect = h.add_rmsnorm(parts, residual=residual)
    check_norm(expect, dtype, norm_reference(parts, residual, None, 1e-6), None)
    a = _ops.RmsNormArgs()
    ptrs = (ctypes.c_void_p * p)(*[t.data_ptr() for t in parts])
    a.parts, a.p, a.dtype, a.rows, a.dim, a.eps = ctypes.addressof(ptrs), p, rar.DTYPE_CODES[str(dtype)[6:]], rows, dim, 1e-6
    a.part_stride, a.residual_stride, a.sum_stride, a.out_stride = dim + 16, dim + 32, dim + 32, dim + 16
    a.residual = a.sum = residual.data_ptr()
    a.out = parts[2].data_ptr()
    assert rar.load_library().rar_add_rmsnorm(h.h, ctypes.byref(a), torch.cuda.current_stream().cuda_stream) == 0
    assert torch.equal(residual, expect.sum) and torch.equal(parts[2], expect.out)
    h.check()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("p,rows,dim,group", [
    (5, 700, 1001, 128), (3, 333, 4097, None), (8, 9, 2047, 32), (2, 64, 9001, 0), (1, 2000, 65, 64), (4, 31, 777, 0),
    (9, 40, 1027, 96), (1, 1, 3, 32), (6, 1500, 515, None),
])
def test_odd_rows(h, dtype, p, rows, dim, group):  # noqa: F811
    g = gen(rows + dim)
    parts = [normal(g, rows, dim, dtype=dtype) for _ in range(p)]
    residual, weight = normal(g, rows, dim, dtype=dtype, std=2.0), normal(g, dim, dtype=dtype)
    r = h.add_rmsnorm(parts, weight, residual=residual, eps=1e-5, quant_group=group, keep_out=True)
    check_norm(r, dtype, norm_reference(parts, residual, weight, 1e-5), group)
    if dtype == torch.float32:
        codes = h.add_rmsnorm(parts, weight, residual=residual, eps=1e-5, quant_group=32, keep_out=True)
        q = codes.out / codes.scales.repeat_interleave(32, 1)[:, :dim]
        assert torch.equal(codes.out8.view(torch.uint8), q.to(torch.float8_e4m3fn).view(torch.uint8))
        plain = h.add_rmsnorm(parts)
        copies = [t.clone() for t in parts]
        h.allreduce(copies)
        assert torch.equal(plain.sum, copies[0])


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows,dim,plain", [
    (2500, 1024, False), (2433, 2048, True), (1300, 4096, False), (700, 8192, False), (1300, 1001, False), (700, 4097, True),
    (3, 1001, False), (2000, 67, False), (609, 9001, False), (5000, 264, False),
])
def test_gradient_of_many_and_odd_rows(h, dtype, rows, dim, plain):  # noqa: F811
    g = gen(rows + dim)
    s, dout = normal(g, rows, dim, dtype=dtype, std=2.0), normal(g, rows, dim, dtype=dtype)
    dsum = None if plain else normal(g, rows, dim, dtype=dtype)
    weight = None if plain else normal(g, dim, dtype=dtype)
    rstd = ((s.double() ** 2).mean(1) + 1e-6).rsqrt().float()
    dx, dweight = h.add_rmsnorm_grad(dout, s, rstd, weight, dsum=dsum)
    check_norm_grad(dx, dweight, dout, s, rstd, weight, dsum)
    again = h.add_rmsnorm_grad(dout, s, rstd, weight, dsum=dsum)
    assert torch.equal(dx, again[0]) and torch.equal(dweight, again[1])
    h.check()


def test_status_and_send_counts(h):  # noqa: F811
    """The status of a call whose waits all end is RAR_OK, and a later call's
    send counts are zeros."""
    g = gen(1)
    parts = [normal(g, 2500, 1024) for _ in range(2)]
    h.add_rmsnorm(parts)
    assert h.status() == 0 and h.send_counts(2) == [0, 0]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("accumulate", [False, True])
@pytest.mark.parametrize("lengths,dim", [
    ([1, 15, 16, 17, 31, 32, 33, 1, 47, 48, 49, 64], 72), ([16] * 9, 264), ([32, 16, 48], 24), ([5, 27, 32], 8),
    ([16, 1, 15, 300, 1, 2, 3], 1025), ([31, 1], 64), ([40, 8], 520), ([3000], 2056),
])
def test_runs_against_the_chunks(h, dtype, accumulate, lengths, dim):  # noqa: F811
    """Runs of equal tokens that begin and end anywhere in the chunks of 16,
    cover chunks, and end with the last token."""
    from tests.test_model_ops import check_embedding_grad, pieces
    g = gen(sum(lengths) + dim)
    for left_out in (0, 7):
        tok = torch.cat([torch.full((n,), 3 * k + 1, device="cuda") for k, n in enumerate(lengths)]
                        + [torch.full((left_out,), -5, device="cuda")])
        tok = tok[torch.randperm(len(tok), generator=g, device="cuda")]
        vocab = 3 * len(lengths) + 2
        dout = normal(g, len(tok), dim, dtype=dtype)
        old = normal(g, vocab, dim, dtype=dtype)
        into = old.clone()
        h.embedding_grad(dout, tok, pieces(into, 3), scale=0.5, accumulate=accumulate)
        check_embedding_grad(into, dout, tok, old if accumulate else None, vocab, 0.5)

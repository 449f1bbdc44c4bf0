"""The norm where a thread adds up many squares: long rows of matrices with gaps, large chunks, and the second pass over
values whose squares overflow or vanish in 32 bits.

Squares of normal values lie close to 0 more often than not, so that a long run of additions comes out low.  A thread adds at
most 18 squares one after the other (16 from its loads, an element at each end of a run), two more for its four
accumulators, the batches without a rounding but the last, then 5 + 8 partial sums of the CTA; the chunks' are added in
64 bits.  All are positive: the sum of squares is off by at most 34 F of itself (F = 2^-24), its root by half of
that, and by the rounding to 32 bits before it and its own: 18.5 F.
"""
import pytest
import torch

from tests.test_model_ops import DTYPES, F, gen, h  # noqa: F401

pytestmark = pytest.mark.gpu

TOL = 19 * F


def squares(t):
    """In 64 bits, some 2^25 elements at a time."""
    rows = max(1, (1 << 25) // t.shape[1]) if t.dim() == 2 else 1 << 25
    return float(sum(part.double().square().sum() for part in t.split(rows)))


def check(h, tensors):  # noqa: F811
    one = {id(t): squares(t) for t in tensors}
    r = h.grad_norm(tensors)
    for got, t in zip(r.norms.tolist(), tensors):
        assert abs(got / one[id(t)] ** 0.5 - 1) <= TOL
    want = sum(one[id(t)] for t in tensors) ** 0.5
    assert abs(float(r.norm) / want - 1) <= TOL
    h.check()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows,cols,gap,times", [(300, 1 << 18, 24, 8), (70, 65536, 8, 1), (2, 1000003, 5, 3)])
def test_long_rows_with_gaps(h, dtype, rows, cols, gap, times):  # noqa: F811
    """A tensor given several times counts several times: the chunks grow with it (the first: to 2^18 elements)."""
    x = torch.randn(rows, cols + gap, generator=gen(cols), device="cuda").to(dtype)[:, :cols]
    check(h, [x] * times)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("cols,gap", [(1 << 27, 0), (60, 4)])
def test_large_chunks(h, dtype, cols, gap):  # noqa: F811
    """Chunks of 2^20 elements and more, without gaps and in rows too short for a warp."""
    x = torch.randn((1 << 27) // cols, cols + gap, generator=gen(cols), device="cuda").to(dtype)[:, :cols]
    check(h, [x] * 33)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("cols,gap", [(1 << 27, 0), (8192, 8), (60, 4)])
def test_the_second_pass(h, dtype, cols, gap):  # noqa: F811
    """Squares that vanish, and that overflow, in chunks of 2^20 elements and more.  (fp16 knows no such values
    but below its normal ones, where a few bits are left: exact all the same.)"""
    for size in (2.0 ** -70, 2.0 ** 62) if dtype != torch.float16 else (2.0 ** -23,):
        x = (torch.randn((1 << 27) // cols, cols + gap, generator=gen(3), device="cuda") * size).to(dtype)[:, :cols]
        check(h, [x] * 33)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_infinities_and_nan_among_large_values(h, dtype):  # noqa: F811
    x = torch.full((30, 9000), 2.0 ** 100, dtype=dtype, device="cuda")
    for view in (x, x[:, :8000], x[:, :50]):
        y = view.clone() if view is x else view
        y[7, 33] = float("inf")
        assert float(h.grad_norm([y]).norm) == float("inf")
        y[7, 34] = float("nan")
        assert bool(h.grad_norm([y]).norm.isnan())
        y[7, 33], y[7, 34] = 2.0 ** 100, 1.0
    assert abs(float(h.grad_norm([x]).norm) / (2.0 ** 100 * (30 * 9000 - 1) ** 0.5) - 1) <= TOL

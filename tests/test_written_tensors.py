"""Tensors that a call writes where they lie."""
import pytest
import torch

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

"""What the model operators' calls refuse and what their host code decides
before a launch: matrices that torch holds in ways of its own, sizes far out of
range, calls from several threads, waits that run out."""
import pytest
import torch

import ring_all_reduce_rar_gb300 as rar
from tests.test_model_ops import DTYPES, gen, h, normal, pieces  # noqa: F401  (h is the fixture)

gpu = pytest.mark.gpu


# Every matrix of every call, by name; half types because all calls take them.
EXPANDED = ["part", "residual", "dout", "sum", "dsum", "hidden", "weight piece", "table piece", "lookup gradient", "gradient piece"]


@gpu
@pytest.mark.parametrize("shape", [(4, 64), (2, 8), (4, 1)])
@pytest.mark.parametrize("place", EXPANDED)
def test_expanded_matrices_are_refused(h, place, shape):  # noqa: F811
    """One row repeated by expand() lies in memory once: its row stride of 0
    must not pass for packed rows."""
    rows, dim = shape
    x = torch.ones(rows, dim, dtype=torch.bfloat16, device="cuda")
    e = torch.ones(1, dim, dtype=torch.bfloat16, device="cuda").expand(rows, dim)
    assert e.stride(0) == 0
    tok = torch.zeros(rows, dtype=torch.int64, device="cuda")
    rstd = torch.ones(rows, device="cuda")
    calls = {
        "part": lambda: h.add_rmsnorm([x, e]),
        "residual": lambda: h.add_rmsnorm([x], residual=e),
        "dout": lambda: h.add_rmsnorm_grad(e, x, rstd),
        "sum": lambda: h.add_rmsnorm_grad(x, e, rstd),
        "dsum": lambda: h.add_rmsnorm_grad(x, x, rstd, dsum=e),
        "hidden": lambda: h.vocab_xent(e, [x], tok),
        "weight piece": lambda: h.vocab_xent(x, [x, e], tok),
        "table piece": lambda: h.embedding([e, x], tok),
        "lookup gradient": lambda: h.embedding_grad(e, tok, [x.clone()]),
        "gradient piece": lambda: h.embedding_grad(x, tok, [e]),
    }
    with pytest.raises(ValueError, match="expanded"):
        calls[place]()


@gpu
def test_overlapping_rows_are_refused(h):  # noqa: F811
    memory = torch.ones(1024, dtype=torch.bfloat16, device="cuda")
    windows = memory.as_strided((8, 64), (16, 1))
    with pytest.raises(ValueError, match="overlap"):
        h.add_rmsnorm([windows])


@gpu
def test_one_expanded_row_is_a_row(h):  # noqa: F811
    """A single row has no distance to a next one, whatever its stride says."""
    x = normal(gen(3), 1, 64)
    one = x.as_strided((1, 64), (0, 1))
    assert torch.equal(h.add_rmsnorm([one]).out, h.add_rmsnorm([x]).out)

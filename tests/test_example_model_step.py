"""The example that runs the model operators together: its gradients against
torch's autograd in 64 bits, and a loss that falls."""
import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu


def _example():
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "model_step.py")
    spec = importlib.util.spec_from_file_location("model_step", path)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


def _norm(x, w):
    return x * torch.rsqrt((x * x).mean(1, keepdim=True) + 1e-6) * w


@pytest.mark.parametrize("ranks", [1, 4])
def test_gradients_against_autograd(ranks):
    """Each tensor that a gradient passes through is rounded to 8 bits (2^-8 of
    an element): the chain from the loss back to the table holds fewer than 16
    such roundings, which add up, in the norm, to less than 16 x 2^-8."""
    ex = _example()
    model = ex.Model(ranks, vocab=503, dim=128, inner=256)
    tokens = torch.randint(0, 503, (77,), generator=torch.Generator().manual_seed(5)).cuda()
    targets = tokens.roll(-1)
    loss, grads = model.gradients(tokens, targets)
    wide = [p.double().requires_grad_() for p in model.params]
    table = torch.cat(wide[:ranks])
    x0 = table[tokens] * model.table_scale
    n0 = _norm(x0, wide[-2])
    x1 = x0 + sum(model.rank_part(n0, wide[ranks + 2 * r], wide[ranks + 2 * r + 1]) for r in range(ranks))
    want = torch.nn.functional.cross_entropy(_norm(x1, wide[-1]) @ table.t(), targets)
    want.backward()
    # hidden states with an error of a few 2^-8 move a logit of size ~1 by as much
    assert abs(loss.item() - want.item()) <= 16 * 2 ** -8
    for got, p in zip(grads, wide):
        assert (got.double() - p.grad).norm() <= 16 * 2 ** -8 * p.grad.norm()
    model.handle.check()


def test_loss_falls():
    losses, scores = _example().run(ranks=3, steps=30)
    assert losses[-1] < losses[0] - 1.0
    # 8-bit hidden states (3 bits after the point: 2^-4 of an element) keep the mean loss
    assert abs(scores.mean().item() - losses[-1]) < 0.5

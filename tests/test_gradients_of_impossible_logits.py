"""Gradients of log probabilities where a logit is -infinity, or so low that its product with the scale is: its
probability is 0, and so is p log p, in the limit.  Bounds as in test_vocab_logprobs."""
import math

import pytest
import torch

from tests.test_model_ops import HALF, TINY, U, gen, h, normal, pieces, within, xent_inputs  # noqa: F401
from tests.test_vocab_logprobs import grad_reference

pytestmark = pytest.mark.gpu

# (G in two rows, in one row; logits in one sum, in several)
SHAPES = [(3, 3, 64), (3, 130, 64), (2, 600, 64), (3, 40, 1096), (2, 600, 1096)]
LOW, HIGH, VOCAB = 100, 300, 700


def inputs(p, tokens, dim, dtype):
    g = gen(tokens + dim)
    whole, hidden, targets = xent_inputs(g, tokens, dim, VOCAB, dtype)
    hidden = hidden.abs() + 0.25
    targets = torch.where(targets < 0, targets, targets % LOW)
    return whole, hidden, targets, normal(g, tokens) / tokens, normal(g, tokens, std=0.1) / tokens


@pytest.mark.parametrize("dtype", HALF)
@pytest.mark.parametrize("p,tokens,dim", SHAPES)
@pytest.mark.parametrize("lowest", [True, False])
def test_rows_without_a_share(h, dtype, p, tokens, dim, lowest):  # noqa: F811
    """lowest: rows of the type's lowest value, which products with G's zeros leave finite; else one
    column of -infinity, in which dhidden has 0 x infinity."""
    whole, hidden, targets, a, b = inputs(p, tokens, dim, dtype)
    gone = whole.clone()
    if lowest:
        gone[LOW:HIGH] = torch.finfo(dtype).min
    else:
        gone[LOW:HIGH, 9] = -float("inf")
    rest = torch.cat([whole[:LOW], whole[HIGH:]])
    keep = torch.ones(dim, dtype=torch.bool, device="cuda")
    keep[9] = lowest
    r = h.vocab_logprobs(hidden, pieces(gone, p), targets)
    assert bool(r.lse.isfinite().all()) and bool(r.entropy.isfinite().all())
    for da, db in ((a, None), (a, b), (None, b)):
        dh, dw = h.vocab_logprobs_grad(hidden, pieces(gone, p), targets, r.lse, r.entropy, da, dentropy=db)
        dw = torch.cat(dw)
        assert bool((dw[LOW:HIGH] == 0).all())
        ref = grad_reference(hidden, [rest], targets, r.lse, r.entropy, da, db, 1.0)
        within(torch.cat([dw[:LOW], dw[HIGH:]]), *ref[1], "dweights")
        within(dh[:, keep], ref[0][0][:, keep], ref[0][1][:, keep], "dhidden")
    # the cross entropy of the same rows, whose G is that of a = -token_weight
    weight = a.abs()
    x = h.vocab_xent(hidden, pieces(gone, p), targets, token_weight=weight, grad=True)
    dh, dw = h.vocab_logprobs_grad(hidden, pieces(gone, p), targets, x.lse, None, -weight)
    assert bool((torch.cat(x.dweights)[LOW:HIGH] == 0).all()) and bool((torch.cat(dw)[LOW:HIGH] == 0).all())
    h.check()


@pytest.mark.parametrize("dtype", HALF)
@pytest.mark.parametrize("p,tokens,dim", SHAPES)
def test_an_impossible_target(h, dtype, p, tokens, dim):  # noqa: F811
    """G is a at a target with probability 0, with or without an entropy's gradient."""
    whole, hidden, targets, a, b = inputs(p, tokens, dim, dtype)
    whole[LOW:HIGH, 9] = -float("inf")
    targets[::2] = LOW + 50
    aims = targets == LOW + 50
    r = h.vocab_logprobs(hidden, pieces(whole, p), targets)
    assert bool((r.logprob[aims] == -float("inf")).all())
    for db in (None, b):
        dw = torch.cat(h.vocab_logprobs_grad(hidden, pieces(whole, p), targets, r.lse, r.entropy, a, dentropy=db)[1])
        share = a[aims].double()[:, None] * hidden[aims].double()
        # G and the sum are rounded to the type, the sum's additions to 32 bits; what is below G's steps
        most = float((a.abs() + b.abs() * r.entropy.abs().clamp(min=1)).max())
        bound = (2.1 * U[dtype] + 2.0 ** -20) * share.abs().sum(0) + most * 2.0 ** -37 * hidden.double().abs().sum(0) + TINY[dtype]
        within(dw[LOW + 50], share.sum(0), bound, "dweights")
        others = torch.cat([dw[LOW:LOW + 50], dw[LOW + 51:HIGH]])
        assert bool((others == 0).all())


@pytest.mark.parametrize("dtype", HALF)
@pytest.mark.parametrize("tokens", [5, 150, 600])
def test_logits_that_overflow_with_the_scale(h, dtype, tokens):  # noqa: F811
    """Two logits of 0, all others below -2^9, with a scale of 2^126."""
    g = gen(tokens)
    scale, vocab, dim = 2.0 ** 126, 600, 16
    hidden = torch.randint(1, 5, (tokens, dim), generator=g, device="cuda").to(dtype)
    whole = torch.zeros(vocab, dim, dtype=dtype, device="cuda")
    whole[2:, 0] = -1024.0
    targets = torch.randint(0, 2, (tokens,), generator=g, device="cuda")
    # (weights that leave the gradients within the type)
    size = 2.0 ** (-60 if dtype == torch.bfloat16 else -120)
    a, b = normal(g, tokens) * size, normal(g, tokens) * size
    r = h.vocab_logprobs(hidden, pieces(whole, 2), targets, logit_scale=scale)
    assert bool(((r.lse.double() - math.log(2)).abs() < 2.0 ** -20).all())
    for da, db in ((a, None), (a, b), (None, b)):
        dh, dw = h.vocab_logprobs_grad(hidden, pieces(whole, 2), targets, r.lse, r.entropy, da, dentropy=db, logit_scale=scale)
        dw = torch.cat(dw)
        ref = grad_reference(hidden, [whole[:2]], targets, r.lse, r.entropy, da, db, scale)
        within(dw[:2], *ref[1], "dweights")
        assert bool((dw[2:] == 0).all()) and bool((dh == 0).all())
    h.check()


@pytest.mark.parametrize("dtype", HALF)
@pytest.mark.parametrize("p,tokens,dim", SHAPES)
def test_a_logit_that_is_nan_is_not_hidden(h, dtype, p, tokens, dim):  # noqa: F811
    """NaN in a row of the vocabulary: every log probability is NaN, and so is every gradient that uses it."""
    whole, hidden, targets, a, b = inputs(p, tokens, dim, dtype)
    whole[LOW, 9] = float("nan")
    used, keep = targets >= 0, torch.arange(dim, device="cuda") != 9
    r = h.vocab_logprobs(hidden, pieces(whole, p), targets)
    assert bool(r.lse.isnan().all())
    for db in (None, b):
        dh, dw = h.vocab_logprobs_grad(hidden, pieces(whole, p), targets, r.lse, r.entropy, a, dentropy=db)
        assert bool(dh[used].isnan().all()) and bool((dh[~used][:, keep] == 0).all()) and bool(torch.cat(dw).isnan().all())
    # with the statistics of clean rows only the row itself is
    clean = h.vocab_logprobs(hidden, pieces(torch.cat([whole[:LOW], whole[LOW + 1:]]), p), targets)
    dw = torch.cat(h.vocab_logprobs_grad(hidden, pieces(whole, p), targets, clean.lse, clean.entropy, a, dentropy=b)[1])
    assert bool(dw[LOW].isnan().all()) and bool(dw[:LOW].isfinite().all()) and bool(dw[LOW + 1:].isfinite().all())

"""The cross entropy's forms for a dim above 1024 (sums of 1024 each) and for
a vocabulary in several windows, and the lookup of many single elements,
against plain forms in 64 bits.  The bounds are those of test_model_ops."""
import pytest
import torch

from tests.test_model_ops import (DTYPES, F, HALF, TINY, U, check_xent, gen, h, normal, pieces, within,  # noqa: F401
                                  xent_inputs, xent_reference)

pytestmark = pytest.mark.gpu


def check_gradients(h, tokens, dim, vocab, p, dtype):  # noqa: F811
    g = gen(tokens + dim)
    whole, hidden, targets = xent_inputs(g, tokens, dim, vocab, dtype)
    tw = torch.rand(tokens, generator=g, device="cuda") / tokens
    r = h.vocab_xent(hidden, pieces(whole, p), targets, token_weight=tw, grad=True)
    check_xent(r, xent_reference(hidden, pieces(whole, p), targets, tw), True)
    alone = h.vocab_xent(hidden, pieces(whole, p), targets)
    assert torch.equal(alone.loss, r.loss) and torch.equal(alone.lse, r.lse)
    again = h.vocab_xent(hidden, pieces(whole, p), targets, token_weight=tw, grad=True)
    assert torch.equal(again.dhidden, r.dhidden) and all(torch.equal(x, y) for x, y in zip(again.dweights, r.dweights))
    h.check()


@pytest.mark.parametrize("dtype", HALF)
@pytest.mark.parametrize("p,tokens,dim,vocab", [
    (3, 333, 1032, 5003),   # one sum and a step of 8
    (1, 16, 2048, 4099),    # two whole sums, few tokens
    (8, 515, 2048, 10007),
    (5, 257, 2056, 1999),   # two and a step of 8
    (2, 1, 4104, 301),
    (2, 700, 1088, 40001),  # one sum and a whole step; tiles for more than a wave
])
def test_sums_of_1024(h, dtype, p, tokens, dim, vocab):  # noqa: F811
    check_gradients(h, tokens, dim, vocab, p, dtype)


def positive_inputs(dim, dtype, tokens=40, vocab=300):
    """(hidden, whole, targets, logits in 64 bits, bound of a logit by sums of 1024):
    products that are all positive, so that every cut goes the same way.  An instruction
    adds 16 products: they are aligned to the largest term and the accumulator is cut
    to its 24 bits, two errors of up to 2^-23 of the accumulator, which here is a
    prefix of the sum."""
    g = gen(dim)
    hidden = (0.5 + 0.5 * torch.rand(tokens, dim, generator=g, device="cuda")).to(dtype)
    whole = (0.5 + 0.5 * torch.rand(vocab, dim, generator=g, device="cuda")).to(dtype)
    targets = torch.randint(0, vocab, (tokens,), generator=g, device="cuda")
    steps = torch.nn.functional.pad(hidden.double()[:, None, :] * whole.double()[None], (0, -dim % 1024)).view(tokens, vocab, -1, 64, 16).sum(-1)
    z, sums = steps.sum((2, 3)), steps.shape[2]
    return hidden, whole, targets, z, (2 * 2.0 ** -23 * steps.cumsum(3).sum((2, 3)) + sums * F * z).amax(1)


@pytest.mark.parametrize("dtype", HALF)
@pytest.mark.parametrize("dim", [1000, 8192, 16384])
def test_gradients_are_those_of_sums_of_1024(h, dtype, dim):  # noqa: F811
    """G = softmax - onehot takes an error of the logits as its own relative
    error: the pass that makes it needs the logits as well as the one that makes lse."""
    hidden, whole, targets, z, dz = positive_inputs(dim, dtype)
    tokens, vocab = z.shape
    r = h.vocab_xent(hidden, pieces(whole, 2), targets, grad=True)
    lse = torch.logsumexp(z, 1)
    dlse = dz + 2.0 ** -18 + 4 * F * lse
    prob = torch.exp(z - lse[:, None])
    gmat = prob.scatter_add(1, targets[:, None], -torch.ones_like(lse)[:, None])
    u = U[dtype]
    dg = torch.expm1(dz + dlse + 2.0 ** -18 + 8 * F * lse)[:, None] * prob + (u + 4 * F) * gmat.abs() + 2.0 ** -37
    hid, w = hidden.double(), whole.double()
    for got, ref, mag, err, n in ((r.dhidden, gmat @ w, gmat.abs() @ w, dg @ w, vocab),
                                  (torch.cat(r.dweights), gmat.T @ hid, gmat.abs().T @ hid, dg.T @ hid, tokens)):
        err = err + 2 * (n + 8) * F * mag
        within(got, ref, err + u * (ref.abs() + err) + TINY[dtype], "gradient")


@pytest.mark.parametrize("dtype", HALF)
@pytest.mark.parametrize("dim", [1032, 16384])
def test_lse_is_that_of_sums_of_1024(h, dtype, dim):  # noqa: F811
    """With an accumulator a 1024 of dim a logit's error is a sum over at most 64
    prefixes; one accumulator for all of dim 16384 would lose some sixteen times that."""
    hidden, whole, targets, z, dz = positive_inputs(dim, dtype)
    r = h.vocab_xent(hidden, pieces(whole, 2), targets)
    lse = torch.logsumexp(z, 1)
    # exponentials, their sum, and the rounding of lse itself
    dlse = dz + 2.0 ** -18 + 4 * F * lse
    within(r.lse, lse, dlse, "lse")
    zt = z.gather(1, targets[:, None])[:, 0]
    within(r.loss, lse - zt, dlse + dz + 4 * F * lse, "loss")


@pytest.mark.parametrize("dtype", HALF)
@pytest.mark.parametrize("p,tokens,dim,vocab", [
    (1, 4096, 256, 33000),   # windows of 128 blocks and 1; dhidden's sum in 9 parts, then in 1
    (3, 8192, 1288, 16700),  # windows of 64 blocks and 2; dhidden written by the last one
    (2, 2050, 64, 131073),   # windows of 255 blocks, 255 and 3, the second begins inside a piece
])
def test_windows_of_the_vocabulary(h, dtype, p, tokens, dim, vocab):  # noqa: F811
    check_gradients(h, tokens, dim, vocab, p, dtype)


@pytest.mark.parametrize("dtype", DTYPES)
def test_lookup_of_many_single_elements(h, dtype):  # noqa: F811
    g = gen(8)
    tokens, dim, vocab = 701, 1001, 5003
    whole = normal(g, vocab, dim, dtype=dtype)
    tok = torch.randint(-1, vocab + 1, (tokens,), generator=g, device="cuda")
    counts = (tok >= 0) & (tok < vocab)
    y = h.embedding(pieces(whole, 3), tok, scale=0.3)
    # the product in 32 bits, rounded once
    ref = torch.where(counts[:, None], whole[tok.clamp(0, vocab - 1)].float() * torch.tensor(0.3, device="cuda"), torch.zeros((), device="cuda"))
    assert torch.equal(y, ref.to(dtype))

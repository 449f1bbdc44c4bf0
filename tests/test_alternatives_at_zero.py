"""Alternatives whose logits are 0, where the pairs of CTAs tell each other how far their lists have come (more
blocks of the vocabulary than pairs on a row of tiles): the values on both sides of 0 are the only neighbours whose bits
are far apart.

Values are whole numbers and sixteenths, so that sums of their products are exact; tokens are compared as they are, never
used as indices.
"""
import math

import pytest
import torch

from tests.test_model_ops import F, HALF, gen, h, normal, pieces  # noqa: F401

pytestmark = pytest.mark.gpu

SHARED = [(4, 600, 24, 70000), (3, 1300, 16, 8191), (2, 256, 64, 32768), (8, 2048, 16, 50021), (1, 150, 1032, 33000)]


def in_order(z, top):
    return torch.sort(z + 0.0, dim=1, descending=True, stable=True).indices[:, :top]  # (no -0)


@pytest.mark.parametrize("dtype", HALF)
@pytest.mark.parametrize("p,tokens,dim,vocab", SHARED)
def test_hidden_states_of_zeros(h, dtype, p, tokens, dim, vocab):  # noqa: F811
    g = gen(vocab)
    hidden = torch.randint(-4, 5, (tokens, dim), generator=g, device="cuda").to(dtype)
    hidden[::3] = 0.0
    hidden[1::9] = -0.0
    whole = (torch.randint(-4, 5, (vocab, dim), generator=g, device="cuda") / 16).to(dtype)
    none = torch.full((tokens,), -1, device="cuda")
    zero = (hidden == 0).all(1)
    order = in_order(hidden.float() @ whole.float().T, 32)
    for top in (1, 8, 32):
        r = h.vocab_logprobs(hidden, pieces(whole, p), none, top=top)
        assert torch.equal(r.top_token, order[:, :top])
        # S is the vocabulary's size, as a sum of ones in 32 bits
        assert bool(((r.top_logprob[zero].double() + math.log(vocab)).abs() <= 2.0 ** -17).all())
    h.check()


@pytest.mark.parametrize("dtype", HALF)
@pytest.mark.parametrize("zeros", [5, 40, 4000])
@pytest.mark.parametrize("p,tokens,dim,vocab", SHARED)
def test_the_last_alternative_is_zero(h, dtype, zeros, p, tokens, dim, vocab):  # noqa: F811
    """Three logits above 0, some of 0, on both sides of the blocks' borders too, and all others below."""
    g = gen(zeros)
    whole = torch.zeros(vocab, dim, dtype=dtype, device="cuda")
    whole[:, 0] = -1.0 - torch.arange(vocab, device="cuda") % 7 / 16
    places = torch.randint(0, vocab, (zeros,), generator=g, device="cuda")
    places[::2] = places[::2] // 256 * 256 + 255 * torch.randint(0, 2, places[::2].shape, generator=g, device="cuda")
    whole[places.clamp(max=vocab - 1)] = 0.0
    whole[torch.randint(0, vocab, (3,), generator=g, device="cuda"), 0] = 1.0
    hidden = torch.zeros(tokens, dim, dtype=dtype, device="cuda")
    hidden[:, 0] = 2.0 ** -(torch.arange(tokens, device="cuda") % 5).float()
    hidden[:, 1] = torch.randint(-4, 5, (tokens,), generator=g, device="cuda").to(dtype)  # (against columns of zeros)
    order = in_order(hidden.float() @ whole.float().T, 32)
    none = torch.full((tokens,), -1, device="cuda")
    for top in (4, 8, 20, 32):
        assert torch.equal(h.vocab_logprobs(hidden, pieces(whole, p), none, top=top).top_token, order[:, :top])
    h.check()


@pytest.mark.parametrize("dtype", HALF)
def test_padded_places_of_a_prompt(h, dtype):  # noqa: F811
    """Tokens that are left out: zeros from the table, through the norm, to the alternatives."""
    g = gen(12)
    p, tokens, dim, vocab = 4, 400, 64, 33000
    table = pieces(normal(g, vocab, dim, dtype=dtype, std=0.1), p)
    prompt = torch.randint(0, vocab, (tokens,), generator=g, device="cuda")
    padded = torch.arange(tokens, device="cuda") % 100 >= 70
    prompt[padded] = -1
    n = h.add_rmsnorm([h.embedding(table, prompt)])
    assert bool((n.out[padded] == 0).all())
    r = h.vocab_logprobs(n.out, table, prompt, top=8)
    want = torch.arange(8, device="cuda").expand(int(padded.sum()), 8)
    assert torch.equal(r.top_token[padded], want)
    assert bool(((r.top_logprob[padded].double() + math.log(vocab)).abs() <= 2.0 ** -17).all())
    assert bool((r.logprob[padded] == 0).all())
    # (two roundings of a logit's place between the list and the sums)
    assert bool((r.top_logprob[~padded, 0] <= 8 * F * r.lse[~padded].abs()).all())

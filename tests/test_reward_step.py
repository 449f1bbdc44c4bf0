"""The operators of a step on rewards, run together as the example runs them: embedding, norms, log
probabilities, their gradients, the table's gradient, and clipping."""
import pytest
import torch

import ring_all_reduce_rar_gb300 as rar
from tests.test_example_model_step import _example, _norm
from tests.test_model_ops import gen, h, normal, pieces  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("ranks", [1, 4])
@pytest.mark.parametrize("max_norm", [1e-3, 1e9])
def test_gradients_against_autograd(ranks, max_norm):
    """The chain from the loss back to the table rounds fewer than 16 tensors to 8 bits, as in the
    cross entropy's test; clipping rounds once more and scales all alike."""
    ex = _example()
    model = ex.Model(ranks, vocab=503, dim=128, inner=256)
    g = torch.Generator().manual_seed(5)
    tokens, actions = (torch.randint(0, 503, (77,), generator=g).cuda() for _ in range(2))
    advantage = torch.randn(77, generator=g).cuda()
    actions[::9] = -1  # places that have no action
    logprob, norm, grads = model.reward_gradients(tokens, actions, advantage, bonus=0.1, max_norm=max_norm)
    wide = [p.double().requires_grad_() for p in model.params]
    table = torch.cat(wide[:ranks])
    x0 = table[tokens] * model.table_scale
    n0 = _norm(x0, wide[-2])
    x1 = x0 + sum(model.rank_part(n0, wide[ranks + 2 * r], wide[ranks + 2 * r + 1]) for r in range(ranks))
    logp = torch.log_softmax(_norm(x1, wide[-1]) @ table.t(), 1)
    has = (actions >= 0).double()
    own = logp.gather(1, actions.clamp(min=0)[:, None])[:, 0]
    (-(has * (advantage.double() * own - 0.1 * (logp.exp() * logp).sum(1))).mean()).backward()
    # hidden states with an error of a few 2^-8 move a logit of size ~1 by as much
    assert float((logprob.double() - has * own.detach()).abs().max()) <= 16 * 2 ** -8 * float(own.detach().abs().max())
    total = torch.linalg.vector_norm(torch.stack([p.grad.norm() for p in wide]))
    assert abs(float(norm.double() - total)) <= 16 * 2 ** -8 * float(total)
    scale = min(1.0, max_norm / float(norm))
    for got, p in zip(grads, wide):
        assert (got.double() - scale * p.grad).norm() <= scale * 17 * 2 ** -8 * p.grad.norm()
    model.handle.check()


def test_the_example_runs():
    before, after, norms = _example().run_rewards(ranks=3, steps=2)
    assert before.shape == after.shape == (333,) and bool(before.isfinite().all()) and bool(after.isfinite().all())
    assert norms.shape == (2,) and bool((norms > 0).all())


def test_a_step_in_a_graph(h):  # noqa: F811
    """All of a step's calls in one captured graph, replayed with new inputs in the same places."""
    g = gen(7)
    dim, vocab, tokens, p = 128, 777, 200, 3
    whole = normal(g, vocab, dim, dtype=torch.bfloat16, std=0.1)
    weights, part = pieces(whole, p), normal(g, tokens, dim, dtype=torch.bfloat16)
    tok, act = (torch.randint(0, vocab, (tokens,), generator=g, device="cuda") for _ in range(2))
    adv, bonus = normal(g, tokens), torch.full((tokens,), 0.01, device="cuda")

    def step():
        n = h.add_rmsnorm([part], residual=h.embedding(weights, tok, scale=3.0))
        r = h.vocab_logprobs(n.out, weights, act, top=4)
        dh, dw = h.vocab_logprobs_grad(n.out, weights, act, r.lse, r.entropy, adv, dentropy=bonus)
        dx, dnorm = h.add_rmsnorm_grad(dh, n.sum, n.rstd)
        h.embedding_grad(dx, tok, dw, scale=3.0, accumulate=True)
        total = h.grad_clip([*dw, dnorm], 0.01)
        return [*r, total, dnorm, *dw]

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = step()
    for _ in range(3):
        tok.copy_(torch.randint(0, vocab, (tokens,), generator=g, device="cuda"))
        act.copy_(torch.randint(-1, vocab, (tokens,), generator=g, device="cuda"))
        part.normal_(generator=g)
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in held]
        assert all(torch.equal(x, y) for x, y in zip(step(), got))
    h.check()


def test_two_handles_at_once(h):  # noqa: F811
    """Two threads, a handle and a stream each, whose calls differ in size."""
    import threading
    g = gen(8)
    whole, hidden = normal(g, 9000, 256, dtype=torch.bfloat16, std=0.1), normal(g, 700, 256, dtype=torch.bfloat16)
    tok = torch.randint(0, 9000, (700,), generator=g, device="cuda")
    sizes, wrong = [(5, 3), (700, 20)], []
    ref = {n: h.vocab_logprobs(hidden[:n], pieces(whole, 3), tok[:n], top=k) for n, k in sizes}
    norm = h.grad_norm([whole, hidden])
    torch.cuda.synchronize()

    def work(n, k):
        stream = torch.cuda.Stream()
        with torch.cuda.stream(stream), rar.Handle(0) as mine:
            for _ in range(200):
                r = mine.vocab_logprobs(hidden[:n], pieces(whole, 3), tok[:n], top=k)
                s = mine.grad_norm([whole, hidden])
            stream.synchronize()
            if not (all(torch.equal(x, y) for x, y in zip(r, ref[n])) and torch.equal(s.norm, norm.norm)):
                wrong.append(n)
            mine.check()

    threads = [threading.Thread(target=work, args=s) for s in sizes]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong

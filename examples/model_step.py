"""Training steps and a scoring step of a small tensor-parallel language model
whose p ranks live on one GPU: embedding, a gated block whose ranks' partial
outputs are summed, residual joins with RMS norms, and the cross entropy over
the (tied) vocabulary, forward and backward.

    python examples/model_step.py [--ranks 4] [--steps 30]

What the library does in a step, in order: embedding, add_rmsnorm (one part),
add_rmsnorm (p parts), vocab_xent with gradients, add_rmsnorm_grad, allreduce
of the ranks' gradients for the block's input, add_rmsnorm_grad, and
embedding_grad added into vocab_xent's gradient of the tied table.  The ranks'
own matrix products are torch's.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import ring_all_reduce_rar_gb300 as rar  # noqa: E402


class Model:
    """Parameters in bfloat16 with float32 copies that the steps are made on."""

    def __init__(self, ranks=4, vocab=1003, dim=256, inner=512, dtype=torch.bfloat16, seed=0, device="cuda"):
        g = torch.Generator().manual_seed(seed)

        def normal(rows, cols, std):
            return torch.randn(rows, cols, generator=g) * std

        share = [vocab // ranks + (r < vocab % ranks) for r in range(ranks)]  # rank r's rows of the vocabulary
        self.table_scale = dim ** 0.5
        masters = [normal(n, dim, dim ** -0.5) for n in share]
        for _ in range(ranks):
            masters += [normal(dim, 2 * (inner // ranks), dim ** -0.5), normal(inner // ranks, dim, inner ** -0.5)]
        masters += [torch.ones(dim), torch.ones(dim)]
        self.masters = [m.to(device) for m in masters]
        self.params = [m.to(dtype) for m in self.masters]
        self.ranks = ranks
        self.handle = rar.Handle(0)

    @property
    def table(self):
        return self.params[:self.ranks]

    def block(self, r):
        """Rank r's two matrices."""
        at = self.ranks + 2 * r
        return self.params[at], self.params[at + 1]

    @staticmethod
    def rank_part(x, up, down):
        gate, value = (x @ up).chunk(2, dim=1)
        return (torch.nn.functional.silu(gate) * value) @ down

    def hidden(self, tokens, quant_group=None):
        """(first norm, ranks' graphs, last norm) for the tokens."""
        h, (w0, w1) = self.handle, self.params[-2:]
        n0 = h.add_rmsnorm([h.embedding(self.table, tokens, scale=self.table_scale)], w0)
        graphs = []
        for r in range(self.ranks):
            inputs = [t.detach().requires_grad_() for t in (n0.out, *self.block(r))]
            with torch.enable_grad():
                graphs.append((self.rank_part(*inputs), inputs))
        n1 = h.add_rmsnorm([part.detach() for part, _ in graphs], w1, residual=n0.sum, quant_group=quant_group,
                           keep_out=True)
        return n0, graphs, n1

    def gradients(self, tokens, targets):
        """(mean loss, a gradient per parameter)."""
        h, (w0, w1) = self.handle, self.params[-2:]
        n0, graphs, n1 = self.hidden(tokens)
        weight = torch.full((tokens.numel(),), 1.0 / tokens.numel(), device=tokens.device)
        x = h.vocab_xent(n1.out, self.table, targets, token_weight=weight, grad=True)
        dx1, dw1 = h.add_rmsnorm_grad(x.dhidden, n1.sum, n1.rstd, w1)
        per_rank = [torch.autograd.grad(part, inputs, dx1) for part, inputs in graphs]
        partial = [d[0].contiguous() for d in per_rank]
        if self.ranks > 1:
            h.allreduce(partial, op="sum")
        dx0, dw0 = h.add_rmsnorm_grad(partial[0], n0.sum, n0.rstd, w0, dsum=dx1)
        dtable = h.embedding_grad(dx0, tokens, x.dweights, scale=self.table_scale, accumulate=True)
        return x.loss.mean(), [*dtable, *(d for one in per_rank for d in one[1:]), dw0, dw1]

    def step(self, tokens, targets, rate=0.05):
        loss, grads = self.gradients(tokens, targets)
        for master, param, grad in zip(self.masters, self.params, grads):
            master.sub_(grad.float(), alpha=rate)
            param.copy_(master)
        return loss

    def score(self, tokens, targets):
        """Loss of each token with the last hidden states in 8 bits (a scale per 128 columns)."""
        n1 = self.hidden(tokens, quant_group=128)[2]
        codes, scales = n1.out8.float(), n1.scales.repeat_interleave(128, dim=1)
        return self.handle.vocab_xent((codes * scales[:, :codes.shape[1]]).to(n1.out.dtype), self.table, targets).loss


def run(ranks=4, steps=30, tokens=333, vocab=1003, seed=0):
    """Trains on one batch; (losses, loss of each token afterwards)."""
    model = Model(ranks, vocab, seed=seed)
    g = torch.Generator().manual_seed(seed + 1)
    text = torch.randint(0, vocab, (tokens + 1,), generator=g).cuda()
    losses = torch.stack([model.step(text[:-1], text[1:]) for _ in range(steps)])
    scores = model.score(text[:-1], text[1:])
    model.handle.check()
    return losses.tolist(), scores


if __name__ == "__main__":
    ap = argparse.ArgumentParser()
    ap.add_argument("--ranks", type=int, default=4)
    ap.add_argument("--steps", type=int, default=30)
    a = ap.parse_args()
    losses, scores = run(a.ranks, a.steps)
    print("losses:", " ".join(f"{v:.3f}" for v in losses))
    print(f"after the steps, from 8-bit hidden states: {scores.mean().item():.3f}")

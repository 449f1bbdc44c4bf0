"""The operators at which a tensor-parallel language model reduces over its ranks, as cases to measure.

    norm         s = residual + the sum of the p ranks' partial rows; y = s / rms(s) * w, in 16 or 32 bits, or in
                 8 bits (e4m3) with a scale for each group of columns
    norm_grad    its gradient for the residual stream (and every partial) and for w
    xent         softmax cross entropy from hidden states over a vocabulary held in p pieces, no logits kept
    xent_grad    the same with the gradients of hidden states and pieces
    embed        scaled lookup in a table held in the same p pieces
    embed_grad   its gradient by sorted tokens, written whole or added into what is there

Rank r's piece is rows [start_r, start_(r+1)) of the vocabulary, the first V mod p pieces one row longer.  A target or
token outside the vocabulary is left out: loss 0, no gradient, a row of zeros.
"""
import math

import torch

own = False

DTYPES = {"float32": torch.float32, "bfloat16": torch.bfloat16, "float16": torch.float16}
SIZE = {"float32": 4, "bfloat16": 2, "float16": 2}
EPS = 1e-6


def listed():
    return [
        # four sequences decode one token each: the join after a layer, 8-bit input for the next product
        {"name": "norm_decode", "op": "norm", "p": 8, "rows": 4, "dim": 2048, "dtype": "bfloat16", "group": 128},
        # a prompt of 4096 tokens through the same join
        {"name": "norm_prefill", "op": "norm", "p": 8, "rows": 4096, "dim": 4096, "dtype": "bfloat16", "group": 128},
        # training in 32 bits on a short batch, a width that no vector divides
        {"name": "norm_grad_odd", "op": "norm_grad", "rows": 1027, "dim": 1001, "dtype": "float32"},
        # a training step's micro-batch of 8192 tokens
        {"name": "norm_grad_train", "op": "norm_grad", "rows": 8192, "dim": 4096, "dtype": "bfloat16"},
        # scoring the next token of 16 sequences against the whole vocabulary
        {"name": "xent_score", "op": "xent", "p": 4, "tokens": 16, "dim": 2048, "vocab": 32768, "dtype": "bfloat16"},
        # held-out loss on 2048 tokens, a vocabulary that neither tiles nor ranks divide
        {"name": "xent_eval", "op": "xent", "p": 8, "tokens": 2048, "dim": 2048, "vocab": 50021, "dtype": "float16"},
        # fine-tuning on a ragged batch of a small model
        {"name": "xent_grad_odd", "op": "xent_grad", "p": 3, "tokens": 333, "dim": 520, "vocab": 10007, "dtype": "float16"},
        # a training step's micro-batch of 8192 tokens
        {"name": "xent_grad_train", "op": "xent_grad", "p": 8, "tokens": 8192, "dim": 4096, "vocab": 65536, "dtype": "bfloat16"},
        # four sequences' next tokens enter the model
        {"name": "embed_decode", "op": "embed", "p": 8, "tokens": 4, "dim": 2048, "vocab": 65536, "dtype": "bfloat16"},
        # a micro-batch of 8192 tokens enters the model
        {"name": "embed_train", "op": "embed", "p": 8, "tokens": 8192, "dim": 4096, "vocab": 65536, "dtype": "bfloat16"},
        # its gradient, written whole
        {"name": "embed_grad_train", "op": "embed_grad", "p": 8, "tokens": 8192, "dim": 4096, "vocab": 65536, "dtype": "bfloat16",
         "add": False},
        # tied weights in 32 bits: added into the output layer's gradient
        {"name": "embed_grad_tied", "op": "embed_grad", "p": 3, "tokens": 4095, "dim": 1001, "vocab": 10007, "dtype": "float32",
         "add": True},
    ]


def draw(rng):
    def size(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(("norm", "norm_grad", "xent", "xent_grad", "embed", "embed_grad"))
    p = rng.choice((1, 2, 3, 4, 8, 16))
    if op in ("norm", "norm_grad"):
        case = {"op": op, "rows": size(1, 8192), "dim": size(64, 8192), "dtype": rng.choice(("bfloat16", "float16", "float32"))}
        if op == "norm":
            # -1: no 8-bit output, 0: one scale a row
            case.update(p=p, group=rng.choice((-1, 0, 128)))
        return case
    case = {"op": op, "p": p, "tokens": size(1, 8192)}
    if op in ("xent", "xent_grad"):
        case.update(dim=8 * size(8, 512), vocab=size(256, 65536), dtype=rng.choice(("bfloat16", "float16")))
    else:
        case.update(dim=size(64, 4096), vocab=size(256, 65536), dtype=rng.choice(("bfloat16", "float16", "float32")))
        if op == "embed_grad":
            case["add"] = rng.random() < 0.5
    return case


def work(case):
    op, e = case["op"], SIZE[case["dtype"]]
    if op == "norm":
        t, d, g = case["rows"], case["dim"], case["group"]
        out = t * d * e if g < 0 else t * d + 4 * t * (-(-d // g) if g else 1)
        return {"bytes": (case["p"] + 2) * t * d * e + d * e + out + 4 * t, "flops": (case["p"] + 4) * t * d}
    if op == "norm_grad":
        t, d = case["rows"], case["dim"]
        return {"bytes": 4 * t * d * e + 2 * d * e + 4 * t, "flops": 9 * t * d}
    t, d, v = case["tokens"], case["dim"], case["vocab"]
    if op == "xent":
        return {"bytes": (t + v) * d * e + 16 * t, "flops": 2 * t * v * d}
    if op == "xent_grad":
        return {"bytes": 2 * (t + v) * d * e + 20 * t, "flops": 6 * t * v * d}
    if op == "embed":
        return {"bytes": 2 * t * d * e + 8 * t, "flops": t * d}
    used = min(t, v)
    return {"bytes": t * d * e + 8 * t + (2 * used * d * e if case["add"] else v * d * e), "flops": t * d}


def _pieces(whole, p):
    """Views of the ranks' rows: the first V mod p pieces are one row longer."""
    base, extra = divmod(whole.shape[0], p)
    return list(whole.split([base + 1] * extra + [base] * (p - extra)))


def _tokens(n, vocab, gen):
    """Token ids as text has them: few frequent, many rare; in no order of the ids; a few places are padding."""
    u = torch.rand(n, generator=gen, device="cuda", dtype=torch.float64)
    rank = torch.exp(u * math.log(vocab + 1.0)).long() - 1  # density ~ 1 / rank
    rank = rank.clamp_(0, vocab - 1)
    ids = torch.randperm(vocab, generator=gen, device="cuda")[rank]
    pad = torch.rand(n, generator=gen, device="cuda") < 0.02
    return torch.where(pad, torch.full_like(ids, -1), ids)


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    dt, op = DTYPES[case["dtype"]], case["op"]

    def normal(*shape, std=1.0):
        return (torch.randn(*shape, generator=gen, device="cuda", dtype=torch.float32) * std).to(dt)

    s = {"case": dict(case)}
    if op == "norm":
        t, d, p = case["rows"], case["dim"], case["p"]
        s["partials"] = normal(p, t, d, std=0.5 / math.sqrt(p))
        s["parts"] = list(s["partials"].unbind(0))
        s["residual"] = normal(t, d, std=2.0)
        s["weight"] = (1.0 + 0.1 * torch.randn(d, generator=gen, device="cuda")).to(dt)
    elif op == "norm_grad":
        t, d = case["rows"], case["dim"]
        s["sum"] = normal(t, d, std=2.0)
        s["weight"] = (1.0 + 0.1 * torch.randn(d, generator=gen, device="cuda")).to(dt)
        s["rstd"] = torch.rsqrt(s["sum"].double().square().mean(1) + EPS).float()
        s["dout"] = normal(t, d, std=1e-2)
        s["dsum"] = normal(t, d, std=1e-2)
    elif op in ("xent", "xent_grad"):
        t, d, v = case["tokens"], case["dim"], case["vocab"]
        s["whole"] = normal(v, d, std=2.0 / math.sqrt(d))
        s["pieces"] = _pieces(s["whole"], case["p"])
        s["targets"] = _tokens(t, v, gen)
        # half of the tokens are foreseen: their hidden state leans to the target's row (its logit rises by about 8)
        lean = 2.0 * (torch.rand(t, 1, generator=gen, device="cuda") < 0.5)
        s["hidden"] = (normal(t, d).float() + lean * s["whole"][s["targets"].clamp(min=0)].float()).to(dt)
        # the mean over the tokens that count
        s["token_weight"] = torch.full((t,), 1.0 / t, device="cuda")
    else:
        t, d, v = case["tokens"], case["dim"], case["vocab"]
        s["tokens"] = _tokens(t, v, gen)
        s["scale"] = math.sqrt(d)
        if op == "embed":
            s["whole"] = normal(v, d, std=0.02)
        else:
            s["dout"] = normal(t, d, std=1e-3)
            s["whole"] = normal(v, d, std=1e-2) if case["add"] else torch.empty(v, d, device="cuda", dtype=dt)
        s["pieces"] = _pieces(s["whole"], case["p"])
    return s


_kept = {}


def _handle():
    """The library handle that a program creates once."""
    if "handle" not in _kept:
        import ring_all_reduce_rar_gb300 as rar
        _kept["handle"] = rar.Handle(0, skip_pointer_check=True)
    return _kept["handle"]


def _run_own(s):
    h, case = _handle(), s["case"]
    op = case["op"]
    if op == "norm":
        g = case["group"]
        r = h.add_rmsnorm(s["parts"], s["weight"], residual=s["residual"], eps=EPS, quant_group=None if g < 0 else g)
        return [r.sum, r.rstd, r.out] if g < 0 else [r.sum, r.rstd, r.out8, r.scales]
    if op == "norm_grad":
        return list(h.add_rmsnorm_grad(s["dout"], s["sum"], s["rstd"], s["weight"], dsum=s["dsum"]))
    if op == "xent":
        r = h.vocab_xent(s["hidden"], s["pieces"], s["targets"])
        return [r.loss, r.lse]
    if op == "xent_grad":
        r = h.vocab_xent(s["hidden"], s["pieces"], s["targets"], token_weight=s["token_weight"], grad=True)
        return [r.loss, r.lse, r.dhidden, list(r.dweights)]
    if op == "embed":
        return h.embedding(s["pieces"], s["tokens"], scale=s["scale"])
    return list(h.embedding_grad(s["dout"], s["tokens"], s["pieces"], scale=s["scale"], accumulate=case["add"]))


def _plain_norm(s):
    case = s["case"]
    dt, g = DTYPES[case["dtype"]], case["group"]
    x = s["partials"].float().sum(0) + s["residual"].float()
    rstd = 1.0 / torch.sqrt((x * x).mean(1) + EPS)
    y = x * rstd[:, None] * s["weight"].float()
    if g < 0:
        return [x.to(dt), rstd, y.to(dt)]
    t, d = y.shape
    g = g or d
    groups = -(-d // g)
    padded = torch.zeros(t, groups * g, device=y.device)
    padded[:, :d] = y
    padded = padded.view(t, groups, g)
    tiny, huge = torch.finfo(torch.float32).tiny, torch.finfo(torch.float32).max
    scales = (padded.abs().amax(2).clamp(max=huge) / 448.0).clamp(min=tiny)
    q = (padded / scales[:, :, None]).reshape(t, groups * g)[:, :d]
    return [x.to(dt), rstd, q.to(torch.float8_e4m3fn), scales]


def _plain_norm_grad(s):
    dt = s["sum"].dtype
    x, dy, w, rstd = s["sum"].float(), s["dout"].float(), s["weight"].float(), s["rstd"][:, None]
    n = x * rstd
    wdy = w * dy
    dx = s["dsum"].float() + rstd * (wdy - n * (wdy * n).mean(1, keepdim=True))
    return [dx.to(dt), (dy * n).sum(0).to(dt)]


def _plain_xent(s):
    case = s["case"]
    dt, v = DTYPES[case["dtype"]], case["vocab"]
    h, w, target = s["hidden"].float(), s["whole"].float(), s["targets"]
    z = h @ w.t()
    m = z.amax(1)
    lse = m + torch.log(torch.exp(z - m[:, None]).sum(1))
    counts = (target >= 0) & (target < v)
    at = target.clamp(0, v - 1)[:, None]
    loss = torch.where(counts, lse - z.gather(1, at)[:, 0], torch.zeros_like(lse))
    if case["op"] == "xent":
        return [loss, lse]
    g = torch.exp(z - lse[:, None])
    g.scatter_add_(1, at, torch.full_like(lse, -1.0)[:, None])
    g *= torch.where(counts, s["token_weight"], torch.zeros_like(lse))[:, None]
    return [loss, lse, (g @ w).to(dt), _pieces((g.t() @ h).to(dt), case["p"])]


def _plain_embed(s):
    case = s["case"]
    dt, v, tok = DTYPES[case["dtype"]], case["vocab"], s["tokens"]
    counts = (tok >= 0) & (tok < v)
    if case["op"] == "embed":
        rows = s["whole"][tok.clamp(0, v - 1)].float() * s["scale"]
        return torch.where(counts[:, None], rows, torch.zeros_like(rows)).to(dt)
    rows = torch.where(counts[:, None], s["dout"].float(), torch.zeros((), device=tok.device))
    total = torch.zeros(v, case["dim"], device=tok.device)
    total.index_add_(0, tok.clamp(0, v - 1), rows)
    total *= s["scale"]
    if case["add"]:
        total += s["whole"].float()
    s["whole"].copy_(total)
    return list(s["pieces"])


PLAIN = {"norm": _plain_norm, "norm_grad": _plain_norm_grad, "xent": _plain_xent, "xent_grad": _plain_xent,
         "embed": _plain_embed, "embed_grad": _plain_embed}


def run(state):
    return _run_own(state) if own else PLAIN[state["case"]["op"]](state)


def exact(case, seed):
    """The definitions in 64 bits.  8-bit codes are given as the quotients that they round."""
    s, op = prepare(case, seed), case["op"]
    if op == "norm":
        x = s["residual"].double()
        for part in s["parts"]:
            x = x + part.double()
        ms = (x ** 2).sum(1) / case["dim"] + EPS
        y = x / ms.sqrt()[:, None] * s["weight"].double()
        if case["group"] < 0:
            return [x, ms.rsqrt(), y]
        g = case["group"] or case["dim"]
        codes, scales = [], []
        for lo in range(0, case["dim"], g):
            block = y[:, lo:lo + g]
            scale = (block.abs().max(1).values / 448).clamp(min=2.0 ** -126)
            scales.append(scale)
            codes.append(block / scale[:, None])
        return [x, ms.rsqrt(), torch.cat(codes, 1), torch.stack(scales, 1)]
    if op == "norm_grad":
        # d/dx of sum(dy w x r(x)) + sum(dsum x), r as it was kept
        x, dy, r = s["sum"].double(), s["dout"].double(), s["rstd"].double()
        a = dy * s["weight"].double()
        inner = torch.einsum("td,td->t", a, x)
        dx = s["dsum"].double() + a * r[:, None] - x * (r ** 3 * inner / case["dim"])[:, None]
        return [dx, torch.einsum("td,td,t->d", dy, x, r)]
    if op in ("xent", "xent_grad"):
        t, v, grad = case["tokens"], case["vocab"], op == "xent_grad"
        w = s["whole"].double()
        loss = torch.zeros(t, dtype=torch.float64, device="cuda")
        lse = torch.zeros_like(loss)
        dh = torch.zeros(t, case["dim"], dtype=torch.float64, device="cuda") if grad else None
        dw = torch.zeros_like(w) if grad else None
        step = max(1, (1 << 27) // v)
        for lo in range(0, t, step):
            h = s["hidden"][lo:lo + step].double()
            target = s["targets"][lo:lo + step]
            z = torch.matmul(h, w.T)
            lse[lo:lo + step] = torch.logsumexp(z, 1)
            row = torch.nonzero((target >= 0) & (target < v))[:, 0]
            loss[lo + row] = lse[lo + row] - z[row, target[row]]
            if grad:
                prob = torch.softmax(z, 1)
                prob[row, target[row]] -= 1
                weight = torch.zeros(len(h), dtype=torch.float64, device="cuda")
                weight[row] = s["token_weight"][lo + row].double()
                prob *= weight[:, None]
                dh[lo:lo + step] = torch.matmul(prob, w)
                dw += torch.matmul(prob.T, h)
        return [loss, lse, dh, _pieces(dw, case["p"])] if grad else [loss, lse]
    tok = s["tokens"]
    row = torch.nonzero((tok >= 0) & (tok < case["vocab"]))[:, 0]
    if op == "embed":
        y = torch.zeros(len(tok), case["dim"], dtype=torch.float64, device="cuda")
        y[row] = s["whole"][tok[row]].double() * s["scale"]
        return y
    total = s["whole"].double() if case["add"] else torch.zeros(case["vocab"], case["dim"], dtype=torch.float64, device="cuda")
    total.index_put_((tok[row],), s["dout"][row].double() * s["scale"], accumulate=True)
    return _pieces(total, case["p"])

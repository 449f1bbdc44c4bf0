"""What a tensor-parallel language model answers with, and the end of its training step, as cases to measure.

    logprobs       log probabilities of given tokens, entropy and the most likely alternatives, from hidden states over a
                   vocabulary held in p pieces, no logits kept
    logprobs_grad  gradients of hidden states and pieces from those of the log probabilities and of the entropy
    grad_norm      the norm of all gradients together, and of each
    grad_clip      that norm, and the gradients scaled down to a largest norm, into tensors of the optimizer's

Rank r's piece is rows [start_r, start_(r+1)) of the vocabulary, the first V mod p pieces one row longer.  A target
outside the vocabulary is left out: log probability 0, no gradient; entropy and alternatives are still those of its place.

Hidden states and pieces are normal values on a grid of a few bits less than their type has, so that every sum of their
products is exact in 32 bits: which alternative comes first then does not hang on the order of a summation, and equal
logits are equal on every side (they do occur, and go to the lowest token).
"""
import math

import torch

own = False

DTYPES = {"float32": torch.float32, "bfloat16": torch.bfloat16, "float16": torch.float16}
SIZE = {"float32": 4, "bfloat16": 2, "float16": 2}
CLIP_EPS = 1e-6


def listed():
    return [
        # the next token of one sequence, with its 20 alternatives
        {"name": "logprobs_token", "op": "logprobs", "p": 4, "tokens": 1, "dim": 2048, "vocab": 32768, "dtype": "bfloat16", "top": 20,
         "scale": 1.0},
        # 16 sequences decode one token each
        {"name": "logprobs_decode", "op": "logprobs", "p": 8, "tokens": 16, "dim": 4096, "vocab": 65536, "dtype": "bfloat16", "top": 5,
         "scale": 1.25},
        # a ragged batch of drafted tokens, checked against the whole vocabulary of a small model
        {"name": "logprobs_odd", "op": "logprobs", "p": 3, "tokens": 333, "dim": 520, "vocab": 10007, "dtype": "float16", "top": 1,
         "scale": 1.0},
        # a prompt of 2048 tokens with 8 alternatives each, a vocabulary that neither tiles nor ranks divide
        {"name": "logprobs_prompt", "op": "logprobs", "p": 8, "tokens": 2048, "dim": 2048, "vocab": 50021, "dtype": "float16", "top": 8,
         "scale": 1.0},
        # sampled sequences of 8192 tokens scored again before a training step
        {"name": "logprobs_rollout", "op": "logprobs", "p": 8, "tokens": 8192, "dim": 4096, "vocab": 65536, "dtype": "bfloat16", "top": 0,
         "scale": 1.0},
        # fine-tuning on rewards, a ragged batch of a small model
        {"name": "logprobs_grad_odd", "op": "logprobs_grad", "p": 3, "tokens": 333, "dim": 520, "vocab": 10007, "dtype": "float16",
         "entropy": False, "scale": 1.0},
        # the same with an entropy bonus on a micro-batch of 8192 tokens
        {"name": "logprobs_grad_train", "op": "logprobs_grad", "p": 8, "tokens": 8192, "dim": 4096, "vocab": 65536, "dtype": "bfloat16",
         "entropy": True, "scale": 1.0},
        # a model of one block: 14 tensors, 1.3 MB
        {"name": "grad_norm_small", "op": "grad_norm", "p": 4, "vocab": 1003, "dim": 256, "inner": 512, "layers": 1, "dtype": "bfloat16",
         "mixed": False},
        # a model of four wide blocks: 80 tensors, 2.1 GB, norm weights in 32 bits
        {"name": "grad_norm_train", "op": "grad_norm", "p": 8, "vocab": 65536, "dim": 4096, "inner": 16384, "layers": 4, "dtype": "bfloat16",
         "mixed": True},
        # many tensors whose rows no vector divides, in 32 bits: 440 tensors, 0.6 GB
        {"name": "grad_norm_many", "op": "grad_norm", "p": 8, "vocab": 10007, "dim": 1001, "inner": 2048, "layers": 24, "dtype": "float32",
         "mixed": False},
        # two blocks of a small model, fp16
        {"name": "grad_clip_odd", "op": "grad_clip", "p": 3, "vocab": 10007, "dim": 520, "inner": 1536, "layers": 2, "dtype": "float16",
         "mixed": True, "wide": False},
        # the four wide blocks, clipped gradients in 32 bits for the optimizer
        {"name": "grad_clip_train", "op": "grad_clip", "p": 8, "vocab": 65536, "dim": 4096, "inner": 16384, "layers": 4, "dtype": "bfloat16",
         "mixed": True, "wide": True},
    ]


def draw(rng):
    def size(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(("logprobs", "logprobs", "logprobs_grad", "grad_norm", "grad_clip"))
    case = {"op": op, "p": rng.choice((1, 2, 3, 4, 8, 16))}
    if op in ("logprobs", "logprobs_grad"):
        case.update(tokens=size(1, 8192), dim=8 * size(8, 512), vocab=size(256, 65536), dtype=rng.choice(("bfloat16", "float16")),
                    scale=rng.choice((1.0, 1.0, 0.5, 1.25)))
        if op == "logprobs":
            case["top"] = rng.choice((0, 1, 2, 5, 8, 20, 32))
        else:
            case["entropy"] = rng.random() < 0.5
    else:
        case.update(vocab=size(256, 65536), dim=size(64, 4096), inner=size(64, 8192), layers=size(1, 24),
                    dtype=rng.choice(("bfloat16", "float16", "float32")), mixed=rng.random() < 0.5)
        if op == "grad_clip":
            case["wide"] = rng.random() < 0.5
    return case


def _shapes(case):
    """(shape, dtype) of the gradients: every rank's piece of the table, its two matrices of every block, and the blocks'
    two norm weights, which the ranks share and which count once."""
    p, d, kind = case["p"], case["dim"], case["dtype"]
    shapes = [((case["vocab"] // p + (r < case["vocab"] % p), d), kind) for r in range(p)]
    for _ in range(case["layers"]):
        for r in range(p):
            n = case["inner"] // p + (r < case["inner"] % p)
            shapes += [((d, 2 * n), kind), ((n, d), kind)]
        shapes += [((d,), "float32" if case["mixed"] else kind)] * 2
    return shapes


def work(case):
    if case["op"] in ("logprobs", "logprobs_grad"):
        t, d, v, e = case["tokens"], case["dim"], case["vocab"], SIZE[case["dtype"]]
        if case["op"] == "logprobs":
            return {"bytes": (t + v) * d * e + 20 * t + 12 * t * case["top"], "flops": 2 * t * v * d}
        return {"bytes": 2 * (t + v) * d * e + (24 if case["entropy"] else 16) * t, "flops": 6 * t * v * d}
    shapes = _shapes(case)
    n = sum(math.prod(shape) for shape, _ in shapes)
    read = sum(math.prod(shape) * SIZE[kind] for shape, kind in shapes)
    if case["op"] == "grad_norm":
        return {"bytes": read + 4 * len(shapes) + 4, "flops": 2 * n}
    return {"bytes": read + (4 * n if case["wide"] else read) + 4, "flops": 3 * n}


def _pieces(whole, p):
    """Views of the ranks' rows: the first V mod p pieces are one row longer."""
    base, extra = divmod(whole.shape[0], p)
    return list(whole.split([base + 1] * extra + [base] * (p - extra)))


def _flat(shapes, kinds, dtypes):
    """A zeroed buffer for each kind, and a view of its own in them for every shape, each beginning at a multiple of 64
    elements."""
    ends, places = {}, []
    for shape, kind in zip(shapes, kinds):
        places.append(ends.get(kind, 0))
        ends[kind] = places[-1] + (math.prod(shape) + 63) // 64 * 64
    flat = {kind: torch.zeros(n, dtype=dtypes[kind], device="cuda") for kind, n in sorted(ends.items())}
    views = [flat[kind][at:at + math.prod(shape)].view(shape) for shape, kind, at in zip(shapes, kinds, places)]
    return list(flat.values()), views


def _grid(x, step, most):
    """x on the multiples of step up to most of them."""
    return (x / step).round_().clamp_(-most, most).mul_(step)


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    dt = DTYPES[case["dtype"]]

    def normal(*shape, std=1.0):
        return torch.randn(*shape, generator=gen, device="cuda", dtype=torch.float32) * std

    s = {"case": dict(case)}
    if case["op"] in ("grad_norm", "grad_clip"):
        # tensors of a model learn at different rates: each has its own size of gradients
        sizes = torch.randn(len(_shapes(case)), generator=gen, device="cuda").mul_(1.5).sub_(8.0).exp2_().tolist()
        s["grads"] = [normal(*shape, std=size).to(DTYPES[kind]) for (shape, kind), size in zip(_shapes(case), sizes)]
        if case["op"] == "grad_clip":
            n = sum(g.numel() for g in s["grads"])
            s["max_norm"] = 2.0 ** -10 * math.sqrt(n)  # about a fifth of their norm
            # the optimizer's gradients lie one after the other in a buffer for each type
            kinds = ["float32" if case["wide"] else kind for _, kind in _shapes(case)]
            s["flat"], s["out"] = _flat([g.shape for g in s["grads"]], kinds, {k: DTYPES[k] for k in set(kinds)})
        return s

    t, d, v = case["tokens"], case["dim"], case["vocab"]
    std = 2.0 / math.sqrt(d)
    step = 2.0 ** math.floor(math.log2(std / 12))
    whole = _grid(normal(v, d, std=std), step, 127)
    # token ids as text has them: few frequent, many rare, in no order of the ids; a few places are padding
    u = torch.rand(t, generator=gen, device="cuda", dtype=torch.float64)
    rank = (torch.exp(u * math.log(v + 1.0)).long() - 1).clamp_(0, v - 1)
    ids = torch.randperm(v, generator=gen, device="cuda")[rank]
    pad = torch.rand(t, generator=gen, device="cuda") < 0.02
    s["targets"] = torch.where(pad, torch.full_like(ids, -1), ids)
    # half of the tokens are foreseen: their hidden state leans to the target's row (its logit rises by about 8)
    lean = 2.0 * (torch.rand(t, 1, generator=gen, device="cuda") < 0.5)
    s["hidden"] = _grid(normal(t, d) + lean * whole[s["targets"].clamp(min=0)], 2.0 ** -5, 127).to(dt)
    s["whole"] = whole.to(dt)
    s["pieces"] = _pieces(s["whole"], case["p"])
    if case["op"] == "logprobs_grad":
        # advantages, and what was kept of the forward pass
        s["dlogprob"] = normal(t) / t
        s["dentropy"] = torch.full((t,), 0.01 / t, device="cuda") if case["entropy"] else None
        parts = []
        for lo in range(0, t, 1024):
            z = (s["hidden"][lo:lo + 1024].float() @ whole.t()) * case["scale"]
            z -= z.amax(1, keepdim=True)  # (the largest is added again below)
            e = z.exp()
            total = e.sum(1)
            parts.append((total.log(), total.log() - (e * z).sum(1) / total))
        s["entropy"] = torch.cat([h for _, h in parts])
        top = torch.cat([((s["hidden"][lo:lo + 1024].float() @ whole.t()) * case["scale"]).amax(1) for lo in range(0, t, 1024)])
        s["lse"] = top + torch.cat([x for x, _ in parts])
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
    if case["op"] == "logprobs":
        r = h.vocab_logprobs(s["hidden"], s["pieces"], s["targets"], top=case["top"], logit_scale=case["scale"])
        return [r.logprob, r.entropy, r.lse] + ([r.top_logprob, r.top_token] if case["top"] else [])
    if case["op"] == "logprobs_grad":
        dhidden, dweights = h.vocab_logprobs_grad(s["hidden"], s["pieces"], s["targets"], s["lse"], s["entropy"], s["dlogprob"],
                                                  dentropy=s["dentropy"], logit_scale=case["scale"])
        return [dhidden, list(dweights)]
    if case["op"] == "grad_norm":
        r = h.grad_norm(s["grads"])
        return [r.norm, r.norms]
    norm = h.grad_clip(s["grads"], s["max_norm"], out=s["out"], eps=CLIP_EPS)
    return [norm, s["flat"]]


def _plain_logprobs(s):
    case = s["case"]
    v, target = case["vocab"], s["targets"]
    z = s["hidden"].float() @ s["whole"].float().t()
    top = []
    if case["top"]:
        # order by logit, then by the lower token: one whole number for both (a 32-bit float's order is that of its bits,
        # those below the sign turned over where it is negative)
        bits = (z + 0.0).view(torch.int32).long()  # (no -0)
        order = torch.where(bits < 0, bits ^ 0x7FFFFFFF, bits)
        order = (order << 20) + (v - 1 - torch.arange(v, device=z.device))
        top_token = (v - 1) - (torch.topk(order, case["top"], dim=1).values & ((1 << 20) - 1))
        top = [top_token]
    z = z * case["scale"]
    m = z.amax(1)
    x = z - m[:, None]
    e = torch.exp(x)
    total = e.sum(1)
    log_total = torch.log(total)
    entropy = log_total - (e * x).sum(1) / total
    counts = (target >= 0) & (target < v)
    logprob = torch.where(counts, x.gather(1, target.clamp(0, v - 1)[:, None])[:, 0] - log_total, torch.zeros_like(m))
    if top:
        top = [x.gather(1, top[0]) - log_total[:, None], top[0]]
    return [logprob, entropy, m + log_total] + top


def _plain_logprobs_grad(s):
    case, dt = s["case"], DTYPES[s["case"]["dtype"]]
    v, target = case["vocab"], s["targets"]
    h, w = s["hidden"].float(), s["whole"].float()
    g = (h @ w.t()) * case["scale"] - s["lse"][:, None]  # log probabilities
    a = s["dlogprob"][:, None]
    if s["dentropy"] is None:
        g = torch.exp(g) * -a
    else:
        g = torch.exp(g) * (-a - s["dentropy"][:, None] * (g + s["entropy"][:, None]))
    counts = ((target >= 0) & (target < v))[:, None]
    g.scatter_add_(1, target.clamp(0, v - 1)[:, None], a)
    g = torch.where(counts, g * case["scale"], torch.zeros((), device=g.device))
    h = torch.where(counts, h, torch.zeros((), device=h.device))
    return [(g @ w).to(dt), _pieces((g.t() @ h).to(dt), case["p"])]


def _plain_norms(s):
    # (sums over up to 10^9 elements, in 64 bits)
    squares = torch.stack([(g.float() * g.float()).sum(dtype=torch.float64) for g in s["grads"]])
    return torch.sqrt(squares.sum()).float(), torch.sqrt(squares).float()


def _plain_grad_norm(s):
    return list(_plain_norms(s))


def _plain_grad_clip(s):
    norm = _plain_norms(s)[0]
    factor = (s["max_norm"] / (norm + CLIP_EPS)).clamp(max=1.0)
    for g, out in zip(s["grads"], s["out"]):
        out.copy_(g.float() * factor)
    return [norm, s["flat"]]


PLAIN = {"logprobs": _plain_logprobs, "logprobs_grad": _plain_logprobs_grad, "grad_norm": _plain_grad_norm, "grad_clip": _plain_grad_clip}


def run(state):
    return _run_own(state) if own else PLAIN[state["case"]["op"]](state)


def exact(case, seed):
    """The definitions in 64 bits."""
    s, op = prepare(case, seed), case["op"]
    if op in ("grad_norm", "grad_clip"):
        norms = torch.stack([torch.linalg.vector_norm(g.reshape(-1), dtype=torch.float64) for g in s["grads"]])
        norm = torch.linalg.vector_norm(norms)
        if op == "grad_norm":
            return [norm, norms]
        factor = min(1.0, s["max_norm"] / (norm.item() + CLIP_EPS))
        kinds = ["float32" if case["wide"] else kind for _, kind in _shapes(case)]
        flat, views = _flat([g.shape for g in s["grads"]], kinds, {k: torch.float64 for k in set(kinds)})
        for g, view in zip(s["grads"], views):
            view.copy_(g).mul_(factor)
        return [norm, flat]
    t, v, k = case["tokens"], case["vocab"], case.get("top", 0)
    w = s["whole"].double()
    rows, dh, dw = [], [], torch.zeros_like(w) if op == "logprobs_grad" else None
    step = max(1, (1 << 26) // v)
    for lo in range(0, t, step):
        h, target = s["hidden"][lo:lo + step].double(), s["targets"][lo:lo + step]
        z = torch.matmul(h, w.T)
        logp = torch.log_softmax(z * case["scale"], 1)
        row = torch.nonzero((target >= 0) & (target < v))[:, 0]
        at = target[row]
        if op == "logprobs":
            logprob = torch.zeros(len(h), dtype=torch.float64, device="cuda")
            logprob[row] = logp[row, at]
            lse = torch.logsumexp(z * case["scale"], 1)
            out = [logprob, -torch.sum(torch.exp(logp) * logp, 1), lse]
            if k:
                token = torch.sort(z, dim=1, descending=True, stable=True).indices[:, :k]
                out += [logp.gather(1, token), token]
            rows.append(out)
            continue
        # with the statistics as they were kept: log probabilities relative to lse, entropy as it stands
        logp = z * case["scale"] - s["lse"][lo:lo + step].double()[:, None]
        prob = torch.exp(logp)
        a = s["dlogprob"][lo:lo + step].double()
        g = prob * -a[:, None]
        if case["entropy"]:
            b = s["dentropy"][lo:lo + step].double()
            g -= prob * (logp + s["entropy"][lo:lo + step].double()[:, None]) * b[:, None]
        g[row, at] += a[row]
        keep = torch.zeros(len(h), 1, dtype=torch.float64, device="cuda")
        keep[row] = case["scale"]
        g *= keep
        dh.append(torch.matmul(g, w))
        dw += torch.matmul(g.T, h)
    if op == "logprobs":
        return [torch.cat(column) for column in zip(*rows)]
    return [torch.cat(dh), _pieces(dw, case["p"])]

"""Log probabilities, entropy and alternatives over a vocabulary in pieces
(rar_vocab_logprobs) and their gradients, against plain forms in 64 bits.

Bounds are derived from the data, as in test_model_ops: u is half a unit in the last
place of the written type, F = 2^-24 that of binary32.
"""
import ctypes
import math
import os
import subprocess
import tempfile

import pytest
import torch

import ring_all_reduce_rar_gb300 as rar
from ring_all_reduce_rar_gb300 import _ops
from tests.conftest import ROOT
from tests.test_model_ops import F, HALF, TINY, U, gen, h, normal, pieces, strided, within, xent_inputs  # noqa: F401

gpu = pytest.mark.gpu


# ------------------------------------------------------------- without a GPU

def test_struct_layouts_match_c():
    structs = {"rar_vocab_logprobs_args": _ops.VocabLogprobsArgs, "rar_vocab_logprobs_grad_args": _ops.VocabLogprobsGradArgs}
    lines = []
    for name, cls in structs.items():
        lines.append(f'printf("%zu", sizeof({name}));')
        lines += [f'printf(" %zu", offsetof({name}, {f[0]}));' for f in cls._fields_]
        lines.append('printf("\\n");')
    src = '#include <stdio.h>\n#include <stddef.h>\n#include "rar.h"\nint main(void) {' + "\n".join(lines) + "return 0; }"
    with tempfile.TemporaryDirectory() as d:
        c, exe = os.path.join(d, "probe.c"), os.path.join(d, "probe")
        with open(c, "w") as f:
            f.write(src)
        subprocess.run(["gcc", "-std=c11", "-I", os.path.join(ROOT, "include"), c, "-o", exe], check=True)
        out = subprocess.run([exe], capture_output=True, text=True, check=True).stdout.splitlines()
    for line, cls in zip(out, structs.values()):
        assert [int(v) for v in line.split()] == [ctypes.sizeof(cls)] + [getattr(cls, f[0]).offset for f in cls._fields_]


def test_refusals_without_a_gpu():
    rar.build()
    lib = rar.load_library()
    for name in ("rar_vocab_logprobs", "rar_vocab_logprobs_grad"):
        assert getattr(lib, name)(None, None, None) == 1  # RAR_EINVAL
    assert lib.rar_vocab_logprobs_workspace(10, 12, 100, 1, 0) == 0  # dim not a multiple of 8
    assert lib.rar_vocab_logprobs_workspace(10, 16, 100, 65, 0) == 0
    assert lib.rar_vocab_logprobs_workspace(10, 16, 100, 1, 33) == 0
    assert lib.rar_vocab_logprobs_workspace(10, 16, 100, 1, -1) == 0
    assert lib.rar_vocab_logprobs_grad_workspace(10, 12, 100, 1) == 0
    assert lib.rar_vocab_logprobs_grad_workspace(1 << 40, 16, 1 << 40, 1) == 0
    # far below the logits
    assert 0 < lib.rar_vocab_logprobs_workspace(65536, 1024, 262144, 8, 32) < 65536 * 262144 * 4 / 16
    assert 0 < lib.rar_vocab_logprobs_grad_workspace(65536, 1024, 262144, 8) < 65536 * 262144 * 2 / 16
    x, tok = torch.zeros(4, 8), torch.zeros(4, dtype=torch.int64)
    for call in (lambda: rar.rar_vocab_logprobs(None, x, [x], tok), lambda: rar.rar_vocab_logprobs_grad(None, x, [x], tok, x[:, 0], None, x[:, 0])):
        with pytest.raises(ValueError):
            call()


# ------------------------------------------------------------------- forward

def reference(hidden, weights, targets, scale):
    """(name: (value, bound)) in 64 bits, and the log probabilities of everything."""
    w = torch.cat([t.double() for t in weights])
    v, dim = w.shape[0], hidden.shape[1]
    counts = (targets >= 0) & (targets < v)
    z = hidden.double() @ w.T
    # a logit: dim products in any order, cut to the accumulator's 24 bits as they are added
    dz = scale * (2 * dim * F * (hidden.double().abs() @ w.abs().T)).amax(1)
    x = scale * (z - z.amax(1, keepdim=True))
    logp = torch.log_softmax(x, 1)
    prob = logp.exp()
    log_s = -logp.amax(1)
    lse = scale * z.amax(1) + log_s
    ex, ex2 = (prob * -x).sum(1), (prob * x * x).sum(1)
    # S: an exponential is off by (2 + |x|) 2^-23; moving a sum to a higher maximum costs as
    # much again, 16 times at most in sums of random order (the maximum of n batches rises
    # log n times); and the additions
    ds = 2.0 ** -18 + ex * 2.0 ** -22 + (256 + v / 256 + len(weights) + 16) * F
    entropy = log_s + ex
    dentropy = 2 * (entropy + 1) * dz + ds * (1 + ex) + (2 * ex + ex2) * 2.0 ** -22 + 4 * F * (log_s + ex)
    dlse = dz + ds + 4 * F * (lse.abs() + log_s)
    at = targets.clamp(0, v - 1).long()[:, None]
    lp = logp.gather(1, at)[:, 0]
    dlp = dz + dlse + 4 * F * lp.abs()
    zero = torch.zeros_like(lse)
    # (any log probability: its own logit and the sums)
    dany = 2 * dz[:, None] + ds[:, None] + 8 * F * (logp.abs() + log_s[:, None])
    return {"logprob": (torch.where(counts, lp, zero), torch.where(counts, dlp, zero) + 1e-300), "lse": (lse, dlse),
            "entropy": (entropy, dentropy)}, logp, dany


def check(r, ref, top):
    sums, logp, dany = ref
    for name, (value, bound) in sums.items():
        within(getattr(r, name), value, bound, name)
    if not top:
        assert r.top_logprob is None and r.top_token is None
        return
    # each alternative has its own log probability, none comes twice, and the k-th is as likely as the k-th of all
    assert r.top_token.dtype == torch.int64 and r.top_token.shape == (logp.shape[0], top) == r.top_logprob.shape
    assert bool(((r.top_token >= 0) & (r.top_token < logp.shape[1])).all())
    within(r.top_logprob, logp.gather(1, r.top_token), dany.gather(1, r.top_token), "alternatives")
    best = torch.topk(logp, top, dim=1)
    within(r.top_logprob, best.values, dany.amax(1, keepdim=True).expand_as(best.values), "alternatives' order")
    assert bool((r.top_logprob[:, 1:] <= r.top_logprob[:, :-1]).all())
    ordered = r.top_token.sort(1).values
    assert bool((ordered[:, 1:] > ordered[:, :-1]).all())


SHAPES = [
    (1, 1, 8, 1), (1, 1, 8, 2), (2, 1, 64, 300), (3, 2, 72, 1000), (4, 127, 64, 255), (4, 129, 128, 1025), (8, 128, 256, 2048),
    (8, 300, 520, 5003), (16, 33, 8, 9), (5, 513, 200, 3001), (64, 20, 64, 64), (64, 5, 16, 3), (2, 1100, 136, 777),
    (3, 256, 1024, 4099), (1, 640, 64, 16384), (4, 1, 2048, 32768), (8, 16, 4096, 10007), (3, 17, 1032, 5003), (8, 64, 2048, 20011),
    (1, 65, 2056, 3001), (2, 40, 16384, 700), (6, 2600, 64, 4100),
    (3, 128, 2048, 1501), (2, 129, 2048, 9000), (1, 64, 8192, 900), (2, 65, 8192, 300), (2, 90, 4104, 601), (1, 16, 32768, 130), (1, 17, 32768, 70),
    (2, 16700, 64, 1500), (1, 2304, 24, 70000),
]


@gpu
@pytest.mark.parametrize("dtype", HALF)
@pytest.mark.parametrize("p,tokens,dim,vocab", SHAPES)
def test_logprobs(h, dtype, p, tokens, dim, vocab):  # noqa: F811
    g = gen(tokens * 7 + vocab)
    whole, hidden, targets = xent_inputs(g, tokens, dim, vocab, dtype)
    weights = pieces(whole, p)
    first = None
    for top, scale in ((0, 1.0), (min(5, vocab), 1.0), (min(32, vocab), 0.7), (1, 3.0)):
        r = h.vocab_logprobs(hidden, weights, targets, top=top, logit_scale=scale)
        check(r, reference(hidden, weights, targets, scale), top)
        if scale == 1.0:  # the alternatives change nothing else, nor does another call
            first = first or r
            assert torch.equal(first.logprob, r.logprob) and torch.equal(first.entropy, r.entropy) and torch.equal(first.lse, r.lse)
        again = h.vocab_logprobs(hidden, weights, targets.int(), top=top, logit_scale=scale)
        assert all(x is y or torch.equal(x, y) for x, y in zip(again, r))
    h.check()


def grid_inputs(g, tokens, dim, vocab, dtype, levels=4):
    """Values whose sums of products are exact in any order, and logits that often are equal."""
    hidden = torch.randint(-levels, levels + 1, (tokens, dim), generator=g, device="cuda").to(dtype)
    whole = (torch.randint(-levels, levels + 1, (vocab, dim), generator=g, device="cuda") / 16).to(dtype)
    targets = torch.randint(0, vocab, (tokens,), generator=g, device="cuda")
    return whole, hidden, targets


@gpu
@pytest.mark.parametrize("dtype", HALF)
@pytest.mark.parametrize("p,tokens,dim,vocab", [(1, 1, 16, 4000), (3, 5, 8, 999), (4, 16, 64, 30011), (8, 64, 2048, 9001), (2, 70, 24, 5000),
                                                (5, 300, 40, 2000), (3, 1300, 16, 8191), (1, 3, 8, 40),
                                                (2, 17000, 16, 900), (4, 600, 24, 70000), (1, 2, 16, 300000)])
def test_equal_logits_go_to_the_lowest_token(h, dtype, p, tokens, dim, vocab):  # noqa: F811
    whole, hidden, targets = grid_inputs(gen(dim + vocab), tokens, dim, vocab, dtype)
    z = hidden.double() @ whole.double().T
    order = torch.sort(z, dim=1, descending=True, stable=True).indices
    assert z[0].unique().numel() < vocab  # there are equal ones
    for top in (1, 2, 7, 20, 32):
        r = h.vocab_logprobs(hidden, pieces(whole, p), targets, top=top)
        assert torch.equal(r.top_token, order[:, :top])


@gpu
@pytest.mark.parametrize("dtype", HALF)
@pytest.mark.parametrize("rising", [True, False])
@pytest.mark.parametrize("tokens", [3, 80, 300])
def test_alternatives_in_any_order_of_the_vocabulary(h, dtype, rising, tokens):  # noqa: F811
    """Logits that rise, or fall, along the vocabulary: every one is better, or worse, than all before."""
    vocab = 3000
    digits = torch.arange(vocab, device="cuda").flip(0) if not rising else torch.arange(vocab, device="cuda")
    whole = torch.zeros(vocab, 16, dtype=dtype, device="cuda")
    whole[:, 0], whole[:, 1], whole[:, 2] = digits % 16, digits // 16 % 16, digits // 256
    hidden = torch.zeros(tokens, 16, dtype=dtype, device="cuda")
    hidden[:, 0], hidden[:, 1], hidden[:, 2] = 2.0 ** -8, 2.0 ** -4, 1.0
    none = torch.zeros(tokens, dtype=torch.int64, device="cuda")
    assert torch.equal(h.vocab_logprobs(hidden * 0, pieces(whole, 3), none, top=32).top_token, torch.arange(32, device="cuda").expand(tokens, 32))  # all equal
    r = h.vocab_logprobs(hidden, pieces(whole, 3), none, top=32)
    want = torch.arange(32, device="cuda")
    assert torch.equal(r.top_token, (vocab - 1 - want if rising else want).expand(tokens, 32))


@gpu
@pytest.mark.parametrize("dtype", HALF)
@pytest.mark.parametrize("tokens", [7, 200])
def test_strides_and_targets_left_out(h, dtype, tokens):  # noqa: F811
    g = gen(4)
    whole, hidden, targets = xent_inputs(g, tokens, 96, 1000, dtype)
    targets[::3], targets[1::5] = 1000, -(1 << 40)
    weights = [strided(t, 24) for t in pieces(whole, 3)]
    r = h.vocab_logprobs(strided(hidden, 8, 8), weights, targets, top=3)
    check(r, reference(hidden, weights, targets, 1.0), 3)
    out = (targets < 0) | (targets >= 1000)
    assert bool((r.logprob[out] == 0).all()) and bool((r.logprob[~out] != 0).all())


@gpu
@pytest.mark.parametrize("tokens", [5, 150])
@pytest.mark.parametrize("dtype", HALF)
def test_bad_rows_stay_alone(h, dtype, tokens):  # noqa: F811
    """NaN in a hidden state: NaN in its own results and no alternatives; rows of the vocabulary
    with NaN or logits of -infinity are no alternatives either."""
    g = gen(16)
    whole, hidden, targets = xent_inputs(g, tokens, 64, 900, dtype)
    targets = targets.clamp(min=0)
    clean = h.vocab_logprobs(hidden, pieces(whole, 4), targets, top=8)
    bad = hidden.clone()
    bad[3, 5] = float("nan")
    r = h.vocab_logprobs(bad, pieces(whole, 4), targets, top=8)
    keep = torch.arange(tokens, device="cuda") != 3
    for x, y in zip(r, clean):
        assert torch.equal(x[keep], y[keep])
    assert bool(r.logprob[3].isnan()) and bool(r.lse[3].isnan()) and bool(r.entropy[3].isnan())
    assert bool((r.top_token[3] == -1).all()) and bool((r.top_logprob[3] == -float("inf")).all())
    # a vocabulary of 20 rows: one NaN, five -infinity
    few, ones = torch.zeros(20, 64, dtype=dtype, device="cuda"), torch.ones(tokens, 64, dtype=dtype, device="cuda")
    few[:, 0] = torch.arange(20, device="cuda")
    few[4, 7] = float("nan")
    few[10:15, 3] = -float("inf")
    r = h.vocab_logprobs(ones, pieces(few, 3), torch.zeros(tokens, dtype=torch.int64, device="cuda"), top=18)
    want = [t for t in range(19, -1, -1) if t != 4 and not 10 <= t < 15] + [-1] * 4
    assert r.top_token.tolist() == [want] * tokens
    assert bool((r.top_logprob[:, 14:] == -float("inf")).all()) and bool(r.lse.isnan().all())


@gpu
@pytest.mark.parametrize("tokens", [5, 200])
@pytest.mark.parametrize("dtype", HALF)
def test_runs_of_nan_in_the_vocabulary(h, dtype, tokens):  # noqa: F811
    """Logits around runs of rows that hold NaN are still listed, in their order."""
    vocab = 1500
    whole, hidden, targets = grid_inputs(gen(6), tokens, 16, vocab, dtype)
    z = hidden.double() @ whole.double().T
    for runs in ([(4, 8)], [(0, 64), (128, 256), (300, 304)], [(0, vocab - 40)], [(20, vocab)]):
        bad = whole.clone()
        left = torch.ones(vocab, dtype=torch.bool, device="cuda")
        for lo, hi in runs:
            bad[lo:hi, 3] = float("nan")
            left[lo:hi] = False
        order = torch.sort(torch.where(left, z, torch.full_like(z, -1e9)), dim=1, descending=True, stable=True).indices
        for top in (1, 8, 16, 32):
            r = h.vocab_logprobs(hidden, pieces(bad, 3), targets, top=top)
            n = min(top, int(left.sum()))
            assert torch.equal(r.top_token[:, :n], order[:, :n]) and bool((r.top_token[:, n:] == -1).all())


@gpu
@pytest.mark.parametrize("tokens", [3, 130])
@pytest.mark.parametrize("dtype", HALF)
def test_impossible_and_far_logits(h, dtype, tokens):  # noqa: F811
    """Rows with logits of -infinity have no part in the sums; logits of several hundred
    neither overflow nor leave an entropy below 0."""
    g = gen(21)
    whole, hidden, targets = xent_inputs(g, tokens, 64, 700, dtype, std=60.0)
    hidden = hidden.abs() + 0.25
    targets = targets.clamp(min=0)
    check(h.vocab_logprobs(hidden, pieces(whole, 3), targets, top=4), reference(hidden, pieces(whole, 3), targets, 1.0), 4)
    gone = whole.clone()
    gone[100:300, 9] = -float("inf")
    targets = targets % 100
    r = h.vocab_logprobs(hidden, pieces(gone, 3), targets, top=4)
    rest = torch.cat([whole[:100], whole[300:]])
    ref = reference(hidden, [rest], targets, 1.0)
    for name, (value, bound) in ref[0].items():
        within(getattr(r, name), value, bound, name)
    assert not bool(((r.top_token >= 100) & (r.top_token < 300)).any())


@gpu
@pytest.mark.parametrize("tokens", [3, 200])
def test_scales_at_the_ends(h, tokens):  # noqa: F811
    """A distribution that is uniform, or a single token."""
    whole, hidden, targets = grid_inputs(gen(2), tokens, 16, 700, torch.bfloat16)
    z = hidden.double() @ whole.double().T
    flat = h.vocab_logprobs(hidden, [whole], targets, logit_scale=1e-30, top=2)
    for x in (flat.lse, flat.entropy, -flat.logprob, -flat.top_logprob[:, 1]):
        assert bool(((x.double() - math.log(700)).abs() < 2.0 ** -17).all())
    sharp = h.vocab_logprobs(hidden, [whole], targets, logit_scale=2.0 ** 126, top=1)
    ties = (z == z.amax(1, keepdim=True)).sum(1).double()
    assert bool(((sharp.entropy.double() - ties.log()).abs() < 2.0 ** -17).all())
    assert bool(((sharp.top_logprob[:, 0].double() + ties.log()).abs() < 2.0 ** -17).all())


@gpu
def test_single_rows_with_any_stride(h):  # noqa: F811
    g = gen(9)
    hidden, whole = normal(g, 1, 64, dtype=torch.bfloat16), normal(g, 3, 64, dtype=torch.bfloat16)
    tok = torch.tensor([2], device="cuda")
    ref = h.vocab_logprobs(hidden, pieces(whole, 3), tok, top=2)
    lib = rar.load_library()
    for stride in (65, 68, 1 << 45):
        need = lib.rar_vocab_logprobs_workspace(1, 64, 3, 3, 2)
        out, ws = torch.empty(5, device="cuda"), torch.empty(need, dtype=torch.uint8, device="cuda")
        tokens = torch.empty(2, dtype=torch.int64, device="cuda")
        a = _ops.VocabLogprobsArgs()
        ptrs = (ctypes.c_void_p * 3)(*[t.data_ptr() for t in pieces(whole, 3)])
        a.hidden, a.hidden_stride, a.weights, a.weight_stride = hidden.data_ptr(), stride, ctypes.addressof(ptrs), stride
        a.p, a.dtype, a.tokens, a.dim, a.vocab, a.targets, a.index_bytes = 3, 2, 1, 64, 3, tok.data_ptr(), 8
        a.logit_scale, a.top, a.logprob, a.top_logprob, a.top_token = 1.0, 2, out.data_ptr(), out.data_ptr() + 4, tokens.data_ptr()
        a.workspace, a.workspace_bytes = ws.data_ptr(), need
        assert lib.rar_vocab_logprobs(h.h, ctypes.byref(a), torch.cuda.current_stream().cuda_stream) == 0, rar.rar_last_error(h.h)
        assert torch.equal(out[:1], ref.logprob) and torch.equal(out[1:3], ref.top_logprob[0]) and torch.equal(tokens, ref.top_token[0])


@gpu
def test_no_tokens(h):  # noqa: F811
    w = torch.randn(40, 16, device="cuda").bfloat16()
    e, none, nothing = torch.empty(0, 16, device="cuda", dtype=torch.bfloat16), torch.empty(0, dtype=torch.int64, device="cuda"), torch.empty(0, device="cuda")
    r = h.vocab_logprobs(e, pieces(w, 3), none, top=4)
    assert r.logprob.shape == (0,) and r.top_token.shape == (0, 4)
    dh, dw = h.vocab_logprobs_grad(e, pieces(w, 3), none, nothing, nothing, nothing, dentropy=nothing)
    assert dh.shape == (0, 16) and bool((torch.cat(dw) == 0).all())
    h.check()


# ------------------------------------------------------------------ gradients

def grad_reference(hidden, weights, targets, lse, entropy, a, b, scale):
    """(dhidden, dweights) in 64 bits with their bounds, from lse and entropy as they are given."""
    w = torch.cat([t.double() for t in weights])
    v, (tokens, dim) = w.shape[0], hidden.shape
    counts = (targets >= 0) & (targets < v)
    zero = torch.zeros(tokens, dtype=torch.float64, device="cuda")
    a = zero if a is None else torch.where(counts, a.double(), zero)
    b = zero if b is None else torch.where(counts, b.double(), zero)
    used = (a != 0) | (b != 0)
    hid = torch.where(used[:, None], hidden.double(), torch.zeros_like(hidden.double()))
    ent = torch.where(b != 0, entropy.double(), zero) if entropy is not None else zero
    lse = torch.where(used, lse.double(), zero)
    z = scale * (hid @ w.T)
    dz = scale * (2 * dim * F * (hid.abs() @ w.abs().T)).amax(1, keepdim=True)
    logq = z - lse[:, None]
    dlogq = dz + 4 * F * (z.abs() + lse.abs()[:, None])
    q = torch.exp(logq)
    dq = q * (dlogq + 2.0 ** -22 * (2 + logq.abs()))
    slope = a[:, None] + b[:, None] * (logq + ent[:, None])
    size = a.abs()[:, None] + b.abs()[:, None] * (logq.abs() + ent.abs()[:, None])
    at = targets.clamp(0, v - 1).long()[:, None]
    gmat = (-q * slope).scatter_add(1, at, a[:, None])
    gmat = torch.where(used[:, None], gmat, torch.zeros_like(gmat))
    u = U[hidden.dtype]
    most = float((a.abs() + b.abs() * ent.abs().clamp(min=1)).max()) if tokens else 0.0
    # q, the slope, their product and the target's part; the rounding to 16 bits, and what lies below the smallest of them
    onehot = torch.zeros_like(q).scatter_(1, at, a.abs()[:, None])
    dg = dq * slope.abs() + q * (b.abs()[:, None] * dlogq + 8 * F * size) + 4 * F * onehot
    dg = dg * (1 + u) + (u + 4 * F) * gmat.abs() + most * 2.0 ** -37
    dg = torch.where(used[:, None], dg, torch.zeros_like(dg))
    dh, mh = gmat @ w, gmat.abs() @ w.abs()
    ddh = dg @ w.abs() + 2 * v * F * mh
    dw, mw = gmat.T @ hid, gmat.abs().T @ hid.abs()
    ddw = dg.T @ hid.abs() + 2 * (tokens + 8) * F * mw
    tiny = TINY[hidden.dtype]
    return [(scale * x, scale * (e + u * (x.abs() + e)) * (1 + 4 * F) + tiny) for x, e in ((dh, ddh), (dw, ddw))]


def check_grad(got, ref, what=""):
    within(got[0], *ref[0], what + " dhidden")
    within(torch.cat(got[1]), *ref[1], what + " dweights")


@gpu
@pytest.mark.parametrize("dtype", HALF)
@pytest.mark.parametrize("p,tokens,dim,vocab", [
    (1, 1, 8, 2), (2, 1, 64, 300), (4, 127, 64, 255), (4, 129, 128, 1025), (8, 300, 520, 5003), (16, 33, 8, 9), (64, 5, 16, 3),
    (2, 1100, 136, 777), (3, 256, 1024, 4099), (3, 333, 1032, 5003), (8, 515, 2048, 10007), (1, 4096, 256, 33000), (3, 8192, 1288, 16700),
    (16, 1569, 480, 854), (8, 2000, 64, 3001), (1, 512, 64, 900), (1, 513, 64, 900),
])
def test_gradients(h, dtype, p, tokens, dim, vocab):  # noqa: F811
    g = gen(tokens * 7 + vocab)
    whole, hidden, targets = xent_inputs(g, tokens, dim, vocab, dtype)
    weights = pieces(whole, p)
    a, b = normal(g, tokens) / tokens, normal(g, tokens, std=0.1) / tokens
    for scale, da, db in ((1.0, a, None), (1.0, a, b), (0.6, None, b), (1.7, a, b)):
        r = h.vocab_logprobs(hidden, weights, targets, logit_scale=scale)
        call = lambda t=targets: h.vocab_logprobs_grad(hidden, weights, t, r.lse, r.entropy, da, dentropy=db, logit_scale=scale)  # noqa: E731
        got = call()
        check_grad(got, grad_reference(hidden, weights, targets, r.lse, r.entropy, da, db, scale), f"{scale}")
        again = call(targets.int())
        assert torch.equal(again[0], got[0]) and all(torch.equal(x, y) for x, y in zip(again[1], got[1]))
    h.check()


@gpu
@pytest.mark.parametrize("dtype", HALF)
def test_gradient_of_a_loss_is_that_of_the_cross_entropy(h, dtype):  # noqa: F811
    """With a = -token_weight it is the cross entropy's gradient, from the same sums in another order."""
    g = gen(3)
    whole, hidden, targets = xent_inputs(g, 333, 520, 5003, dtype)
    tw = torch.rand(333, generator=g, device="cuda") / 333
    x = h.vocab_xent(hidden, pieces(whole, 3), targets, token_weight=tw, grad=True)
    ref = grad_reference(hidden, pieces(whole, 3), targets, x.lse, None, -tw, None, 1.0)
    check_grad((x.dhidden, x.dweights), ref)
    check_grad(h.vocab_logprobs_grad(hidden, pieces(whole, 3), targets, x.lse, None, -tw), ref)


@gpu
@pytest.mark.parametrize("dtype", HALF)
def test_gradients_of_tokens_left_out(h, dtype):  # noqa: F811
    """Tokens without a target or without weights hold infinities and NaN."""
    g = gen(6)
    whole, hidden, targets = xent_inputs(g, 200, 64, 600, dtype)
    a, b = normal(g, 200), normal(g, 200)
    a[::7] = b[::7] = 0.0
    out = (targets < 0) | (a == 0)
    r = h.vocab_logprobs(hidden, pieces(whole, 2), targets)
    ref = grad_reference(hidden, [whole], targets, r.lse, r.entropy, a, b, 1.0)
    bad = hidden.clone()
    bad[out] = float("nan")
    bad[int(out.nonzero()[0]), 3] = float("inf")
    s = h.vocab_logprobs(bad, pieces(whole, 2), targets)
    got = h.vocab_logprobs_grad(bad, pieces(whole, 2), targets, s.lse, s.entropy, a, dentropy=b)
    assert bool((got[0][out] == 0).all())
    check_grad(got, ref)
    for none in (torch.full_like(targets, 600), torch.full_like(targets, -1)):
        got = h.vocab_logprobs_grad(bad, pieces(whole, 2), none, s.lse, s.entropy, a, dentropy=b)
        assert bool((got[0] == 0).all()) and bool((torch.cat(got[1]) == 0).all())
    zero = torch.zeros(200, device="cuda")
    got = h.vocab_logprobs_grad(bad, pieces(whole, 2), targets, s.lse, s.entropy, zero, dentropy=zero)
    assert bool((got[0] == 0).all()) and bool((torch.cat(got[1]) == 0).all())


@gpu
@pytest.mark.parametrize("dtype", HALF)
def test_gradients_with_weights_far_apart(h, dtype):  # noqa: F811
    """Token weights over twelve powers of ten, peaked distributions."""
    g = gen(26)
    whole, hidden, targets = xent_inputs(g, 130, 128, 700, dtype, std=20.0)
    a = 10.0 ** (-12 * torch.rand(130, generator=g, device="cuda"))
    b = -0.01 * a
    r = h.vocab_logprobs(hidden, pieces(whole, 3), targets)
    got = h.vocab_logprobs_grad(hidden, pieces(whole, 3), targets, r.lse, r.entropy, a, dentropy=b)
    check_grad(got, grad_reference(hidden, pieces(whole, 3), targets, r.lse, r.entropy, a, b, 1.0))


@gpu
@pytest.mark.parametrize("dtype", HALF)
def test_gradients_against_differences(h, dtype):  # noqa: F811
    g = gen(41)
    tokens, dim, vocab, scale = 24, 64, 333, 1.3
    whole, hidden, targets = xent_inputs(g, tokens, dim, vocab, dtype)
    a, b = normal(g, tokens), normal(g, tokens)
    r = h.vocab_logprobs(hidden, pieces(whole, 3), targets, logit_scale=scale)
    dh, dw = h.vocab_logprobs_grad(hidden, pieces(whole, 3), targets, r.lse, r.entropy, a, dentropy=b, logit_scale=scale)
    ref = grad_reference(hidden, pieces(whole, 3), targets, r.lse, r.entropy, a, b, scale)
    counts = (targets >= 0).double()

    def value(hid, w):
        logp = torch.log_softmax(scale * (hid @ w.T), 1)
        lp = logp.gather(1, targets.clamp(min=0)[:, None])[:, 0]
        return float((counts * (a.double() * lp - b.double() * (logp.exp() * logp).sum(1))).sum())

    for _ in range(4):
        eh, ew = normal(g, tokens, dim).double(), normal(g, vocab, dim).double()
        step = 1e-5
        diff = (value(hidden.double() + step * eh, whole.double() + step * ew) - value(hidden.double() - step * eh, whole.double() - step * ew)) / (2 * step)
        own = float((dh.double() * eh).sum() + (torch.cat(dw).double() * ew).sum())
        bound = float((ref[0][1] * eh.abs()).sum() + (ref[1][1] * ew.abs()).sum())
        # lse and entropy are off by their own bounds, which a step of 1e-5 does not reach: 1e-3 of
        # the differences' curvature and of 64-bit cancellation together
        assert abs(own - diff) <= bound + 1e-3 * (1 + abs(diff))


@gpu
def test_gradients_separately(h):  # noqa: F811
    """dhidden without dweights and the other way round, through the C call, into matrices with gaps."""
    g = gen(31)
    whole, hidden, targets = xent_inputs(g, 90, 64, 500, torch.bfloat16)
    a = normal(g, 90)
    r = h.vocab_logprobs(hidden, [whole], targets)
    ref = h.vocab_logprobs_grad(hidden, [whole], targets, r.lse, None, a)
    lib = rar.load_library()
    need = lib.rar_vocab_logprobs_grad_workspace(90, 64, 500, 1)
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    for which in ("dhidden", "dweights"):
        k = _ops.VocabLogprobsGradArgs()
        wp = (ctypes.c_void_p * 1)(whole.data_ptr())
        k.hidden, k.weights, k.p, k.dtype = hidden.data_ptr(), ctypes.addressof(wp), 1, 2
        k.tokens, k.dim, k.vocab, k.targets, k.index_bytes, k.logit_scale = 90, 64, 500, targets.data_ptr(), 8, 1.0
        k.lse, k.dlogprob, k.workspace, k.workspace_bytes = r.lse.data_ptr(), a.data_ptr(), ws.data_ptr(), need
        like = ref[0] if which == "dhidden" else ref[1][0]
        big = torch.full((like.shape[0], 80), 7.0, dtype=torch.bfloat16, device="cuda")
        op = (ctypes.c_void_p * 1)(big.data_ptr())
        if which == "dhidden":
            k.dhidden, k.dhidden_stride = big.data_ptr(), 80
        else:
            k.dweights, k.dweight_stride = ctypes.addressof(op), 80
        assert lib.rar_vocab_logprobs_grad(h.h, ctypes.byref(k), torch.cuda.current_stream().cuda_stream) == 0
        assert torch.equal(big[:, :64], like) and bool((big[:, 64:] == 7).all())


# ------------------------------------------- streams, graphs, waits, refusals

@gpu
@pytest.mark.parametrize("tokens", [9, 96])
def test_on_another_stream_and_in_a_graph(h, tokens):  # noqa: F811
    g = gen(61)
    dim, vocab, p = 256, 1000, 4
    whole = normal(g, vocab, dim, dtype=torch.bfloat16, std=0.1)
    weights, hidden = pieces(whole, p), normal(g, tokens, dim, dtype=torch.bfloat16)
    tok = torch.randint(0, vocab, (tokens,), generator=g, device="cuda")
    a, b = normal(g, tokens), normal(g, tokens)

    def step(stream=None):
        r = h.vocab_logprobs(hidden, weights, tok, top=6, logit_scale=0.9, stream=stream)
        dh, dw = h.vocab_logprobs_grad(hidden, weights, tok, r.lse, r.entropy, a, dentropy=b, logit_scale=0.9, stream=stream)
        return list(r) + [dh] + dw

    first = step()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    other = step(side)
    side.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(first, other))
    graphs = []
    for _ in range(2):  # two graphs, each with workspaces of its own, replayed in turn
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            held = step()
        graphs.append((graph, held))
    for k in range(4):
        tok.copy_(torch.randint(0, vocab, (tokens,), generator=g, device="cuda"))
        hidden.normal_(generator=g)
        graph, held = graphs[k % 2]
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in held]
        assert all(torch.equal(x, y) for x, y in zip(step(), got))


@gpu
@pytest.mark.parametrize("mute", [0, 2])
@pytest.mark.parametrize("tokens,dim,vocab", [(300, 256, 5000), (4, 64, 40), (16, 1288, 20000), (600, 1288, 9000)])
def test_a_muted_piece_times_out(h, tokens, dim, vocab, mute):  # noqa: F811
    g = gen(tokens + mute)
    hidden, whole = normal(g, tokens, dim, dtype=torch.bfloat16), normal(g, vocab, dim, dtype=torch.bfloat16, std=0.1)
    targets = torch.randint(0, vocab, (tokens,), generator=g, device="cuda")
    a = normal(g, tokens)
    ref = h.vocab_logprobs(hidden, pieces(whole, 3), targets, top=5)
    grads = h.vocab_logprobs_grad(hidden, pieces(whole, 3), targets, ref.lse, None, a)
    for call, want in ((lambda m: list(m.vocab_logprobs(hidden, pieces(whole, 3), targets, top=5)), list(ref)),
                       (lambda m: [(r := m.vocab_logprobs_grad(hidden, pieces(whole, 3), targets, ref.lse, None, a))[0], *r[1]], [grads[0], *grads[1]])):
        with rar.Handle(0, fault_rank=mute, timeout_ns=50_000_000, fault_mode="mute") as faulty:
            call(faulty)
            assert faulty.status() == 5  # RAR_ETIMEOUT
            assert "log probabilities" in rar.rar_last_error(faulty.h)
            assert faulty.status() == 0
            faulty.set_options()
            assert all(torch.equal(x, y) for x, y in zip(call(faulty), want))
            faulty.check()


@gpu
def test_refusals(h):  # noqa: F811
    half = torch.ones(4, 64, dtype=torch.bfloat16, device="cuda")
    tok, one = torch.zeros(4, dtype=torch.int64, device="cuda"), torch.ones(4, device="cuda")
    for call in (lambda: h.vocab_logprobs(half, [half, half[:2]], tok), lambda: h.vocab_logprobs(half, [half], tok[:2]),
                 lambda: h.vocab_logprobs(half, [half], tok.float()), lambda: h.vocab_logprobs(half, [half], tok, top=5),
                 lambda: h.vocab_logprobs(half, [half], tok, top=-1), lambda: h.vocab_logprobs(half.expand(4, 64)[:1].expand(4, 64), [half], tok),
                 lambda: h.vocab_logprobs(half, [torch.ones(40, 64, dtype=torch.bfloat16, device="cuda")], tok, top=33),
                 lambda: h.vocab_logprobs_grad(half, [half], tok, one, one, None), lambda: h.vocab_logprobs_grad(half, [half], tok, one, None, one, dentropy=one),
                 lambda: h.vocab_logprobs_grad(half, [half], tok, one[:2], None, one), lambda: h.vocab_logprobs_grad(half, [half], tok, None, None, one),
                 lambda: h.vocab_logprobs_grad(half, [half], tok, one, None, one.half())):
        with pytest.raises(ValueError):
            call()
    x = torch.ones(4, 64, device="cuda")
    for code, call in ((2, lambda: h.vocab_logprobs(x, [x], tok)), (1, lambda: h.vocab_logprobs(half[:, :60], [half[:, :60]], tok)),
                       (1, lambda: h.vocab_logprobs(strided(half, 1), [half], tok)),
                       (1, lambda: h.vocab_logprobs(half, pieces(torch.zeros(65, 64, dtype=torch.bfloat16, device="cuda"), 65), tok)),
                       (1, lambda: h.vocab_logprobs(half, [half], tok, logit_scale=0.0)), (1, lambda: h.vocab_logprobs(half, [half], tok, logit_scale=float("nan"))),
                       (1, lambda: h.vocab_logprobs(half, [half], tok, logit_scale=float("inf"))), (1, lambda: h.vocab_logprobs(half, [half], tok, logit_scale=-1.0)),
                       (1, lambda: h.vocab_logprobs(half, [half], tok, logit_scale=2.0 ** 127)),
                       (1, lambda: h.vocab_logprobs_grad(half, [half], tok, one, None, one, logit_scale=0.0)),
                       (2, lambda: h.vocab_logprobs_grad(x, [x], tok, one, None, one))):
        with pytest.raises(rar.RarError) as e:
            call()
        assert e.value.code == code
    # through the C call: a short workspace, an output that lies on an input, alternatives without a place
    lib, stream = rar.load_library(), torch.cuda.current_stream().cuda_stream
    need = lib.rar_vocab_logprobs_workspace(4, 64, 4, 1, 0)
    ws, out = torch.empty(need, dtype=torch.uint8, device="cuda"), torch.empty(8, device="cuda")
    wp = (ctypes.c_void_p * 1)(half.data_ptr())

    def args(**kw):
        a = _ops.VocabLogprobsArgs()
        a.hidden, a.weights, a.p, a.dtype = half.data_ptr(), ctypes.addressof(wp), 1, 2
        a.tokens, a.dim, a.vocab, a.targets, a.index_bytes, a.logit_scale = 4, 64, 4, tok.data_ptr(), 8, 1.0
        a.logprob, a.workspace, a.workspace_bytes = out.data_ptr(), ws.data_ptr(), need
        for k, v in kw.items():
            setattr(a, k, v)
        return ctypes.byref(a)

    for bad in (dict(workspace_bytes=need - 1), dict(workspace=None), dict(logprob=half.data_ptr()), dict(entropy=out.data_ptr() + 8), dict(top=2),
                dict(top=33), dict(top=-1), dict(index_bytes=2), dict(p=0), dict(dim=0), dict(vocab=0), dict(weights=None), dict(targets=None),
                dict(tokens=1 << 60), dict(lse=ws.data_ptr())):
        assert lib.rar_vocab_logprobs(h.h, args(**bad), stream) == 1, bad
    assert lib.rar_vocab_logprobs(h.h, args(), stream) == 0
    h.check()

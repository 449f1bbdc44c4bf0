"""The model operators (rar_add_rmsnorm, rar_vocab_xent, rar_embedding and
their gradients) against plain forms in 64 bits.

Tolerances are bounds, element by element, derived from the data: u is half a
unit in the last place of the written type (2^-8 for the 8 significant bits of
bfloat16, 2^-11 for the 11 of float16), F = 2^-24 that of binary32.  A sum of
n binary32 terms is off by at most n F times the sum of their magnitudes.
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

F = 2.0 ** -24
U = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
# half the smallest step of the written type
TINY = {torch.float32: 2.0 ** -150, torch.bfloat16: 2.0 ** -134, torch.float16: 2.0 ** -25}
DTYPES = [torch.float32, torch.bfloat16, torch.float16]
HALF = [torch.bfloat16, torch.float16]
gpu = pytest.mark.gpu


@pytest.fixture(scope="module")
def h():
    rar.build()
    with rar.Handle(0) as handle:
        yield handle


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def normal(g, *shape, dtype=torch.float32, std=1.0):
    return (torch.randn(*shape, generator=g, device="cuda") * std).to(dtype)


def strided(t, extra, offset=0):
    """The same values with `extra` columns between the rows, the first row
    `offset` elements into its memory."""
    rows, cols = t.shape
    big = torch.full((rows * (cols + extra) + offset,), float("nan"), dtype=t.dtype, device=t.device)
    view = big[offset:].view(rows, cols + extra)[:, :cols]
    view.copy_(t)
    return view


def pieces(whole, p):
    base, extra = divmod(whole.shape[0], p)
    return list(whole.split([base + 1] * extra + [base] * (p - extra)))


def within(got, ref, tol, what):
    got = got.double()
    assert got.shape == ref.shape, what
    bad = ~((got - ref).abs() <= tol)
    assert not bool(bad.any()), f"{what}: {int(bad.sum())} of {bad.numel()} off, worst {float(((got - ref).abs() / tol)[bad].max())} x"


# ------------------------------------------------------------- without a GPU

def test_struct_layouts_match_c():
    structs = {"rar_rmsnorm_args": _ops.RmsNormArgs, "rar_rmsnorm_grad_args": _ops.RmsNormGradArgs,
               "rar_vocab_xent_args": _ops.VocabXentArgs, "rar_embedding_args": _ops.EmbeddingArgs,
               "rar_embedding_grad_args": _ops.EmbeddingGradArgs}
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


def test_null_handles_are_refused():
    rar.build()
    lib = rar.load_library()
    for name in ("rar_add_rmsnorm", "rar_add_rmsnorm_grad", "rar_vocab_xent", "rar_embedding", "rar_embedding_grad"):
        assert getattr(lib, name)(None, None, None) == 1  # RAR_EINVAL


def test_workspace_sizes():
    rar.build()
    lib = rar.load_library()
    assert lib.rar_add_rmsnorm_grad_workspace(10, 0) == 0
    assert lib.rar_vocab_xent_workspace(10, 12, 100, 1, 1) == 0  # dim not a multiple of 8
    assert lib.rar_vocab_xent_workspace(10, 16, 100, 65, 1) == 0
    few, many = (lib.rar_vocab_xent_workspace(t, 64, 50000, 8, 1) for t in (16, 4096))
    assert 0 < few < many
    # far below the logits
    assert lib.rar_vocab_xent_workspace(65536, 1024, 262144, 8, 1) < 65536 * 262144 * 2 / 16


def test_cpu_tensors_are_refused():
    x = torch.zeros(4, 8)
    with pytest.raises(ValueError):
        rar.rar_add_rmsnorm(None, [x])
    with pytest.raises(ValueError):
        rar.rar_embedding(None, [x], torch.zeros(2, dtype=torch.int64))
    with pytest.raises(ValueError):
        rar.rar_vocab_xent(None, x, [x], torch.zeros(4, dtype=torch.int64))


# -------------------------------------------------------------- add_rmsnorm

def norm_reference(parts, residual, weight, eps):
    """(s, rstd, y) in 64 bits and the bounds of their binary32 values."""
    n, p, dim = parts[0].shape[1], len(parts), parts[0].shape[1]
    s = sum(t.double() for t in parts)
    mag = sum(t.double().abs() for t in parts)
    if residual is not None:
        s, mag = s + residual.double(), mag + residual.double().abs()
    w = torch.ones(n, dtype=torch.float64, device="cuda") if weight is None else weight.double()
    ms = (s ** 2).mean(1) + eps
    rstd = ms.rsqrt()
    ds = (p + 1) * F * mag
    # squares: n + 4 roundings, and the error of s itself
    dms = (dim + 4) * F * ms + 2 * (s.abs() * ds).mean(1)
    drel = 0.5 * dms / ms + 4 * F  # of rstd
    y = s * rstd[:, None] * w
    dy = y.abs() * (drel[:, None] + 4 * F) + ds * rstd[:, None] * w.abs()
    return s, rstd, y, ds, drel, dy


def check_norm(r, dtype, ref, group):
    s, rstd, y, ds, drel, dy = ref
    within(r.sum, s, U[dtype] * (s.abs() + ds) + ds + TINY[dtype], "sum")
    within(r.rstd, rstd, rstd * drel, "rstd")
    if r.out is not None:
        within(r.out, y, U[dtype] * (y.abs() + dy) + dy + TINY[dtype], "out")
    if group is None:
        assert r.out8 is None and r.scales is None
        return
    dim = y.shape[1]
    g = group or dim
    for k, lo in enumerate(range(0, dim, g)):
        block, db = y[:, lo:lo + g], dy[:, lo:lo + g]
        amax = block.abs().amax(1)
        scale = (amax / 448).clamp(min=2.0 ** -126)
        within(r.scales[:, k], scale, scale * 4 * F + db.amax(1) / 448 + TINY[torch.float32], "scales")
        mine = r.scales[:, k].double()[:, None]
        back = r.out8[:, lo:lo + g].float().double() * mine
        # 3 bits of mantissa; steps of 2^-9 below the normal codes; two roundings of the quotient
        within(back, block, (block.abs() + db) * (2.0 ** -4 + 4 * F) + mine * 2.0 ** -10 + db, "codes")
    assert r.scales.shape[1] == -(-dim // g)


@gpu
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("p,rows,dim,group", [
    (1, 1, 1, None), (1, 1, 1, 0), (2, 3, 7, 0), (3, 5, 33, 32), (4, 17, 128, 128), (8, 4, 2048, 128), (8, 1, 4096, 0),
    (5, 9, 1001, 128), (16, 33, 520, 64), (7, 300, 1024, None), (2, 2000, 264, 128), (64, 3, 96, 32), (70, 2, 40, None),
    (8, 21, 8192, 128), (2, 3, 12288, 0), (3, 2, 32768, 4096), (2, 2, 20001, 96),
])
def test_add_rmsnorm(h, dtype, p, rows, dim, group):
    g = gen(p * 1000 + rows)
    parts = [normal(g, rows, dim, dtype=dtype) for _ in range(p)]
    residual, weight = normal(g, rows, dim, dtype=dtype, std=2.0), normal(g, dim, dtype=dtype)
    r = h.add_rmsnorm(parts, weight, residual=residual, eps=1e-5, quant_group=group, keep_out=True)
    check_norm(r, dtype, norm_reference(parts, residual, weight, 1e-5), group)
    again = h.add_rmsnorm(parts, weight, residual=residual, eps=1e-5, quant_group=group)
    assert torch.equal(r.sum, again.sum) and torch.equal(r.rstd, again.rstd)
    if group is not None:
        assert again.out is None
        assert torch.equal(r.out8.view(torch.uint8), again.out8.view(torch.uint8)) and torch.equal(r.scales, again.scales)
    h.check()


@gpu
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("extra,offset", [(0, 1), (3, 0), (8, 8), (5, 2)])
def test_add_rmsnorm_strides_and_alignment(h, dtype, extra, offset):
    g = gen(5)
    p, rows, dim = 3, 11, 264
    parts = [strided(normal(g, rows, dim, dtype=dtype), extra, offset) for _ in range(p)]
    residual = strided(normal(g, rows, dim, dtype=dtype), extra + 1, 0)
    r = h.add_rmsnorm(parts, None, residual=residual, quant_group=64, keep_out=True)
    check_norm(r, dtype, norm_reference(parts, residual, None, 1e-6), 64)
    r = h.add_rmsnorm(parts)
    check_norm(r, dtype, norm_reference(parts, None, None, 1e-6), None)


@gpu
@pytest.mark.parametrize("p,rows,dim", [(3, 5, 33), (4, 1, 4099), (8, 40, 1024), (16, 1, 7)])
def test_add_rmsnorm_sum_has_the_rings_order(h, p, rows, dim):
    """Without a residual, the float32 sum is rar_allreduce's, bit for bit."""
    g = gen(p)
    parts = [normal(g, rows, dim) for _ in range(p)]
    r = h.add_rmsnorm(parts)
    copies = [t.clone() for t in parts]
    h.allreduce(copies)
    assert torch.equal(r.sum, copies[0])


@gpu
def test_add_rmsnorm_codes_are_the_rounded_quotients(h):
    g = gen(9)
    x = normal(g, 64, 1024) * torch.exp(4 * torch.randn(64, 1, generator=g, device="cuda"))
    r = h.add_rmsnorm([x], quant_group=128, keep_out=True)
    q = (r.out.view(64, 8, 128) / r.scales[:, :, None]).view(64, 1024).to(torch.float8_e4m3fn)
    assert torch.equal(r.out8.view(torch.uint8), q.view(torch.uint8))


@gpu
@pytest.mark.parametrize("dtype", DTYPES)
def test_add_rmsnorm_special_values(h, dtype):
    """Rows of zeros, of the smallest values, with an infinity, with a NaN."""
    dim = 256
    x = torch.ones(6, dim, dtype=dtype, device="cuda")
    x[0] = 0
    x[1] = torch.finfo(dtype).smallest_normal
    x[2, 7] = float("inf")
    x[3, 200] = float("nan")
    x[4] = torch.finfo(dtype).max if dtype != torch.float16 else 60000.0
    w = torch.ones(dim, dtype=dtype, device="cuda")
    w[3] = float("inf")
    r = h.add_rmsnorm([x], quant_group=128, keep_out=True)
    codes = r.out8.float()
    assert bool((r.out[0] == 0).all()) and bool((codes[0] == 0).all()) and bool((r.scales[0] == 2.0 ** -126).all())
    assert bool(torch.isfinite(r.out[1].float()).all()) and bool(torch.isfinite(codes[1]).all())
    # inf: rstd 0, its own value NaN, the others 0
    assert bool(r.out[2, 7].isnan()) and bool(codes[2, 7].isnan()) and int(codes[2].isnan().sum()) == 1
    assert bool((codes[2, 128:] == 0).all())
    assert bool(r.out[3].isnan().all()) and bool(codes[3].isnan().all()) and bool(torch.isfinite(r.scales).all())
    if dtype != torch.float32:  # the squares of float32's largest values are out of range: rstd 0
        assert bool(((r.out[4].float() - 1).abs() < 2.0 ** -7).all()) or dtype == torch.bfloat16
    # ones: 1 / sqrt(1 + eps), a few roundings of binary32 and one of the type
    one = (1 + 1e-6) ** -0.5
    assert bool(((r.out[5].double() - one).abs() <= U[dtype] + 8 * F).all())
    # an infinite weight: its value saturates, NaN-free elsewhere
    r = h.add_rmsnorm([x[5:]], w, quant_group=128)
    assert float(r.out8[0, 3].float()) == 448.0 and bool(torch.isfinite(r.scales).all())
    assert bool((r.out8[0, 128:].float() == 448.0).all())


@gpu
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("dim", [130, 1024])
def test_add_rmsnorm_in_place(h, dtype, dim):
    """sum over the residual and out over a part, through the C call."""
    g = gen(77)
    p, rows = 4, 37
    parts = [normal(g, rows, dim, dtype=dtype) for _ in range(p)]
    residual = normal(g, rows, dim, dtype=dtype)
    ref = norm_reference(parts, residual, None, 1e-6)
    expect = h.add_rmsnorm(parts, residual=residual)
    a = _ops.RmsNormArgs()
    ptrs = (ctypes.c_void_p * p)(*[t.data_ptr() for t in parts])
    a.parts, a.p, a.dtype, a.rows, a.dim, a.eps = ctypes.addressof(ptrs), p, rar.DTYPE_CODES[str(dtype)[6:]], rows, dim, 1e-6
    a.residual = a.sum = residual.data_ptr()
    a.out = parts[2].data_ptr()
    assert rar.load_library().rar_add_rmsnorm(h.h, ctypes.byref(a), torch.cuda.current_stream().cuda_stream) == 0
    assert torch.equal(residual, expect.sum) and torch.equal(parts[2], expect.out)
    check_norm(expect, dtype, ref, None)


@gpu
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows,dim,plain", [
    (1, 1, False), (1, 8, True), (3, 33, False), (17, 256, True), (1027, 1001, False), (2100, 264, False), (64, 4096, False),
    (5, 12296, False), (2, 32768, False), (700, 2048, False), (9, 8192, True),
])
def test_add_rmsnorm_grad(h, dtype, rows, dim, plain):
    g = gen(rows + dim)
    s, dout = normal(g, rows, dim, dtype=dtype, std=2.0), normal(g, rows, dim, dtype=dtype)
    dsum = None if plain else normal(g, rows, dim, dtype=dtype)
    weight = None if plain else normal(g, dim, dtype=dtype)
    rstd = ((s.double() ** 2).mean(1) + 1e-6).rsqrt().float()
    dx, dweight = h.add_rmsnorm_grad(dout, s, rstd, weight, dsum=dsum)
    check_norm_grad(dx, dweight, dout, s, rstd, weight, dsum)
    again = h.add_rmsnorm_grad(dout, s, rstd, weight, dsum=dsum)
    assert torch.equal(dx, again[0]) and torch.equal(dweight, again[1])


def check_norm_grad(dx, dweight, dout, s, rstd, weight, dsum):
    dtype, (rows, dim) = s.dtype, s.shape
    x, dy, r = s.double(), dout.double(), rstd.double()[:, None]
    a = dy if weight is None else dy * weight.double()
    add = torch.zeros_like(x) if dsum is None else dsum.double()
    dot, mag = (a * x).sum(1, keepdim=True), (a * x).abs().sum(1, keepdim=True)
    ref = add + a * r - x * r ** 3 * dot / dim
    # 8 roundings of each term, and dim + 2 of the dot product's magnitudes
    dref = 8 * F * (add.abs() + a.abs() * r + x.abs() * r ** 3 * dot.abs() / dim) + x.abs() * r ** 3 * (dim + 2) * F * mag / dim
    within(dx, ref, U[dtype] * (ref.abs() + dref) + dref + TINY[dtype], "dx")
    terms = dy * x * r
    ref, dref = terms.sum(0), (rows + 3) * F * terms.abs().sum(0)
    within(dweight, ref, U[dtype] * (ref.abs() + dref) + dref + TINY[dtype], "dweight")


@gpu
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("extra,offset", [(0, 1), (3, 0), (8, 8)])
def test_add_rmsnorm_grad_strides(h, dtype, extra, offset):
    g = gen(3)
    rows, dim = 13, 520
    s, dout, dsum = (strided(normal(g, rows, dim, dtype=dtype), extra, offset) for _ in range(3))
    rstd = ((s.double() ** 2).mean(1) + 1e-6).rsqrt().float()
    check_norm_grad(*h.add_rmsnorm_grad(dout, s, rstd, None, dsum=dsum), dout, s, rstd, None, dsum)


@gpu
def test_add_rmsnorm_grad_empty_and_in_place(h):
    e = torch.empty(0, 64, device="cuda")
    dx, dw = h.add_rmsnorm_grad(e, e, torch.empty(0, device="cuda"))
    assert dx.shape == (0, 64) and bool((dw == 0).all())
    for dim in (130, 2048):
        g = gen(8)
        s, dout, dsum = (normal(g, 40, dim, dtype=torch.bfloat16) for _ in range(3))
        rstd = ((s.double() ** 2).mean(1) + 1e-6).rsqrt().float()
        expect = h.add_rmsnorm_grad(dout, s, rstd, None, dsum=dsum)
        for over in (dout, dsum):
            d = {"dout": dout.clone(), "dsum": dsum.clone()}
            dw = torch.empty(dim, dtype=torch.bfloat16, device="cuda")
            need = rar.load_library().rar_add_rmsnorm_grad_workspace(40, dim)
            ws = torch.empty(need, dtype=torch.uint8, device="cuda")
            a = _ops.RmsNormGradArgs()
            a.dtype, a.rows, a.dim, a.sum, a.rstd = 2, 40, dim, s.data_ptr(), rstd.data_ptr()
            a.dout, a.dsum, a.dweight = d["dout"].data_ptr(), d["dsum"].data_ptr(), dw.data_ptr()
            a.dx = d["dout" if over is dout else "dsum"].data_ptr()
            a.workspace, a.workspace_bytes = ws.data_ptr(), need
            assert rar.load_library().rar_add_rmsnorm_grad(h.h, ctypes.byref(a), torch.cuda.current_stream().cuda_stream) == 0
            assert torch.equal(d["dout" if over is dout else "dsum"], expect[0]) and torch.equal(dw, expect[1])


@gpu
def test_add_rmsnorm_grad_against_differences(h):
    """<gradient, direction> against central differences of the 64-bit forward
    pass, L = sum(dout y) + sum(dsum s)."""
    g = gen(21)
    rows, dim = 6, 200
    s, dout, dsum, w = normal(g, rows, dim), normal(g, rows, dim), normal(g, rows, dim), normal(g, dim)
    rstd = ((s.double() ** 2).mean(1) + 1e-6).rsqrt().float()
    dx, dweight = h.add_rmsnorm_grad(dout, s, rstd, w, dsum=dsum)

    def loss(x, weight):
        y = x * ((x ** 2).mean(1, keepdim=True) + 1e-6).rsqrt() * weight
        return float((dout.double() * y).sum() + (dsum.double() * x).sum())

    for k in range(5):
        dirx, dirw = normal(g, rows, dim).double(), normal(g, dim).double()
        step = 1e-5
        diff = (loss(s.double() + step * dirx, w.double() + step * dirw) -
                loss(s.double() - step * dirx, w.double() - step * dirw)) / (2 * step)
        own = float((dx.double() * dirx).sum() + (dweight.double() * dirw).sum())
        # binary32 gradients of magnitude ~ 1 in ~ 1400 places, rounding of the loss / step
        mag = float((dx.double() * dirx).abs().sum() + (dweight.double() * dirw).abs().sum())
        assert abs(own - diff) < 64 * F * mag + 1e-6


# --------------------------------------------------------------- vocab_xent

def xent_reference(hidden, weights, targets, token_weight):
    """Loss, lse and gradients in 64 bits, with their bounds."""
    w = torch.cat([t.double() for t in weights])
    v, (tokens, dim) = w.shape[0], hidden.shape
    hid = hidden.double()
    counts = (targets >= 0) & (targets < v)
    z = hid @ w.T
    # a logit: dim products, whatever order the tensor cores add them in (their
    # alignment may drop bits as a truncation does: twice the bound of rounding)
    dz = (2 * dim * F * (hid.abs() @ w.abs().T)).amax(1)
    lse = torch.logsumexp(z, 1)
    # exponentials good to 2^-20, sums of at most 256 + blocks + 16 terms
    dlse = dz + 2.0 ** -20 + (256 + v / 256 + len(weights) + 16) * F + 4 * F * lse.abs()
    at = targets.clamp(0, v - 1).long()[:, None]
    zt = z.gather(1, at)[:, 0]
    loss = torch.where(counts, lse - zt, torch.zeros_like(lse))
    dloss = torch.where(counts, dlse + dz + 2 * F * zt.abs(), torch.zeros_like(lse))
    tw = torch.ones(tokens, dtype=torch.float64, device="cuda") if token_weight is None else token_weight.double()
    tw = torch.where(counts, tw, torch.zeros_like(tw))
    prob = torch.exp(z - lse[:, None])
    gmat = prob.scatter_add(1, at, -torch.ones_like(tw)[:, None]) * tw[:, None]
    u = U[hidden.dtype]
    dprob = prob * (dz + dlse + 2.0 ** -20 + 8 * F * z.abs().amax(1))[:, None]
    dg = dprob * tw.abs()[:, None] + (u + 4 * F) * gmat.abs() + float(tw.abs().max() if tokens else 0) * 2.0 ** -37
    hid = torch.where(counts[:, None], hid, torch.zeros_like(hid))
    dh, mh = gmat @ w, gmat.abs() @ w.abs()
    ddh = dg @ w.abs() + 2 * v * F * mh
    dw, mw = gmat.T @ hid, gmat.abs().T @ hid.abs()
    ddw = dg.T @ hid.abs() + 2 * (tokens + 8) * F * mw
    tiny = TINY[hidden.dtype]
    return {"loss": (loss, dloss + 1e-300), "lse": (lse, dlse), "dhidden": (dh, ddh + u * (dh.abs() + ddh) + tiny),
            "dweights": (dw, ddw + u * (dw.abs() + ddw) + tiny)}


def check_xent(r, ref, grad):
    within(r.loss, *ref["loss"], "loss")
    within(r.lse, *ref["lse"], "lse")
    if grad:
        within(r.dhidden, *ref["dhidden"], "dhidden")
        within(torch.cat(r.dweights), *ref["dweights"], "dweights")


def xent_inputs(g, tokens, dim, vocab, dtype, index=torch.int64, std=2.0):
    whole = normal(g, vocab, dim, dtype=dtype, std=std / math.sqrt(dim))
    hidden = normal(g, tokens, dim, dtype=dtype)
    targets = torch.randint(0, vocab, (tokens,), generator=g, device="cuda").to(index)
    targets[torch.rand(tokens, generator=g, device="cuda") < 0.1] = -100
    return whole, hidden, targets


@gpu
@pytest.mark.parametrize("dtype", HALF)
@pytest.mark.parametrize("p,tokens,dim,vocab", [
    (1, 1, 8, 1), (1, 1, 8, 2), (2, 1, 64, 300), (3, 2, 72, 1000), (4, 127, 64, 255), (4, 129, 128, 1025), (8, 128, 256, 2048),
    (8, 300, 520, 5003), (16, 33, 8, 9), (5, 513, 200, 3001), (64, 20, 64, 64), (64, 5, 16, 3), (2, 1100, 136, 777),
    (3, 256, 1024, 4099), (1, 640, 64, 16384),
])
def test_vocab_xent(h, dtype, p, tokens, dim, vocab):
    g = gen(tokens * 7 + vocab)
    whole, hidden, targets = xent_inputs(g, tokens, dim, vocab, dtype)
    weights = pieces(whole, p)
    tw = torch.rand(tokens, generator=g, device="cuda") / tokens
    ref = xent_reference(hidden, weights, targets, tw)
    r = h.vocab_xent(hidden, weights, targets, token_weight=tw, grad=True)
    check_xent(r, ref, True)
    h.check()
    alone = h.vocab_xent(hidden, weights, targets)
    assert torch.equal(alone.loss, r.loss) and torch.equal(alone.lse, r.lse) and alone.dhidden is None
    again = h.vocab_xent(hidden, weights, targets.int(), token_weight=tw, grad=True)
    assert torch.equal(again.dhidden, r.dhidden) and all(torch.equal(x, y) for x, y in zip(again.dweights, r.dweights))


@gpu
@pytest.mark.parametrize("dtype", HALF)
def test_vocab_xent_strides_and_no_weights(h, dtype):
    g = gen(4)
    whole, hidden, targets = xent_inputs(g, 70, 96, 1000, dtype)
    weights = [strided(t, 24) for t in pieces(whole, 3)]
    hidden = strided(hidden, 8, 8)
    check_xent(h.vocab_xent(hidden, weights, targets, grad=True), xent_reference(hidden, weights, targets, None), True)


@gpu
@pytest.mark.parametrize("dtype", HALF)
def test_vocab_xent_left_out_tokens(h, dtype):
    """Tokens that are left out hold infinities and NaN; all of them left out."""
    g = gen(6)
    whole, hidden, targets = xent_inputs(g, 200, 64, 600, dtype)
    clean = hidden.clone()
    out = (targets < 0)
    assert bool(out.any())
    hidden[out] = float("nan")
    hidden[int(out.nonzero()[0]), 3] = float("inf")
    ref = xent_reference(clean, [whole], targets, None)
    r = h.vocab_xent(hidden, pieces(whole, 2), targets, grad=True)
    within(r.loss, *ref["loss"], "loss")
    assert bool((r.loss[out] == 0).all()) and bool((r.dhidden[out] == 0).all())
    within(r.dhidden, *ref["dhidden"], "dhidden")
    within(torch.cat(r.dweights), *ref["dweights"], "dweights")
    for none in (torch.full_like(targets, 600), torch.full_like(targets, -1)):
        r = h.vocab_xent(hidden, pieces(whole, 2), none, grad=True)
        assert bool((r.loss == 0).all()) and bool((r.dhidden == 0).all()) and bool((torch.cat(r.dweights) == 0).all())
    r = h.vocab_xent(clean, pieces(whole, 2), targets, token_weight=torch.zeros(200, device="cuda"), grad=True)
    assert bool((r.dhidden == 0).all()) and bool((torch.cat(r.dweights) == 0).all())


@gpu
@pytest.mark.parametrize("dtype", HALF)
def test_vocab_xent_bad_rows_stay_alone(h, dtype):
    """A token that counts and holds a NaN: NaN in its own loss and gradient
    row, and nowhere else in loss and dhidden."""
    g = gen(16)
    whole, hidden, targets = xent_inputs(g, 150, 64, 900, dtype)
    targets = targets.clamp(min=0)
    ref = xent_reference(hidden, [whole], targets, None)
    bad = hidden.clone()
    bad[77, 5] = float("nan")
    r = h.vocab_xent(bad, pieces(whole, 4), targets, grad=True)
    keep = torch.arange(150, device="cuda") != 77
    assert bool(r.loss[77].isnan()) and bool(r.lse[77].isnan()) and bool(r.dhidden[77].isnan().all())
    within(r.loss[keep], ref["loss"][0][keep], ref["loss"][1][keep], "loss")
    within(r.dhidden[keep], ref["dhidden"][0][keep], ref["dhidden"][1][keep], "dhidden")


@gpu
@pytest.mark.parametrize("dtype", HALF)
def test_vocab_xent_large_logits_and_weights(h, dtype):
    """Logits of a few hundred (nothing overflows), rows of the vocabulary far
    below the rest, token weights over twelve powers of ten."""
    g = gen(26)
    whole, hidden, targets = xent_inputs(g, 130, 128, 700, dtype, std=60.0)
    whole[100:300] *= 0.0
    tw = 10.0 ** (-12 * torch.rand(130, generator=g, device="cuda"))
    r = h.vocab_xent(hidden, pieces(whole, 3), targets, token_weight=tw, grad=True)
    check_xent(r, xent_reference(hidden, pieces(whole, 3), targets, tw), True)


@gpu
def test_vocab_xent_no_tokens(h):
    w = torch.randn(40, 16, device="cuda").bfloat16()
    e = torch.empty(0, 16, device="cuda", dtype=torch.bfloat16)
    r = h.vocab_xent(e, pieces(w, 3), torch.empty(0, dtype=torch.int64, device="cuda"), grad=True)
    assert r.loss.shape == (0,) and r.dhidden.shape == (0, 16) and bool((torch.cat(r.dweights) == 0).all())
    h.check()


@gpu
def test_vocab_xent_gradients_separately(h):
    """dhidden without dweights and the other way round, through the C call."""
    g = gen(31)
    whole, hidden, targets = xent_inputs(g, 90, 64, 500, torch.bfloat16)
    ref = h.vocab_xent(hidden, [whole], targets, grad=True)
    lib = rar.load_library()
    need = lib.rar_vocab_xent_workspace(90, 64, 500, 1, 1)
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    for which in ("dhidden", "dweights"):
        a = _ops.VocabXentArgs()
        wp = (ctypes.c_void_p * 1)(whole.data_ptr())
        a.hidden, a.weights, a.p, a.dtype = hidden.data_ptr(), ctypes.addressof(wp), 1, 2
        a.tokens, a.dim, a.vocab, a.targets, a.index_bytes = 90, 64, 500, targets.data_ptr(), 8
        a.workspace, a.workspace_bytes = ws.data_ptr(), need
        out = torch.empty_like(ref.dhidden if which == "dhidden" else whole)
        op = (ctypes.c_void_p * 1)(out.data_ptr())
        if which == "dhidden":
            a.dhidden = out.data_ptr()
        else:
            a.dweights = ctypes.addressof(op)
        assert lib.rar_vocab_xent(h.h, ctypes.byref(a), torch.cuda.current_stream().cuda_stream) == 0
        assert torch.equal(out, ref.dhidden if which == "dhidden" else ref.dweights[0])


@gpu
@pytest.mark.parametrize("dtype", HALF)
def test_vocab_xent_grad_against_differences(h, dtype):
    g = gen(41)
    tokens, dim, vocab = 24, 64, 333
    whole, hidden, targets = xent_inputs(g, tokens, dim, vocab, dtype)
    tw = torch.rand(tokens, generator=g, device="cuda")
    r = h.vocab_xent(hidden, pieces(whole, 3), targets, token_weight=tw, grad=True)
    ref = xent_reference(hidden, pieces(whole, 3), targets, tw)
    counts = targets >= 0

    def loss(hid, w):
        z = hid @ w.T
        nll = torch.logsumexp(z, 1) - z.gather(1, targets.clamp(min=0)[:, None])[:, 0]
        return float((nll * tw.double() * counts).sum())

    for _ in range(4):
        dh, dw = normal(g, tokens, dim).double(), normal(g, vocab, dim).double()
        step = 1e-5
        diff = (loss(hidden.double() + step * dh, whole.double() + step * dw) -
                loss(hidden.double() - step * dh, whole.double() - step * dw)) / (2 * step)
        own = float((r.dhidden.double() * dh).sum() + (torch.cat(r.dweights).double() * dw).sum())
        bound = float((ref["dhidden"][1] * dh.abs()).sum() + (ref["dweights"][1] * dw.abs()).sum())
        assert abs(own - diff) < bound + 1e-5


# ---------------------------------------------------------------- embedding

@gpu
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("index", [torch.int32, torch.int64])
@pytest.mark.parametrize("p,vocab,dim,tokens", [
    (1, 1, 1, 1), (2, 5, 3, 4), (8, 1000, 256, 3), (3, 10007, 1001, 513), (64, 64, 40, 200), (70, 50, 64, 99), (4, 4096, 4096, 33),
    (8, 300, 2048, 2000), (2, 77, 10000, 5),
])
def test_embedding(h, dtype, index, p, vocab, dim, tokens):
    g = gen(vocab + dim)
    whole = normal(g, vocab, dim, dtype=dtype)
    tok = torch.randint(-1, vocab + 1, (tokens,), generator=g, device="cuda").to(index)
    y = h.embedding(pieces(whole, p), tok, scale=1.7)
    counts = (tok >= 0) & (tok < vocab)
    ref = whole.double()[tok.clamp(0, vocab - 1).long()] * ctypes.c_float(1.7).value * counts[:, None]
    within(y, ref, (U[dtype] * (1 + F) + F) * ref.abs() + TINY[dtype], "lookup")
    assert bool((y[~counts] == 0).all())


@gpu
@pytest.mark.parametrize("extra,offset", [(0, 1), (3, 0), (8, 8)])
def test_embedding_strides_and_left_out_rows(h, extra, offset):
    g = gen(2)
    whole = normal(g, 50, 264, dtype=torch.bfloat16)
    whole[0] = float("nan")
    tables = [strided(t, extra, offset) for t in pieces(whole, 4)]
    tok = torch.tensor([-1, 3, 49, 50, 2 ** 40, -2 ** 50, 12, 3], device="cuda")
    y = h.embedding(tables, tok)
    for k, t in enumerate(tok.tolist()):
        assert torch.equal(y[k], whole[t] if 0 <= t < 50 else torch.zeros_like(whole[0]))
    assert h.embedding(tables, tok[:0]).shape == (0, 264)


def check_embedding_grad(got, dout, tok, old, vocab, scale):
    dtype, counts = dout.dtype, (tok >= 0) & (tok < vocab)
    rows, at = dout.double()[counts], tok[counts].long()
    total = torch.zeros(vocab, dout.shape[1], dtype=torch.float64, device="cuda")
    mag, n = torch.zeros_like(total), torch.zeros(vocab, dtype=torch.float64, device="cuda")
    total.index_add_(0, at, rows)
    mag.index_add_(0, at, rows.abs())
    n.index_add_(0, at, torch.ones_like(at, dtype=torch.float64))
    scale = ctypes.c_float(scale).value
    total, mag = total * scale, mag * abs(scale)
    if old is not None:
        total, mag = total + old.double(), mag + old.double().abs()
    err = (n[:, None] + 3) * F * mag
    within(got, total, err + U[dtype] * (total.abs() + err) + TINY[dtype], "table gradient")
    untouched = n == 0
    if old is not None:
        assert torch.equal(got[untouched].view(torch.uint8), old[untouched].view(torch.uint8))
    else:
        assert bool((got[untouched] == 0).all())


@gpu
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("accumulate", [False, True])
@pytest.mark.parametrize("p,vocab,dim,tokens,kind", [
    (1, 1, 1, 1, "any"), (2, 5, 3, 4, "any"), (3, 1000, 72, 513, "any"), (8, 300, 264, 5000, "any"), (4, 2000, 129, 3000, "one"),
    (64, 64, 40, 200, "any"), (70, 50, 64, 99, "any"), (8, 70000, 16, 2100, "few"), (2, 77, 3080, 66, "any"),
    (8, 5000, 64, 20000, "few"), (1, 300000, 8, 4097, "any"), (3, 100, 8, 70000, "any"), (2, 100, 24, 64, "none"),
])
def test_embedding_grad(h, dtype, accumulate, p, vocab, dim, tokens, kind):
    g = gen(vocab * 3 + tokens)
    tok = torch.randint(-1, vocab + 1, (tokens,), generator=g, device="cuda")
    if kind == "one":  # one token everywhere
        tok[:] = vocab // 2
    elif kind == "few":  # most places hold one of three
        few = torch.tensor([0, vocab // 3, vocab - 1], device="cuda")
        often = torch.rand(tokens, generator=g, device="cuda") < 0.8
        tok = torch.where(often, few[torch.randint(0, 3, (tokens,), generator=g, device="cuda")], tok)
    elif kind == "none":
        tok[:] = -1
    dout = normal(g, tokens, dim, dtype=dtype)
    dout[tok < 0] = float("nan")  # never read
    old = normal(g, vocab, dim, dtype=dtype)
    into = old.clone()
    out = h.embedding_grad(dout, tok, pieces(into, p), scale=0.75, accumulate=accumulate)
    assert out[0].data_ptr() == into.data_ptr()
    check_embedding_grad(into, dout, tok, old if accumulate else None, vocab, 0.75)
    again = old.clone()
    h.embedding_grad(dout, tok.int(), pieces(again, p), scale=0.75, accumulate=accumulate)
    assert torch.equal(into.view(torch.uint8), again.view(torch.uint8))
    h.check()


@gpu
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("extra,offset", [(0, 1), (3, 0), (8, 8)])
def test_embedding_grad_strides(h, dtype, extra, offset):
    g = gen(12)
    vocab, dim, tokens = 50, 264, 300
    dout = strided(normal(g, tokens, dim, dtype=dtype), extra, offset)
    tok = torch.randint(0, vocab, (tokens,), generator=g, device="cuda")
    for accumulate in (False, True):
        old = normal(g, vocab, dim, dtype=dtype)
        tables = [strided(t, extra, offset) for t in pieces(old, 4)]
        h.embedding_grad(dout, tok, tables, accumulate=accumulate)
        check_embedding_grad(torch.cat(tables), dout, tok, old if accumulate else None, vocab, 1.0)


@gpu
def test_embedding_grad_no_tokens(h):
    e, none = torch.empty(0, 24, device="cuda"), torch.empty(0, dtype=torch.int64, device="cuda")
    t = torch.ones(30, 24, device="cuda")
    h.embedding_grad(e, none, pieces(t, 4), accumulate=True)
    assert bool((t == 1).all())
    h.embedding_grad(e, none, pieces(t, 4))
    assert bool((t == 0).all())


@gpu
def test_embedding_grad_against_differences(h):
    g = gen(51)
    vocab, dim, tokens = 40, 16, 100
    whole, dout = normal(g, vocab, dim), normal(g, tokens, dim)
    tok = torch.randint(-1, vocab, (tokens,), generator=g, device="cuda")
    d = torch.empty_like(whole)
    h.embedding_grad(dout, tok, pieces(d, 3), scale=2.5)
    direction = normal(g, vocab, dim)

    def loss(step):  # linear in the table: the 64-bit difference is exact to rounding
        rows = (whole.double() + step * direction.double())[tok.clamp(min=0)] * (tok >= 0)[:, None] * 2.5
        return float((dout.double() * rows).sum())

    own = float((d.double() * direction.double()).sum())
    mag = float((d.double() * direction.double()).abs().sum())
    assert abs(own - (loss(1.0) - loss(-1.0)) / 2) < 32 * F * mag


# ------------------------------------------- streams, graphs, sizes, refusals

@gpu
def test_on_another_stream_and_in_a_graph(h):
    """The same bits on a side stream, and from replays of a captured graph
    with new inputs in the same places."""
    g = gen(61)
    dim, vocab, tokens, p = 256, 1000, 96, 4
    whole = normal(g, vocab, dim, dtype=torch.bfloat16, std=0.1)
    weights, parts = pieces(whole, p), [normal(g, tokens, dim, dtype=torch.bfloat16) for _ in range(p)]
    tok = torch.randint(0, vocab, (tokens,), generator=g, device="cuda")
    dtab = torch.zeros_like(whole)

    def step():
        x = h.embedding(weights, tok, scale=2.0)
        r = h.add_rmsnorm(parts, residual=x, quant_group=128, keep_out=True)
        y = h.vocab_xent(r.out, weights, tok, grad=True)
        dx, dweight = h.add_rmsnorm_grad(y.dhidden, r.sum, r.rstd)
        h.embedding_grad(dx, tok, pieces(dtab, p), scale=2.0)
        return [x, r.sum, r.out, r.out8.view(torch.uint8), r.scales, y.loss, y.dhidden, dx, dweight, dtab.clone()] + y.dweights

    first = step()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        other = step()
        graph = torch.cuda.CUDAGraph()
    side.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(first, other))
    x = h.embedding(weights, tok, scale=2.0, stream=side)
    side.synchronize()
    assert torch.equal(x, first[0])
    with torch.cuda.graph(graph, stream=side):
        held = step()
    for k in range(2):
        tok.copy_(torch.randint(0, vocab, (tokens,), generator=g, device="cuda"))
        parts[0].normal_(generator=g)
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in held]
        for a, b in zip(step(), got):
            assert torch.equal(a, b)


@gpu
def test_offsets_beyond_32_bits(h):
    """More than 2^31 elements behind a pointer."""
    vocab, dim = 70001, 32768
    table = torch.zeros(vocab, dim, dtype=torch.bfloat16, device="cuda")
    table[vocab - 1] = torch.arange(dim, device="cuda").bfloat16()
    tok = torch.tensor([vocab - 1, 0, vocab], device="cuda")
    y = h.embedding([table], tok, scale=1.0)
    assert torch.equal(y[0], table[vocab - 1]) and bool((y[1:] == 0).all())
    h.embedding_grad(y, tok, [table], accumulate=True)
    assert torch.equal(table[vocab - 1].float(), (y[0].float() * 2).bfloat16().float())
    table[vocab - 2:] = 1.0
    r = h.add_rmsnorm([table], eps=0.0 + 1e-12)
    assert bool((r.out[vocab - 2:].float() == 1).all()) and bool((r.sum[vocab - 1] == 1).all()) and float(r.rstd[vocab - 1]) == 1.0
    del r
    rstd = torch.ones(vocab, device="cuda")
    dx, dw = h.add_rmsnorm_grad(table, table, rstd)
    assert bool((dx[vocab - 1].float() == 0).all()) and bool((dw.float() == 2).all())


@gpu
def test_refusals(h):
    g = gen(71)
    x = normal(g, 4, 64)
    half = x.bfloat16()
    tok = torch.zeros(4, dtype=torch.int64, device="cuda")
    bad = [
        lambda: h.add_rmsnorm([]),
        lambda: h.add_rmsnorm([x, half]),
        lambda: h.add_rmsnorm([x, x[:3]]),
        lambda: h.add_rmsnorm([x], x[0, :63].clone()),
        lambda: h.add_rmsnorm([x.t()]),
        lambda: h.add_rmsnorm([x.double()]),
        lambda: h.add_rmsnorm_grad(x, x, torch.ones(3, device="cuda")),
        lambda: h.vocab_xent(half, [half, half[:2]], tok),
        lambda: h.vocab_xent(half, [half], tok[:2]),
        lambda: h.vocab_xent(half, [half], tok.float()),
        lambda: h.embedding([x], tok.cpu()),
        lambda: h.embedding([x, x[:1]], tok),
        lambda: h.embedding_grad(x, tok[:2], [x]),
    ]
    for k, call in enumerate(bad):
        with pytest.raises(ValueError):
            call()
            print("accepted", k)
    codes = [
        (1, lambda: h.add_rmsnorm([x], eps=-1.0)),
        (1, lambda: h.add_rmsnorm([x], quant_group=20)),
        (2, lambda: h.add_rmsnorm([x.int()])),
        (1, lambda: h.add_rmsnorm([torch.zeros(1, 32769, device="cuda")])),
        (2, lambda: h.vocab_xent(x, [x], tok)),
        (1, lambda: h.vocab_xent(half[:, :60], [half[:, :60]], tok)),
        (1, lambda: h.vocab_xent(strided(half, 1), [half], tok)),
        (1, lambda: h.vocab_xent(half, pieces(torch.zeros(65, 64, dtype=torch.bfloat16, device="cuda"), 65), tok)),
        (1, lambda: h.embedding_grad(x, tok, [x])),  # overlap
        (2, lambda: h.embedding([x.int()], tok)),
    ]
    for code, call in codes:
        with pytest.raises(rar.RarError) as e:
            call()
        assert e.value.code == code and rar.rar_last_error(h.h)
    lib, stream = rar.load_library(), torch.cuda.current_stream().cuda_stream
    assert lib.rar_add_rmsnorm(h.h, None, stream) == 1

    def norm_args(**kw):
        a = _ops.RmsNormArgs()
        a._keep = (ctypes.c_void_p * 1)(x.data_ptr())
        a.parts, a.p, a.dtype, a.rows, a.dim, a.eps = ctypes.addressof(a._keep), 1, 1, 4, 64, 1e-6
        a.out = kw.pop("out", torch.empty_like(x).data_ptr())
        for k, v in kw.items():
            setattr(a, k, v)
        return a

    host = torch.zeros(4, 64)
    for kw in (dict(p=0), dict(p=1025), dict(dtype=7), dict(dim=0), dict(part_stride=63), dict(parts=None),
               dict(out8=x.data_ptr() + 4096), dict(out=x.data_ptr() + 4), dict(out=x.data_ptr() + 2),
               dict(residual=host.data_ptr()), dict(rows=1 << 62), dict(eps=float("nan"))):
        assert lib.rar_add_rmsnorm(h.h, ctypes.byref(norm_args(**kw)), stream) == 1, kw
    assert lib.rar_add_rmsnorm(h.h, ctypes.byref(norm_args(rows=0, parts=None)), stream) == 0
    # a workspace that is too small or off its alignment
    need = lib.rar_vocab_xent_workspace(4, 64, 4, 1, 1)
    ws = torch.empty(need + 256, dtype=torch.uint8, device="cuda")
    weights = half.clone()
    for ptr, size in ((ws.data_ptr(), need - 1), (ws.data_ptr() + 16, need), (None, need)):
        a = _ops.VocabXentArgs()
        wp = (ctypes.c_void_p * 1)(weights.data_ptr())
        dh = torch.empty_like(half)
        a.hidden, a.weights, a.p, a.dtype, a.tokens, a.dim, a.vocab = half.data_ptr(), ctypes.addressof(wp), 1, 2, 4, 64, 4
        a.targets, a.index_bytes, a.dhidden, a.workspace, a.workspace_bytes = tok.data_ptr(), 8, dh.data_ptr(), ptr, size
        assert lib.rar_vocab_xent(h.h, ctypes.byref(a), stream) == 1
    torch.cuda.synchronize()
    # interleaved columns of one matrix do not overlap
    both = torch.randn(6, 128, device="cuda")
    a = norm_args(rows=6, out=both.data_ptr() + 256, out_stride=128, part_stride=128)
    a._keep[0] = both.data_ptr()
    expect = h.add_rmsnorm([both[:, :64].clone()])
    assert lib.rar_add_rmsnorm(h.h, ctypes.byref(a), stream) == 0
    assert torch.equal(both[:, 64:], expect.out)


@gpu
@pytest.mark.parametrize("dtype", HALF)
def test_vocab_xent_equal_weights_round_once(h, dtype):
    """Tokens that weigh the same, a weight halfway between two values of the type: a target's
    row of dweights is off by its own rounding alone.  With p the softmax (logits of a
    spread of 0.04, so p is below 1.5 / 16384), p - 1 is rounded by p at most, and the
    four other tokens' entries of that row, p each, by u p."""
    g = gen(77)
    vocab, dim, tokens = 16384, 64, 5
    u = U[dtype]
    weights = normal(g, vocab, dim, dtype=dtype, std=0.005)
    hidden = normal(g, tokens, dim, dtype=dtype)
    targets = torch.tensor([3, 777, 5000, 9001, 16000], device="cuda")
    w = torch.full((tokens,), 1.0 + u, device="cuda")
    r = h.vocab_xent(hidden, pieces(weights, 3), targets, token_weight=w, grad=True)
    logits = hidden.double() @ weights.double().t()
    gm = torch.softmax(logits, 1)
    gm[torch.arange(tokens), targets] -= 1.0
    ref = ((gm * w.double()[:, None]).t() @ hidden.double())[targets]
    size = hidden.double().abs()
    assert float(torch.softmax(logits, 1).max()) < 1.5 / vocab
    tol = u * ref.abs() + 1.5 / vocab * (1 + u) * (size + 4 * u * size.max()) * (1 + u) + TINY[dtype]
    within(torch.cat(r.dweights)[targets], ref, tol, "dweights")

"""The norm of many tensors (rar_grad_norm) and clipping to it (rar_grad_clip)
against plain forms in 64 bits.

A sum of squares in 32 bits: a thread adds at most 16 of a chunk's in a row, then there are 2 + 5 + 8
partial sums, and the chunks' are added in 64 bits.  All are positive, so the sum is off by at
most 32 F of itself (F = 2^-24; the squares' own rounding counted) and the norm by half of that, and by its own rounding.
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
from tests.test_model_ops import DTYPES, F, gen, h, normal, strided  # noqa: F401

gpu = pytest.mark.gpu
TOL = 17 * F


def test_struct_layouts_match_c():
    structs = {"rar_tensor": _ops.Tensor, "rar_grad_norm_args": _ops.GradNormArgs, "rar_grad_clip_args": _ops.GradClipArgs}
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
    for name in ("rar_grad_norm", "rar_grad_clip"):
        assert getattr(lib, name)(None, None, None) == 1  # RAR_EINVAL
    assert lib.rar_grad_norm_workspace(None, 0) > 0  # (the norm of nothing is 0)
    assert lib.rar_grad_norm_workspace(None, 3) == 0
    t = (_ops.Tensor * 2)(_ops.Tensor(None, 1, 1 << 30, 1 << 30, 0), _ops.Tensor(None, 1, 3, 5, 0))
    assert lib.rar_grad_norm_workspace(t, 2) == 0
    t[0].rows = 1 << 10
    assert lib.rar_grad_norm_workspace(t, 2) == 0  # more than 2^40 elements in all
    t[0].cols = 1 << 20
    assert 0 < lib.rar_grad_norm_workspace(t, 2) < 1 << 20
    for call in (lambda: rar.rar_grad_norm(None, [torch.zeros(4)]), lambda: rar.rar_grad_clip(None, [torch.zeros(4)], 1.0),
                 lambda: rar.rar_grad_norm(None, []), lambda: rar.rar_grad_norm(None, torch.zeros(4))):
        with pytest.raises(ValueError):
            call()


def norms_of(tensors):
    return torch.stack([torch.linalg.vector_norm(t.double().reshape(-1)) for t in tensors])


def check_norm(h, tensors):  # noqa: F811
    r, want = h.grad_norm(tensors), norms_of(tensors)
    total = torch.linalg.vector_norm(want)
    assert r.norm.shape == () and r.norms.shape == (len(tensors),) and r.norm.dtype == r.norms.dtype == torch.float32
    assert bool(((r.norms.double() - want).abs() <= TOL * want).all())
    assert abs(float(r.norm.double() - total)) <= TOL * float(total)
    again = h.grad_norm(tensors)
    assert torch.equal(again.norm, r.norm) and torch.equal(again.norms, r.norms)
    return r


def some_tensors(g, sizes, dtypes):
    return [normal(g, math.prod(s), dtype=dtypes[i % len(dtypes)], std=2.0 ** (i % 7 - 3)).view(s) for i, s in enumerate(sizes)]


ODD = [(1,), (2,), (7, 3), (1001,), (33, 65), (4096,), (4097,), (5, 7, 11), (8192, 3), (), (1, 1), (130, 129), (0,), (3, 0, 2), (12289,)]


@gpu
@pytest.mark.parametrize("dtypes", [[d] for d in DTYPES] + [DTYPES])
@pytest.mark.parametrize("sizes", [[(1,)], ODD, ODD * 5, [(3,)] * 512, [(5, 3)] * 1300, [(300001,), (77,)], [(0,)]])
def test_norms(h, dtypes, sizes):  # noqa: F811
    check_norm(h, some_tensors(gen(len(sizes)), sizes, dtypes))
    h.check()


@gpu
@pytest.mark.parametrize("dtype", DTYPES)
def test_tensors_that_begin_anywhere(h, dtype):  # noqa: F811
    g = gen(2)
    flat = normal(g, 40000, dtype=dtype)
    for lead in range(9):
        for n in (1, 3, 8, 15, 16, 17, 255, 9001):
            check_norm(h, [flat[lead:lead + n]])


@gpu
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows,cols,gap", [(3, 5, 1), (70, 64, 8), (129, 1001, 7), (9000, 2, 3), (1, 50, 6), (50, 1, 4), (70, 63, 2), (3, 20000, 24)])
def test_matrices_with_gaps_and_other_orders(h, dtype, rows, cols, gap):  # noqa: F811
    g = gen(rows + cols)
    t = normal(g, rows, cols, dtype=dtype)
    check_norm(h, [strided(t, gap, 1), t.t(), t, strided(t, gap)])
    cube = normal(g, 6, 5, 7, dtype=dtype)
    check_norm(h, [cube.permute(2, 0, 1), cube.transpose(0, 1)])


@gpu
@pytest.mark.parametrize("dtype", DTYPES)
def test_values_at_the_ends_of_the_type(h, dtype):  # noqa: F811
    """Squares that overflow 32 bits, or vanish in them; chunks of both kinds in one tensor."""
    info = torch.finfo(dtype)
    g = gen(5)
    for size in (info.max, info.max / 64, info.tiny, info.smallest_normal / 4, 2.0 ** -60, 2.0 ** 62 if dtype != torch.float16 else 2.0 ** 14):
        x = (torch.rand(9000, generator=g, device="cuda", dtype=torch.float64) * 0.5 + 0.5).mul_(size).to(dtype)
        want = torch.linalg.vector_norm(x.double())
        if want < torch.finfo(torch.float32).max:
            r = h.grad_norm([x, x[:0]])
            # (a norm below the normal numbers is rounded to their step)
            assert abs(float(r.norms[0].double() - want)) <= TOL * float(want) + 2.0 ** -150
        else:
            assert bool(h.grad_norm([x]).norm.isinf())
    x = torch.zeros(20000, dtype=dtype, device="cuda")
    x[5], x[15000] = info.max / 2, info.tiny
    assert abs(float(h.grad_norm([x]).norm.double()) / (info.max / 2) - 1) <= TOL + torch.finfo(dtype).eps
    assert float(h.grad_norm([torch.zeros(5000, dtype=dtype, device="cuda")]).norm) == 0.0
    assert float(h.grad_norm([torch.full((5000,), -0.0, dtype=dtype, device="cuda")]).norm) == 0.0


@gpu
@pytest.mark.parametrize("dtype", DTYPES)
def test_infinities_and_nan(h, dtype):  # noqa: F811
    a, b = torch.ones(9000, dtype=dtype, device="cuda"), torch.ones(3, 5, dtype=dtype, device="cuda")
    a[8999] = -float("inf")
    r = h.grad_norm([a, b])
    assert bool(r.norm.isinf()) and bool(r.norms[0].isinf()) and abs(float(r.norms[1]) - 15 ** 0.5) <= 4 * TOL
    b[2, 4] = float("nan")
    r = h.grad_norm([a, b])
    assert bool(r.norm.isnan()) and bool(r.norms[0].isinf()) and bool(r.norms[1].isnan())
    # clipping does what its formula says
    norm = h.grad_clip([a], 1.0)
    assert bool(norm.isinf()) and bool((a[:-1] == 0).all()) and bool(a[-1].isnan())
    c = torch.ones(10, dtype=dtype, device="cuda")
    h.grad_clip([c], 1.0, norm=torch.tensor(float("nan"), device="cuda"))
    assert bool(c.isnan().all())


def factor(norm, max_norm, eps):
    d = norm + eps
    # (a tensor over a tensor: a number over a tensor is a product with the reciprocal)
    return torch.where(d <= max_norm, torch.ones_like(d), torch.full_like(d, max_norm) / d)


@gpu
@pytest.mark.parametrize("dtypes", [[d] for d in DTYPES] + [DTYPES])
@pytest.mark.parametrize("sizes", [[(1,)], ODD, [(5, 3)] * 700, [(300001,), (77, 3)]])
@pytest.mark.parametrize("max_norm", [0.0, 0.37, 1e9])
def test_clipping(h, dtypes, sizes, max_norm):  # noqa: F811
    """In place, into tensors of the same types, and into 32 bits, each value rounded once."""
    g = gen(len(sizes) + 1)
    tensors = some_tensors(g, sizes, dtypes)
    norm = h.grad_norm(tensors).norm
    f = factor(norm, max_norm, 1e-6)
    want = [t.float() * f for t in tensors]
    for wide in (False, True):
        out = [torch.full_like(t, 9.0, dtype=torch.float32 if wide else t.dtype) for t in tensors]
        kept = [t.clone() for t in tensors]
        assert torch.equal(h.grad_clip(tensors, max_norm, out=out), norm)
        assert all(torch.equal(o, w.to(o.dtype)) for o, w in zip(out, want))
        assert all(torch.equal(t, k) for t, k in zip(tensors, kept))
    assert torch.equal(h.grad_clip(tensors, max_norm, norm=norm), norm)
    assert all(torch.equal(t, w.to(t.dtype)) for t, w in zip(tensors, want))
    h.check()


@gpu
@pytest.mark.parametrize("dtype", DTYPES)
def test_clipping_at_any_alignment(h, dtype):  # noqa: F811
    g = gen(8)
    flat = normal(g, 20000, dtype=dtype)
    for n in (1, 7, 33, 9001):
        for lead in (0, 1, 5):
            for to in (0, 1, 2, 3, 4, 6):
                for kind in {dtype, torch.float32}:
                    room = torch.full((n + 16,), 5.0, dtype=kind, device="cuda")
                    x, y = flat[lead:lead + n], room[to:to + n]
                    norm = h.grad_clip([x], 0.5, out=[y])
                    assert torch.equal(y, (x.float() * factor(norm, 0.5, 1e-6)).to(kind))
                    assert bool((room[:to] == 5).all()) and bool((room[to + n:] == 5).all())


@gpu
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows,cols,gap", [(3, 5, 1), (129, 1001, 7), (9000, 2, 3), (70, 64, 8), (70, 63, 2), (3, 20000, 24)])
def test_clipping_matrices_with_gaps(h, dtype, rows, cols, gap):  # noqa: F811
    g = gen(rows)
    t = normal(g, rows, cols, dtype=dtype)
    views = [(strided(t, gap, 1), torch.empty_like(t)), (t, strided(torch.zeros_like(t), gap)), (strided(t, gap), strided(torch.zeros_like(t), gap + 2)),
             (t.t(), torch.empty_like(t).t())]
    norm = h.grad_clip([a for a, _ in views], 0.1, out=[b for _, b in views])
    for a, b in views:
        assert torch.equal(b, (a.float() * factor(norm, 0.1, 1e-6)).to(dtype))
    one = strided(t, gap)
    whole = one.as_strided((rows * (cols + gap) - gap,), (1,))
    before = whole.clone()
    norm = h.grad_clip([one], 0.1)
    assert torch.equal(one, (t.float() * factor(norm, 0.1, 1e-6)).to(dtype))
    before.as_strided(one.shape, one.stride()).copy_(one)
    assert torch.equal(whole.isnan(), before.isnan()) and torch.equal(whole.nan_to_num(), before.nan_to_num())
    # two ranges of columns of one matrix, scaled where they lie
    both = torch.cat([t, t], 1).contiguous()
    norm = h.grad_clip([both[:, :cols], both[:, cols:]], 0.1)
    assert torch.equal(both, (torch.cat([t, t], 1).float() * factor(norm, 0.1, 1e-6)).to(dtype))


@gpu
def test_a_tensor_given_twice(h):  # noqa: F811
    x = torch.full((100,), 2.0, device="cuda")
    assert abs(float(h.grad_norm([x, x]).norm) - 800 ** 0.5) <= TOL * 30
    for call in (lambda: h.grad_clip([x, x], 1.0), lambda: h.grad_clip([x[:60], x[40:]], 1.0),
                 lambda: h.grad_clip([x[:50], x[50:]], 1.0, out=[x[50:], x[:50]]), lambda: h.grad_clip([x[:60]], 1.0, out=[x[1:61]]),
                 lambda: h.grad_clip([x], 1.0, norm=x[:1]), lambda: h.grad_clip([x[:9].bfloat16(), x], 1.0, out=[x[:9], x])):
        with pytest.raises(rar.RarError, match="overlap"):
            call()
    assert bool((x == 2).all())
    h.grad_clip([x], 1.0, out=[x])  # the tensor itself
    assert bool((x - 0.1 < 1e-5).all())


@gpu
def test_more_than_32_bits_of_elements(h):  # noqa: F811
    n = (1 << 31) + 4097
    x = torch.zeros(n, dtype=torch.bfloat16, device="cuda")
    x[n - 1], x[1 << 31], x[0] = 2.0, 4.0, 4.0
    assert float(h.grad_norm([x]).norm) == 6.0
    h.grad_clip([x], 3.0, eps=0.0)
    assert x[n - 1] == 1 and x[1 << 31] == 2 and x[0] == 2 and float(x.sum(dtype=torch.float32)) == 5.0


@gpu
def test_on_another_stream_and_in_graphs(h):  # noqa: F811
    g = gen(3)
    a = some_tensors(g, ODD, DTYPES)
    b = some_tensors(g, [(70000,), (5, 3)] * 300, [torch.float32])
    for t in (a, b):
        want = h.grad_norm(t)
        torch.cuda.synchronize()
        side = torch.cuda.Stream()
        r = h.grad_norm(t, stream=side)
        side.synchronize()
        assert torch.equal(r.norm, want.norm) and torch.equal(r.norms, want.norms)
    outs = [[torch.empty_like(t) for t in x] for x in (a, b)]
    graphs = []
    for x, out in zip((a, b), outs):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            norm = h.grad_clip(x, 0.25, out=out)
        graphs.append((graph, norm))
    for k in range(4):
        x, out, (graph, norm) = (a, b)[k % 2], outs[k % 2], graphs[k % 2]
        x[0].normal_(generator=g)
        graph.replay()
        torch.cuda.synchronize()
        want = h.grad_norm(x).norm
        assert torch.equal(norm, want)
        assert all(torch.equal(o, (t.float() * factor(want, 0.25, 1e-6)).to(o.dtype)) for t, o in zip(x, out))


@gpu
def test_refusals(h):  # noqa: F811
    x = torch.ones(6, 8, device="cuda")
    for call in (lambda: h.grad_norm([x.double()]), lambda: h.grad_norm([x, torch.ones(3)]), lambda: h.grad_norm([]), lambda: h.grad_norm([x, 3]),
                 lambda: h.grad_norm([x[:, ::2]]), lambda: h.grad_norm([x.expand(3, 6, 8)]), lambda: h.grad_norm([x[:1].expand(6, 8)]),
                 lambda: h.grad_norm([x.as_strided((5, 8), (4, 1))]), lambda: h.grad_norm([torch.ones(3, 4, 5, device="cuda")[:, :2]]),
                 lambda: h.grad_clip([x], -1.0), lambda: h.grad_clip([x], float("nan")), lambda: h.grad_clip([x], float("inf")),
                 lambda: h.grad_clip([x], 1.0, eps=-1.0), lambda: h.grad_clip([x], 1.0, out=[]), lambda: h.grad_clip([x, x], 1.0, out=[x]),
                 lambda: h.grad_clip([x], 1.0, out=[torch.ones(48, device="cuda")]), lambda: h.grad_clip([x.t()], 1.0, out=[torch.ones(8, 6, device="cuda")]),
                 lambda: h.grad_clip([x], 1.0, norm=torch.ones(2, device="cuda")), lambda: h.grad_clip([x], 1.0, norm=torch.ones(1))):
        with pytest.raises(ValueError):
            call()
    for code, call in ((2, lambda: h.grad_norm([x.int()])), (1, lambda: h.grad_clip([x], 1.0, out=[torch.empty(6, 8, dtype=torch.bfloat16, device="cuda")])),
                       (1, lambda: h.grad_clip([x.half()], 1.0, out=[x.bfloat16()]))):
        with pytest.raises(rar.RarError) as e:
            call()
        assert e.value.code == code
    # through the C calls
    lib, stream = rar.load_library(), torch.cuda.current_stream().cuda_stream
    norm = torch.empty(8, device="cuda")

    def call(given, **kw):
        t = (_ops.Tensor * max(1, len(given)))(*given)
        a = _ops.GradNormArgs()
        a.tensors, a.n, a.norm = ctypes.addressof(t), len(given), norm.data_ptr()
        need = lib.rar_grad_norm_workspace(t, len(given))
        ws = torch.empty(need + 256, dtype=torch.uint8, device="cuda")
        a.workspace, a.workspace_bytes = ws.data_ptr(), need
        for k, v in kw.items():
            setattr(a, k, v)
        return lib.rar_grad_norm(h.h, ctypes.byref(a), stream)

    good = (x.data_ptr(), 1, 6, 8, 0)
    for given, kw in (([_ops.Tensor(None, 1, 6, 8, 0)], {}), ([_ops.Tensor(x.data_ptr() + 2, 1, 6, 8, 0)], {}), ([_ops.Tensor(x.data_ptr(), 1, 6, 8, 7)], {}),
                        ([_ops.Tensor(x.data_ptr(), 9, 6, 8, 0)], {}), ([_ops.Tensor(x.data_ptr(), 1, 1 << 30, 1 << 30, 0)], {}),
                        ([_ops.Tensor(*good)], dict(norm=None)), ([_ops.Tensor(*good)], dict(norm=x.data_ptr())), ([_ops.Tensor(*good)], dict(norms=norm.data_ptr())),
                        ([_ops.Tensor(*good)], dict(workspace=None)), ([_ops.Tensor(*good)], dict(workspace_bytes=8)), ([_ops.Tensor(*good)], dict(tensors=None))):
        assert call(given, **kw) == 1, kw
    assert call([]) == 0 and float(norm[0]) == 0.0
    assert call([_ops.Tensor(*good), _ops.Tensor(None, 1, 0, 8, 0)]) == 0 and abs(float(norm[0]) - 48 ** 0.5) < 1e-5
    c = _ops.GradClipArgs()
    t = (_ops.Tensor * 1)(_ops.Tensor(*good))
    c.tensors, c.n, c.max_norm = ctypes.addressof(t), 1, 1.0
    assert lib.rar_grad_clip(h.h, ctypes.byref(c), stream) == 1  # no norm
    h.check()

"""What the model operators' calls refuse and what their host code decides
before a launch: matrices that torch holds in ways of its own, sizes far out of
range, calls from several threads, waits that run out."""
import contextlib
import ctypes
import threading
import types

import pytest
import torch

import ring_all_reduce_rar_gb300 as rar
from ring_all_reduce_rar_gb300 import _ops
from tests.test_model_ops import DTYPES, gen, h, normal, pieces  # noqa: F401  (h is the fixture)

MUTE = dict(timeout_ns=50_000_000, fault_mode="mute")

gpu = pytest.mark.gpu


# Every matrix of every call, by name; half types because all calls take them.
EXPANDED = ["part", "residual", "dout", "sum", "dsum", "hidden", "weight piece", "table piece", "lookup gradient", "gradient piece"]


@gpu
@pytest.mark.parametrize("shape", [(4, 64), (2, 8), (4, 1)])
@pytest.mark.parametrize("place", EXPANDED)
def test_expanded_matrices_are_refused(h, place, shape):  # noqa: F811
    """One row repeated by expand() lies in memory once: its row stride of 0
    must not pass for packed rows."""
    rows, dim = shape
    x = torch.ones(rows, dim, dtype=torch.bfloat16, device="cuda")
    e = torch.ones(1, dim, dtype=torch.bfloat16, device="cuda").expand(rows, dim)
    assert e.stride(0) == 0
    tok = torch.zeros(rows, dtype=torch.int64, device="cuda")
    rstd = torch.ones(rows, device="cuda")
    calls = {
        "part": lambda: h.add_rmsnorm([x, e]),
        "residual": lambda: h.add_rmsnorm([x], residual=e),
        "dout": lambda: h.add_rmsnorm_grad(e, x, rstd),
        "sum": lambda: h.add_rmsnorm_grad(x, e, rstd),
        "dsum": lambda: h.add_rmsnorm_grad(x, x, rstd, dsum=e),
        "hidden": lambda: h.vocab_xent(e, [x], tok),
        "weight piece": lambda: h.vocab_xent(x, [x, e], tok),
        "table piece": lambda: h.embedding([e, x], tok),
        "lookup gradient": lambda: h.embedding_grad(e, tok, [x.clone()]),
        "gradient piece": lambda: h.embedding_grad(x, tok, [e]),
    }
    with pytest.raises(ValueError, match="expanded"):
        calls[place]()


@gpu
def test_overlapping_rows_are_refused(h):  # noqa: F811
    memory = torch.ones(1024, dtype=torch.bfloat16, device="cuda")
    windows = memory.as_strided((8, 64), (16, 1))
    with pytest.raises(ValueError, match="overlap"):
        h.add_rmsnorm([windows])


@gpu
def test_one_expanded_row_is_a_row(h):  # noqa: F811
    """A single row has no distance to a next one, whatever its stride says."""
    x = normal(gen(3), 1, 64)
    one = x.as_strided((1, 64), (0, 1))
    assert torch.equal(h.add_rmsnorm([one]).out, h.add_rmsnorm([x]).out)


@gpu
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows,dim", [(3, 2048), (5, 200), (4, 33), (700, 1024), (2, 32768)])
@pytest.mark.parametrize("group", [32768, 1 << 32, (1 << 32) + 32, 1 << 62, (1 << 64) - 32])
def test_groups_longer_than_the_row(h, dtype, rows, dim, group):  # noqa: F811
    """A run of columns that covers the row is the row, also where its length
    passes 32 bits."""
    parts = [normal(gen(dim), rows, dim, dtype=dtype) for _ in range(2)]
    ref = h.add_rmsnorm(parts, quant_group=0)
    if group < 1 << 63:
        r = h.add_rmsnorm(parts, quant_group=group)
        assert r.scales.shape == (rows, 1)
        assert torch.equal(r.scales, ref.scales) and torch.equal(r.out8.view(torch.uint8), ref.out8.view(torch.uint8))
    codes, scales = torch.empty(rows, dim, dtype=torch.uint8, device="cuda"), torch.empty(rows, 1, device="cuda")
    a = _ops.RmsNormArgs()
    ptrs = (ctypes.c_void_p * 2)(*[t.data_ptr() for t in parts])
    a.parts, a.p, a.rows, a.dim, a.eps, a.group = ctypes.addressof(ptrs), 2, rows, dim, 1e-6, group
    a.dtype = {torch.float32: 1, torch.bfloat16: 2, torch.float16: 3}[dtype]
    a.out8, a.scales = codes.data_ptr(), scales.data_ptr()
    assert rar.load_library().rar_add_rmsnorm(h.h, ctypes.byref(a), torch.cuda.current_stream().cuda_stream) == 0
    assert torch.equal(scales, ref.scales) and torch.equal(codes, ref.out8.view(torch.uint8))


@gpu
@pytest.mark.parametrize("op,dims", [("norm", (8, 2)), ("norm any", (30011, 17011)), ("gradient any", (30011, 17011))])
def test_two_threads_share_no_launch_state(h, op, dims):  # noqa: F811
    """Two threads, a handle and a stream each, whose calls run one kernel with
    different amounts of shared memory (8 and 2 parts; rows of different lengths)."""
    lib, calls, errors = rar.load_library(), 1500, []
    start = threading.Barrier(2)

    def work(n):
        stream = torch.cuda.Stream()
        with torch.cuda.stream(stream), rar.Handle(0, skip_pointer_check=True) as mine:
            keep = []

            def matrix(rows, cols):
                keep.append(torch.ones(rows, cols, dtype=torch.bfloat16, device="cuda"))
                return keep[-1].data_ptr()
            if op == "norm":
                a = _ops.RmsNormArgs()
                a._parts = (ctypes.c_void_p * n)(*[matrix(640, 2048) for _ in range(n)])
                a.parts, a.p, a.rows, a.dim, a.out = ctypes.addressof(a._parts), n, 640, 2048, matrix(640, 2048)
            elif op == "norm any":
                a = _ops.RmsNormArgs()
                a._parts = (ctypes.c_void_p * 1)(matrix(2, n))
                a.parts, a.p, a.rows, a.dim, a.out = ctypes.addressof(a._parts), 1, 2, n, matrix(2, n)
            else:
                a = _ops.RmsNormGradArgs()
                rstd = torch.ones(2, device="cuda")
                a.rows, a.dim, a.dout, a.sum, a.rstd, a.dx = 2, n, matrix(2, n), matrix(2, n), rstd.data_ptr(), matrix(2, n)
            a.dtype = 2
            call = lib.rar_add_rmsnorm_grad if op == "gradient any" else lib.rar_add_rmsnorm
            start.wait()
            for _ in range(calls):
                if call(mine.h, ctypes.byref(a), stream.cuda_stream):
                    errors.append((n, rar.rar_last_error(mine.h)))
                    break
            stream.synchronize()

    threads = [threading.Thread(target=work, args=(n,)) for n in dims]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors


def check_time_out(call, ref, handle, words):
    """`call` on a handle with a muted rank reports RAR_ETIMEOUT once; the same
    call on it without the fault has the results `ref`."""
    call()
    assert handle.status() == 5  # RAR_ETIMEOUT
    assert words in rar.rar_last_error(handle.h)
    assert handle.status() == 0
    handle.set_options()
    for got, want in zip(call(), ref):
        assert torch.equal(got, want)
    handle.check()


@gpu
@pytest.mark.parametrize("mute", [0, 2])
@pytest.mark.parametrize("p,rows,dim", [(3, 640, 2048), (4, 5000, 4096)])
def test_residual_norm_muted_rank_times_out(h, p, rows, dim, mute):  # noqa: F811
    """A rank whose rows never arrive: the waits for them run out, no stage is
    handed back to the loads before its row has landed, and the kernel ends."""
    g = gen(p + mute)
    parts, res = [normal(g, rows, dim, dtype=torch.bfloat16) for _ in range(p)], normal(g, rows, dim, dtype=torch.bfloat16)
    for group in (None, 128, 0):
        def call(handle):
            r = handle.add_rmsnorm(parts, residual=res, quant_group=group, keep_out=True)
            return [r.sum, r.rstd, r.out] + ([] if group is None else [r.scales])
        with rar.Handle(0, fault_rank=mute, **MUTE) as faulty:
            check_time_out(lambda: call(faulty), call(h), faulty, "residual norm")


@gpu
@pytest.mark.parametrize("mute", [0, 1, 2])
def test_residual_norm_gradient_muted_matrix_times_out(h, mute):  # noqa: F811
    g = gen(mute)
    dout, s, dsum = (normal(g, 5000, 2048, dtype=torch.bfloat16) for _ in range(3))
    rstd = torch.ones(5000, device="cuda")
    with rar.Handle(0, fault_rank=mute, **MUTE) as faulty:
        check_time_out(lambda: faulty.add_rmsnorm_grad(dout, s, rstd, dsum=dsum), h.add_rmsnorm_grad(dout, s, rstd, dsum=dsum), faulty,
                       "residual norm")


@gpu
@pytest.mark.parametrize("mute", [0, 2])
@pytest.mark.parametrize("tokens,dim,vocab,grad", [(300, 256, 5000, True), (20, 64, 40, True), (600, 1288, 20000, False), (130, 1288, 9000, True)])
def test_cross_entropy_muted_piece_times_out(h, tokens, dim, vocab, grad, mute):  # noqa: F811
    """A piece whose tiles never arrive: loads, products and epilogues of both
    CTAs of a pair give up, the products under way are waited for, and the kernels end."""
    g = gen(tokens + mute)
    hidden, whole = normal(g, tokens, dim, dtype=torch.bfloat16), normal(g, vocab, dim, dtype=torch.bfloat16, std=0.1)
    targets = torch.randint(0, vocab, (tokens,), generator=g, device="cuda")

    def call(handle):
        r = handle.vocab_xent(hidden, pieces(whole, 3), targets, grad=grad)
        return [r.loss, r.lse] + ([r.dhidden, *r.dweights] if grad else [])
    with rar.Handle(0, fault_rank=mute, **MUTE) as faulty:
        check_time_out(lambda: call(faulty), call(h), faulty, "vocabulary cross entropy")


OPS = [("add_rmsnorm", lambda t, s: rar.rar_add_rmsnorm(7, [t], stream=s)),
       ("add_rmsnorm_grad", lambda t, s: rar.rar_add_rmsnorm_grad(7, t, t, t, stream=s)),
       ("vocab_xent", lambda t, s: rar.rar_vocab_xent(7, t, [t], t, stream=s)),
       ("embedding", lambda t, s: rar.rar_embedding(7, (t,), t, stream=s)),
       ("embedding_grad", lambda t, s: rar.rar_embedding_grad(7, t, t, [t], stream=s))]


@pytest.mark.parametrize("name,call", OPS)
def test_a_stream_belongs_to_the_tensors_device(monkeypatch, name, call):
    """The current device has no part in a stream that is given as an integer;
    a stream object of another device is refused.  (Stands in for two devices.)"""
    seen = []

    def operator(handle, *args):
        seen.append(("call", handle))
        return (None,) * {"add_rmsnorm": 5, "vocab_xent": 4}.get(name, 1)

    @contextlib.contextmanager
    def current(stream):
        seen.append((stream.cuda_stream, stream.device))
        yield
    # (a stream without a device is one of the current device, 0)
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda ptr, device=torch.device("cuda", 0):
                        types.SimpleNamespace(cuda_stream=ptr, device=device))
    monkeypatch.setattr(torch.cuda, "stream", current)
    monkeypatch.setattr(_ops, "_module", lambda: types.SimpleNamespace(**{name: operator}))
    on = types.SimpleNamespace(device=torch.device("cuda", 1))
    call(on, 1234)
    assert seen == [(1234, torch.device("cuda", 1)), ("call", 7)]
    seen.clear()
    other = types.SimpleNamespace(cuda_stream=5, device=torch.device("cuda", 0))
    with pytest.raises(ValueError, match="stream"):
        call(on, other)
    assert not seen
    call(on, None)
    assert seen == [("call", 7)]


@gpu
def test_a_stream_as_an_integer(h):  # noqa: F811
    g = gen(5)
    table, tok = normal(g, 50, 64), torch.tensor([3, 49, 50, 0], device="cuda")
    ref = h.embedding([table], tok)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    y = h.embedding([table], tok, stream=side.cuda_stream)
    side.synchronize()
    assert torch.equal(y, ref)
    y = h.embedding([table], tok, stream=0)  # the legacy default stream
    torch.cuda.synchronize()
    assert torch.equal(y, ref)


@gpu
@pytest.mark.parametrize("dim", [1 << 31, (1 << 33) + 8, 1 << 57])
def test_lookup_of_rows_beyond_32_bits_is_refused(h, dim):  # noqa: F811
    """Columns are counted in 32 bits.  (Refused before the pointers are looked at:
    the matrices here hold nothing of that length.)"""
    x, tok = torch.zeros(64, device="cuda"), torch.zeros(1, dtype=torch.int64, device="cuda")
    a = _ops.EmbeddingArgs()
    ptrs = (ctypes.c_void_p * 1)(x.data_ptr())
    a.tables, a.p, a.dtype, a.vocab, a.dim, a.tokens = ctypes.addressof(ptrs), 1, 1, 1, dim, tok.data_ptr()
    a.index_bytes, a.n_tokens, a.scale, a.out = 8, 1, 1.0, None
    assert rar.load_library().rar_embedding(h.h, ctypes.byref(a), torch.cuda.current_stream().cuda_stream) == 1
    assert "dim" in rar.rar_last_error(h.h)


@gpu
def test_cross_entropy_of_single_rows_with_any_stride(h):  # noqa: F811
    """One token and pieces of one row each: the strides, which nothing is
    read by, need not suit a tensor map."""
    g = gen(9)
    hidden, whole = normal(g, 1, 64, dtype=torch.bfloat16), normal(g, 3, 64, dtype=torch.bfloat16)
    tok = torch.tensor([2], device="cuda")
    ref = h.vocab_xent(hidden, pieces(whole, 3), tok)
    lib = rar.load_library()
    for stride in (65, 68, 1 << 45):
        loss, ws = torch.empty(1, device="cuda"), torch.empty(lib.rar_vocab_xent_workspace(1, 64, 3, 3, 0), dtype=torch.uint8, device="cuda")
        a = _ops.VocabXentArgs()
        ptrs = (ctypes.c_void_p * 3)(*[t.data_ptr() for t in pieces(whole, 3)])
        a.hidden, a.hidden_stride, a.weights, a.weight_stride = hidden.data_ptr(), stride, ctypes.addressof(ptrs), stride
        a.p, a.dtype, a.tokens, a.dim, a.vocab, a.targets, a.index_bytes = 3, 2, 1, 64, 3, tok.data_ptr(), 8
        a.loss, a.workspace, a.workspace_bytes = loss.data_ptr(), ws.data_ptr(), ws.numel()
        assert lib.rar_vocab_xent(h.h, ctypes.byref(a), torch.cuda.current_stream().cuda_stream) == 0, rar.rar_last_error(h.h)
        assert torch.equal(loss, ref.loss)


@gpu
def test_flags_without_a_truth_value(h):  # noqa: F811
    """An exception while a flag is read is that exception, before anything runs."""
    x, tok = torch.ones(4, 64, dtype=torch.bfloat16, device="cuda"), torch.zeros(4, dtype=torch.int64, device="cuda")
    neither = torch.ones(2)
    for call in (lambda: h.vocab_xent(x, [x], tok, grad=neither), lambda: h.add_rmsnorm([x], keep_out=neither),
                 lambda: h.embedding_grad(x, tok, [x.clone()], accumulate=neither)):
        with pytest.raises(RuntimeError, match="ambiguous"):
            call()


@gpu
def test_a_refused_size_leaves_the_last_call():
    """Too many rows are an argument error: nothing is enqueued, and status and
    send counts still belong to the call before.  (One more row than a launch has
    CTAs; the call is refused on the host.)"""
    with rar.Handle(0, engine="ring", skip_pointer_check=True) as mine:
        bufs = [torch.ones(4096, device="cuda") for _ in range(4)]
        mine.allreduce(bufs)
        counts = mine.send_counts(4)
        assert all(counts)
        a = _ops.RmsNormArgs()
        ptrs = (ctypes.c_void_p * 4)(*[t.data_ptr() for t in bufs])
        a.parts, a.p, a.dtype, a.rows, a.dim, a.eps = ctypes.addressof(ptrs), 4, 2, 1 << 31, 1, 1e-6
        assert rar.load_library().rar_add_rmsnorm(mine.h, ctypes.byref(a), torch.cuda.current_stream().cuda_stream) == 1
        assert "rows" in rar.rar_last_error(mine.h)
        assert mine.send_counts(4) == counts
        mine.check()

"""Host-side refusals and sizes of the clip and of the microscaled operands:
every error returns before any device call, so these run without a GPU."""
import ctypes
import gc
import weakref
from types import SimpleNamespace

import pytest

R = pytest.importorskip("rank_gradient_compression_amd")
B = R.binding

P = 4096  # a 16-byte aligned address that nothing dereferences
F32, BF16, F16 = B.PSGD_DTYPE_F32, B.PSGD_DTYPE_BF16, B.PSGD_DTYPE_F16
BIG = 1 << 31


def refused(fn, *args, status=B.PSGD_ERR_INVALID_ARG, match=None):
    with pytest.raises(B.PsgdError, match=match) as e:
        fn(*args)
    assert e.value.status == status
    assert fn.__name__ in str(e.value)


@pytest.mark.parametrize("rows,cols,codes,scales", [(0, 5, 0, 0), (5, 0, 0, 0), (1, 1, 16, 256), (32, 256, 32 * 128, 256),
                                                    (33, 257, 33 * 9 * 16, 2 * 2 * 256), (4, 11008, 4 * 344 * 16, 43 * 256)])
def test_sizes(rows, cols, codes, scales):
    assert B.psgd_mx_sizes(rows, cols) == (codes, scales)


def test_sizes_refused():
    refused(B.psgd_mx_sizes, -1, 4)
    refused(B.psgd_mx_sizes, 4, BIG)
    assert B.lib.psgd_mx_sizes(1, 1, None, None) == B.PSGD_ERR_INVALID_ARG
    for fn, more in ((B.psgd_mx_linear_workspace, (F32,)), (B.psgd_mx_train_workspace, ())):
        refused(fn, -1, 4, 4, *more)
        refused(fn, 4, 4, BIG, *more)
    refused(B.psgd_mx_linear_workspace, 4, 4, 4, 3, match="type")


def quant(x=P, dtype=F32, rows=4, cols=64, ld=64, rand=0, rc=1 << 20, rs=2 << 20, cc=0, cs=0, values=0, ldv=0):
    B.psgd_mx_quantize(x, dtype, rows, cols, ld, rand, rc, rs, cc, cs, values, ldv)


@pytest.mark.parametrize("kw,match", [
    (dict(dtype=3), "type"), (dict(dtype=-1), "type"), (dict(rows=-1), "negative"), (dict(cols=BIG), "INT32_MAX"),
    (dict(ld=63), "stride"), (dict(ld=BIG), "stride"), (dict(x=0), "NULL"), (dict(x=P + 2), "aligned"),
    (dict(rc=0), "together"), (dict(rs=0), "together"), (dict(cc=1 << 22), "together"),
    (dict(rc=0, rs=0), "no output"), (dict(rc=(1 << 20) + 8), "16-byte"), (dict(rs=(2 << 20) + 4), "16-byte"),
    (dict(rc=P, rs=2 << 20), "overlap"), (dict(rc=1 << 20, rs=1 << 20), "overlap"),
    (dict(values=P + 64, ldv=64), "overlaps x"), (dict(values=P, ldv=80), "overlaps x"),
    (dict(values=1 << 22, ldv=63), "stride"), (dict(values=(1 << 22) + 1, ldv=64), "aligned"),
    (dict(values=1 << 20, ldv=64), "overlap"), (dict(rand=1 << 20), "overlap"),
    (dict(cc=1 << 20, cs=4 << 20), "overlap"),
    (dict(rows=(1 << 31) - 1, cols=(1 << 31) - 1, ld=(1 << 31) - 1, x=1 << 62, rc=0, rs=0, values=1 << 62,
          ldv=(1 << 31) - 1), "too large"),
])
def test_quantize_refused(kw, match):
    with pytest.raises(B.PsgdError, match=match) as e:
        quant(**kw)
    assert e.value.status == B.PSGD_ERR_INVALID_ARG


def test_empty_matrices_are_accepted_without_a_device():
    quant(rows=0)
    quant(cols=0, ld=0)
    B.psgd_mx_dequantize(0, 0, 0, 7, 0, F32, 7)
    B.psgd_mx_product(0, 5, 7, 0, 0, P, P, 0, F32, 5, False)
    B.psgd_mx_linear(0, 5, 7, 0, F32, 7, P, P, 0, F32, 5, 0, 0)


def test_dequantize_refused():
    ok = [1 << 20, 2 << 20, 4, 64, P, F32, 64]
    for at, bad, match in [(0, 0, "NULL"), (1, 0, "NULL"), (0, (1 << 20) + 8, "16-byte"), (2, -1, "negative"),
                           (3, BIG, "INT32_MAX"), (4, 0, "NULL"), (4, P + 1, "aligned"), (5, 9, "type"),
                           (6, 63, "stride"), (4, 1 << 20, "overlaps"), (4, 2 << 20, "overlaps")]:
        args = list(ok)
        args[at] = bad
        refused(B.psgd_mx_dequantize, *args, match=match)


def test_product_refused():
    ok = [8, 8, 64, 1 << 20, 2 << 20, 3 << 20, 4 << 20, P, F32, 8, False]
    for at, bad, match in [(0, -1, "negative"), (1, BIG, "INT32_MAX"), (2, -3, "negative"), (3, 0, "NULL"),
                           (4, 0, "NULL"), (5, 0, "NULL"), (6, (4 << 20) + 1, "16-byte"), (7, 0, "NULL"),
                           (7, P + 2, "aligned"), (8, 5, "type"), (9, 7, "stride"), (7, 1 << 20, "overlaps"),
                           (7, 4 << 20, "overlaps")]:
        args = list(ok)
        args[at] = bad
        refused(B.psgd_mx_product, *args, match=match)


def test_linear_refused():
    m, n, k = 64, 96, 512  # too many activations for one launch: a workspace is needed
    need = B.psgd_mx_linear_workspace(m, n, k, BF16)
    assert need >= sum(B.psgd_mx_sizes(m, k))
    ok = [m, n, k, 1 << 24, BF16, k, 1 << 20, 2 << 20, 1 << 25, BF16, n, 1 << 26, need]
    for at, bad, match in [(3, 0, "NULL"), (4, 4, "type"), (5, k - 1, "stride"), (6, 0, "NULL"), (8, 0, "NULL"),
                           (9, 7, "type"), (10, n - 1, "stride"), (8, 1 << 24, "overlaps")]:
        args = list(ok)
        args[at] = bad
        refused(B.psgd_mx_linear, *args, match=match)
    for at, bad in [(11, 0), (11, (1 << 26) + 128), (12, need - 1)]:
        args = list(ok)
        args[at] = bad
        refused(B.psgd_mx_linear, *args, status=B.PSGD_ERR_WORKSPACE)


def train_args(m=40, n=96, k=70):
    need = B.psgd_mx_train_workspace(m, n, k)
    assert need >= sum(B.psgd_mx_sizes(m, k)) + sum(B.psgd_mx_sizes(n, k))
    assert need >= sum(B.psgd_mx_sizes(m, n)) + sum(B.psgd_mx_sizes(n, m))
    forward = [m, n, k, 1 << 24, BF16, k, 2 << 24, F32, k, 3 << 24, 4 << 24, 5 << 24, 6 << 24, 7 << 24, BF16, n,
               8 << 24, need]
    backward = [m, n, k, 1 << 24, BF16, n, 2 << 24, 3 << 24, 4 << 24, 5 << 24, 6 << 24, 7 << 24, BF16, k, 8 << 24, F32,
                k, False, 9 << 24, need]
    return forward, backward


def test_training_pass_refused():
    forward, backward = train_args()
    for at, bad, match in [(0, -1, "negative"), (2, BIG, "INT32_MAX"), (3, 0, "NULL"), (4, 3, "type"), (5, 69, "stride"),
                           (6, (2 << 24) + 2, "aligned"), (7, 4, "type"), (8, 69, "stride"), (9, 0, "NULL"),
                           (10, (4 << 24) + 1, "16-byte"), (11, 0, "NULL"), (13, 0, "NULL"), (15, 95, "stride"),
                           (13, 1 << 24, "overlaps"), (9, 2 << 24, "overlaps"), (11, 3 << 24, "overlaps"),
                           (16, 7 << 24, "overlaps")]:
        args = list(forward)
        args[at] = bad
        refused(B.psgd_mx_train_forward, *args, match=match)
    for at, bad, match in [(1, -1, "negative"), (0, BIG, "INT32_MAX"), (3, 0, "NULL"), (4, 3, "type"), (5, 95, "stride"),
                           (7, 0, "NULL"), (10, (6 << 24) + 4, "16-byte"), (11, (7 << 24) + 1, "aligned"),
                           (13, 69, "stride"), (15, -1, "type"), (16, 69, "stride"), (11, 8 << 24, "overlaps"),
                           (14, 1 << 24, "overlaps"), (14, 2 << 24, "overlaps"), (11, 3 << 24, "overlaps"),
                           (18, 8 << 24, "overlaps")]:
        args = list(backward)
        args[at] = bad
        refused(B.psgd_mx_train_backward, *args, match=match)
    for fn, ok, ws in ((B.psgd_mx_train_forward, forward, 16), (B.psgd_mx_train_backward, backward, 18)):
        for at, bad in [(ws, 0), (ws, (9 << 24) + 128), (ws + 1, ok[ws + 1] - 1)]:
            args = list(ok)
            args[at] = bad
            refused(fn, *args, status=B.PSGD_ERR_WORKSPACE)
    big = (1 << 31) - 1
    refused(B.psgd_mx_train_forward, big, big, 1, *forward[3:], match="too large")


def test_clip_create_refused():
    refused(B.psgd_clip_create, [-1], [F32], [F32])
    refused(B.psgd_clip_create, [1 << 50], [F32], [F32])
    refused(B.psgd_clip_create, [1 << 46, 1 << 46], [F32] * 2, [F32] * 2)
    refused(B.psgd_clip_create, [1 << 45], [F32], [F32])
    refused(B.psgd_clip_create, [4], [3], [F32])
    refused(B.psgd_clip_create, [4], [F32], [-1])
    out = ctypes.c_void_p(7)
    assert B.lib.psgd_clip_create(-1, None, None, None, ctypes.byref(out)) == B.PSGD_ERR_INVALID_ARG
    assert out.value is None
    assert B.lib.psgd_clip_create(1, None, None, None, ctypes.byref(out)) == B.PSGD_ERR_INVALID_ARG
    assert B.lib.psgd_clip_create(0, None, None, None, None) == B.PSGD_ERR_INVALID_ARG
    with pytest.raises(ValueError):
        B.psgd_clip_create([1, 2], [F32], [F32, F32])


def test_clip_calls_refused():
    c = B.psgd_clip_create([100, 0, 50], [F32, BF16, BF16], [F32, F32, BF16])
    try:
        need = B.psgd_clip_workspace(c)
        ws = 1 << 26
        for bad in ((0, need), (ws + 16, need), (ws, need - 1)):
            refused(B.psgd_clip_workspace_init, c, *bad, status=B.PSGD_ERR_WORKSPACE)
            refused(B.psgd_clip_bind, c, [P, 0, 2 * P], [P, 0, 2 * P], *bad, status=B.PSGD_ERR_WORKSPACE)
            refused(B.psgd_clip_norm, c, 1.0, 1.0, P, *bad, status=B.PSGD_ERR_WORKSPACE)
            refused(B.psgd_clip_apply, c, 1.0, 1.0, P, *bad, status=B.PSGD_ERR_WORKSPACE)
        for ins, outs, match in [([0, 0, 2 * P], None, "NULL"), ([P + 2, 0, 2 * P], None, "aligned"),
                                 ([P, 0, 2 * P + 1], None, "aligned"), ([P, 0, 2 * P], [0, 0, 2 * P], "NULL"),
                                 ([P, 0, 2 * P], [P, 0, P + 64], "two outputs"),
                                 ([P, 0, 2 * P], [P + 64, 0, 4 * P], "overlaps a gradient"),
                                 ([P, 0, 2 * P], [2 * P, 0, 4 * P], "overlaps a gradient")]:
            refused(B.psgd_clip_bind, c, ins, outs, ws, need, match=match)
        assert B.lib.psgd_clip_bind(c, None, None, ws, need, None) == B.PSGD_ERR_INVALID_ARG
        for fn in (B.psgd_clip_norm, B.psgd_clip_apply):
            refused(fn, c, 1.0, 1.0, 0, ws, need, match="stats")
            refused(fn, c, 1.0, 1.0, P + 2, ws, need, match="stats")
            refused(fn, c, -1.0, 1.0, P, ws, need, match="max_norm")
            refused(fn, c, float("nan"), 1.0, P, ws, need, match="max_norm")
            refused(fn, c, 1.0, float("inf"), P, ws, need, match="scale")
            refused(fn, c, 1.0, float("nan"), P, ws, need, match="scale")
    finally:
        B.psgd_clip_destroy(c)


def test_clip_in_place_with_another_element_size_is_refused():
    c = B.psgd_clip_create([100], [BF16], [F32])
    try:
        refused(B.psgd_clip_bind, c, [P], [P], 1 << 26, B.psgd_clip_workspace(c), match="overlaps a gradient")
    finally:
        B.psgd_clip_destroy(c)


def test_null_handles():
    assert B.lib.psgd_clip_workspace(None, None) == B.PSGD_ERR_INVALID_ARG
    refused(B.psgd_clip_norm, None, 1.0, 1.0, P, 1 << 26, 1 << 20)
    B.psgd_clip_destroy(None)


def test_refused_bind_keeps_the_old_tensors_alive(monkeypatch):
    """The device table keeps the old addresses when psgd_clip_bind refuses, so
    the handle has to keep the tensors behind them."""
    torch = pytest.importorskip("torch")
    ops = pytest.importorskip("rank_gradient_compression_amd.torch_ops")
    monkeypatch.setattr(ops, "_stream", lambda device: 0)
    monkeypatch.setattr(ops.GradientClip, "_order", lambda self: None, raising=False)
    c = ops.GradientClip.__new__(ops.GradientClip)  # no device: the refusal comes before any device call
    c.handle = B.psgd_clip_create([8, 8], [F32, F32], [F32, F32])
    c.device, c.ws_bytes = torch.device("cuda", 0), B.psgd_clip_workspace(c.handle)
    buf = torch.empty(c.ws_bytes + 256, dtype=torch.uint8)
    c.workspace = buf[-buf.data_ptr() % 256:]
    old = c.grads = c.outs = [torch.zeros(8), torch.zeros(8)]
    new, out = [torch.zeros(8), torch.zeros(8)], torch.zeros(8)
    with pytest.raises(B.PsgdError, match="two outputs overlap"):
        c._bind(new, [out, out])
    assert c.grads is old and c.outs is old
    c.close()


def test_linear_workspace_over_a_buffer_is_refused():
    m, n, k = 64, 96, 512
    need = B.psgd_mx_linear_workspace(m, n, k, BF16)
    x, codes, scales, y, ws = 1 << 24, 1 << 20, 2 << 20, 1 << 25, 1 << 26
    args = lambda w, f=need: (m, n, k, x, BF16, k, codes, scales, y, BF16, n, w, f)  # noqa: E731
    for other, size in ((x, 2 * m * k), (y, 2 * m * n), (codes, n * k // 2), (scales, n * k // 32)):
        assert size % 256 == 0
        for at in (other, other + size - 256, other - need + 256):
            refused(B.psgd_mx_linear, *args(at), match="workspace overlaps")
    # few activations need none: what is passed is not looked at
    assert B.psgd_mx_linear_workspace(0, n, k, BF16) == 0
    B.psgd_mx_linear(0, n, k, 0, BF16, k, codes, scales, 0, BF16, n, codes, need)


@pytest.mark.parametrize("at", [0, 4 * 64 - 1, 4 - 4 * 4 * 64])
def test_quantize_values_over_the_random_bytes_are_refused(at):
    with pytest.raises(B.PsgdError, match="values overlaps rand") as e:
        quant(rand=1 << 22, values=((1 << 22) + at) // 4 * 4, ldv=64)
    assert e.value.status == B.PSGD_ERR_INVALID_ARG


def strided_layers(torch):
    """(x, w): activations and weights whose rows are not contiguous, or empty."""
    g = torch.Generator().manual_seed(3)
    z = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    yield z(64, 40).t(), z(50, 64)
    yield z(40, 64), z(64, 50).t()
    yield z(40, 128)[:, ::2], z(50, 128)[:, ::2]
    yield z(1, 64).expand(40, 64), z(64).expand(50, 64)
    yield z(6, 64, 7).transpose(1, 2), z(50, 64)
    yield z(64), z(50, 64)
    yield z(3, 0, 64), z(50, 64)
    yield z(3, 2, 0), z(50, 0)
    yield z(3, 2, 64), z(0, 64)


def test_autograd_layer_takes_any_strides(monkeypatch):
    """What reaches the library are matrices with contiguous, separate rows
    (the calls themselves stood in for by fp32 products)."""
    torch = pytest.importorskip("torch")
    ops = pytest.importorskip("rank_gradient_compression_amd.torch_ops")

    def readable(m):
        rows, cols = m.shape
        assert (cols <= 1 or m.stride(1) == 1) and (rows <= 1 or m.stride(0) >= cols)
        return m

    operand = lambda x: SimpleNamespace(buf=readable(x).clone(), shape=tuple(x.shape))  # noqa: E731
    monkeypatch.setattr(ops, "mx_linear_forward", lambda x, w: (x @ w.t(), (operand(x), operand(w))))
    monkeypatch.setattr(ops, "mx_linear_backward", lambda dy, saved, rand=None, need_dx=True, need_dw=True: (
        readable(dy) @ saved[1].buf, dy.t() @ saved[0].buf))
    for x, w in strided_layers(torch):
        x, w = x.requires_grad_(True), w.requires_grad_(True)
        y = ops.mx_linear_train(x, w, stochastic=False)
        want = x.detach() @ w.detach().t()
        assert y.shape == want.shape and torch.allclose(y, want, atol=1e-5)
        got = torch.autograd.grad(y.sum() * 2, (x, w))
        assert got[0].shape == x.shape and got[1].shape == w.shape
        assert torch.allclose(got[0], 2 * w.detach().sum(0).expand(x.shape), atol=1e-4)


def test_autograd_layer_lets_go_of_its_operands(monkeypatch):
    """Behind the backward pass, while the result is still held, and not before."""
    torch = pytest.importorskip("torch")
    ops = pytest.importorskip("rank_gradient_compression_amd.torch_ops")
    kept = []

    def forward(x, w):
        saved = [SimpleNamespace(buf=t.clone(), shape=tuple(t.shape)) for t in (x, w)]
        kept.extend(weakref.ref(s.buf) for s in saved)
        return x @ w.t(), tuple(saved)

    monkeypatch.setattr(ops, "mx_linear_forward", forward)
    monkeypatch.setattr(ops, "mx_linear_backward", lambda dy, saved, rand=None, need_dx=True, need_dw=True: (
        dy @ saved[1].buf, dy.t() @ saved[0].buf))
    x, w = torch.randn(4, 64, requires_grad=True), torch.randn(8, 64, requires_grad=True)
    y = ops.mx_linear_train(x, w, stochastic=False)
    y.sum().backward(retain_graph=True)
    gc.collect()
    assert all(r() is not None for r in kept)
    y.sum().backward()
    gc.collect()
    assert all(r() is None for r in kept)
    assert torch.equal(x.grad, 2 * w.detach().sum(0).expand(4, 64))


def test_clip_calls_wait_for_the_stream_of_the_call_before(monkeypatch):
    """On stand-ins for the streams: the waits that the calls of one handle ask
    for, whose workspace one call writes and the next one reads."""
    torch = pytest.importorskip("torch")
    ops = pytest.importorskip("rank_gradient_compression_amd.torch_ops")
    log, now, capturing = [], [None], [False]

    class Stream:
        def __init__(self, raw):
            self.cuda_stream = raw

        def wait_stream(self, other):
            log.append(("wait", self.cuda_stream, other.cuda_stream))

    class Device:
        def __init__(self, device):
            pass

        __enter__ = __exit__ = lambda *a: None

    workspace = SimpleNamespace(data_ptr=lambda: 256, record_stream=lambda s: log.append(("record", s.cuda_stream)))
    c = ops.GradientClip.__new__(ops.GradientClip)
    a, b = Stream(1), Stream(2)
    now[0] = a
    c.handle, c.device, c.workspace, c.ws_bytes, c._last = 0, torch.device("cuda", 0), workspace, 256, a
    c._numel, c._in, c._out = [], [], []
    monkeypatch.setattr(ops, "_raw_stream", lambda index: now[0].cuda_stream)
    monkeypatch.setattr(ops.torch.cuda, "current_stream", lambda device=None: now[0])
    monkeypatch.setattr(ops.torch.cuda, "device", Device)
    monkeypatch.setattr(ops.torch.cuda, "is_current_stream_capturing", lambda: capturing[0])
    monkeypatch.setattr(ops.torch, "empty", lambda *n, **kw: SimpleNamespace(data_ptr=lambda: 4))
    monkeypatch.setattr(ops, "_call", lambda device, fn, *args: log.append(("call", now[0].cuda_stream)))
    monkeypatch.setattr(ops.B, "psgd_clip_bind", lambda *args: log.append(("bind", args[-1])))
    c.clip(1.0)
    now[0] = b
    c.norm()
    c.clip(1.0)
    now[0] = a
    c.bind([], [])
    now[0], capturing[0] = b, True
    c.clip(1.0)
    capturing[0] = False
    c.clip(1.0)
    to_b, to_a = [("wait", 2, 1), ("record", 2)], [("wait", 1, 2), ("record", 1)]
    assert log == [("call", 1), *to_b, ("call", 2), ("call", 2), *to_a, ("bind", 1), ("call", 2), *to_b, ("call", 2)]


def test_linear_warns_where_a_gradient_would_be_lost():
    torch = pytest.importorskip("torch")
    ops = pytest.importorskip("rank_gradient_compression_amd.torch_ops")
    with pytest.warns(UserWarning, match="mx_linear_train"), pytest.raises(ValueError, match="on the GPU"):
        ops.mx_linear(torch.zeros(4, 64, requires_grad=True), SimpleNamespace())

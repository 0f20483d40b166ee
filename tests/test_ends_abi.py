"""Host-side refusals and workspaces of the vocabulary cross entropy and of the
orthogonalised step: every error returns before any device call, so these run
without a GPU."""
import ctypes

import pytest

R = pytest.importorskip("rank_gradient_compression_amd")
B = R.binding

F32, BF16, F16 = B.PSGD_DTYPE_F32, B.PSGD_DTYPE_BF16, B.PSGD_DTYPE_F16
MB = 1 << 20
MAX = 2000000


def refused(fn, *args, status=B.PSGD_ERR_INVALID_ARG, match=None):
    with pytest.raises(B.PsgdError, match=match) as e:
        fn(*args)
    assert e.value.status == status
    assert fn.__name__ in str(e.value)


# addresses that nothing dereferences, a megabyte apart
def xent(**kw):
    a = B.psgd_xent_t()
    base = dict(tokens=10, vocab=64, dim=32, x=1 * MB, ldx=32, w=2 * MB, ldw=32, bias=0, targets=3 * MB, ignore_index=-100,
                weights=0, loss=4 * MB, lse=5 * MB, dx=6 * MB, lddx=32, dw=7 * MB, lddw=32, dbias=0, scale=1.0, mean=1,
                dtype=BF16, dw_dtype=F32, accumulate=0, reserved=0)
    base.update(kw)
    for k, v in base.items():
        setattr(a, k, v)
    return a


WS = 64 * MB


def run(train, ws=WS, nbytes=None, **kw):
    a = xent(**kw)
    fn = B.psgd_xent_train if train else B.psgd_xent_forward
    fn(a, ws, (1 << 40) if nbytes is None else nbytes)


@pytest.mark.parametrize("train", [False, True])
@pytest.mark.parametrize("kw,match", [
    (dict(reserved=1), "reserved"), (dict(dtype=3), "type"), (dict(dtype=-1), "type"), (dict(tokens=-1), "tokens"),
    (dict(tokens=1 << 31), "tokens"), (dict(vocab=0), "vocab"), (dict(dim=0), "dim"), (dict(vocab=MAX + 1), "MAX_DIM"),
    (dict(dim=MAX + 1), "MAX_DIM"), (dict(ldx=31), "stride"), (dict(ldw=31), "stride"), (dict(x=0), "NULL"),
    (dict(w=0), "NULL"), (dict(targets=0), "NULL"), (dict(loss=0), "NULL"), (dict(lse=0), "NULL"),
    (dict(x=MB + 1), "aligned"), (dict(w=2 * MB + 1), "aligned"), (dict(targets=3 * MB + 4), "aligned"),
    (dict(loss=4 * MB + 2), "aligned"), (dict(bias=8 * MB + 1), "aligned"), (dict(weights=8 * MB + 2), "aligned"),
    (dict(scale=float("nan")), "scale"), (dict(scale=float("inf")), "scale"), (dict(loss=5 * MB), "overlap"),
    (dict(loss=1 * MB), "overlap"), (dict(lse=2 * MB + 64), "overlap"), (dict(lse=3 * MB), "overlap"),
    (dict(bias=4 * MB), "overlap"), (dict(ldw=MAX + 8, vocab=2, w=1 << 40), "in place"),
])
def test_xent_refused(train, kw, match):
    fn = B.psgd_xent_train if train else B.psgd_xent_forward
    with pytest.raises(B.PsgdError, match=match) as e:
        run(train, **kw)
    assert e.value.status == B.PSGD_ERR_INVALID_ARG and fn.__name__ in str(e.value)


@pytest.mark.parametrize("kw,match", [
    (dict(dw_dtype=7), "type"), (dict(lddx=31), "stride"), (dict(lddw=31), "stride"), (dict(dx=6 * MB + 1), "aligned"),
    (dict(dw=7 * MB + 2), "aligned"), (dict(dbias=8 * MB + 1), "aligned"), (dict(dx=1 * MB), "overlap"),
    (dict(dw=2 * MB), "overlap"), (dict(dx=7 * MB), "overlap"), (dict(dbias=4 * MB), "overlap"),
    (dict(weights=6 * MB), "overlap"), (dict(dbias=9 * MB, bias=9 * MB), "overlap"),
])
def test_xent_train_refused(kw, match):
    with pytest.raises(B.PsgdError, match=match) as e:
        run(True, **kw)
    assert e.value.status == B.PSGD_ERR_INVALID_ARG


@pytest.mark.parametrize("train", [False, True])
def test_xent_workspace_refused(train):
    need = B.psgd_xent_workspace(xent(), train)
    assert need >= 256 and need % 256 == 0
    for ws, n in ((0, need), (WS + 128, need), (WS, need - 1)):
        with pytest.raises(B.PsgdError, match="workspace") as e:
            run(train, ws=ws, nbytes=n)
        assert e.value.status == B.PSGD_ERR_WORKSPACE
    with pytest.raises(B.PsgdError, match="overlap"):
        run(train, ws=1 * MB)
    lib = B.lib
    out = ctypes.c_size_t()
    assert lib.psgd_xent_workspace(None, 0, ctypes.byref(out)) == B.PSGD_ERR_INVALID_ARG
    assert lib.psgd_xent_workspace(ctypes.byref(xent()), 0, None) == B.PSGD_ERR_INVALID_ARG
    assert lib.psgd_xent_forward(None, WS, 1 << 30, None) == B.PSGD_ERR_INVALID_ARG
    refused(B.psgd_xent_workspace, xent(dim=-1), train)


def test_xent_workspace_does_not_grow_with_the_batch():
    """What a block of tokens needs is bounded; copies of x are all that grows."""
    one = B.psgd_xent_workspace(xent(tokens=16384, vocab=32000, ldx=32), True)
    two = B.psgd_xent_workspace(xent(tokens=1 << 20, vocab=32000, ldx=32), True)
    assert one < (1 << 30) + (1 << 28)
    assert two - one < (1 << 20) * 64 * 2 + (1 << 28)
    # nothing of the logits is kept for the loss alone: sums of 64 columns
    assert B.psgd_xent_workspace(xent(tokens=4096, vocab=32000), False) < 4096 * 501 * 8 + (1 << 16)
    # copies where the operands cannot be read in place
    plain = B.psgd_xent_workspace(xent(), False)
    assert B.psgd_xent_workspace(xent(w=2 * MB + 2), False) > plain
    assert B.psgd_xent_workspace(xent(ldx=33), False) > plain
    assert B.psgd_xent_workspace(xent(dim=31), False) > plain


# ------------------------------------------------------------------ the step
def matrix(**kw):
    base = dict(grad=1 * MB, ldg=16, momentum=2 * MB, param=3 * MB, ldp=16, update=0, ldu=16, rows=8, cols=16, lr_scale=1.0,
                grad_dtype=BF16, param_dtype=BF16, update_dtype=BF16)
    base.update(kw)
    return base


def table(*mats):
    t = (B.psgd_muon_tensor_t * len(mats))()
    for x, m in zip(t, mats):
        for k, v in m.items():
            setattr(x, k, v)
    return t


def opts(**kw):
    base = dict(lr=0.1, momentum=0.9, weight_decay=0.0, a=3.4445, b=-4.7750, c=2.0315, eps=1e-7, steps=5, nesterov=1,
                pieces=0)
    base.update(kw)
    return B.psgd_muon_opts_t(**base)


@pytest.mark.parametrize("kw,match", [
    (dict(rows=-1), "size"), (dict(cols=1000001), "MAX_DIM"), (dict(ldg=15), "stride"), (dict(ldp=15), "stride"),
    (dict(update=4 * MB, ldu=15), "stride"), (dict(grad=0), "NULL"), (dict(param=0), "neither"),
    (dict(grad=MB + 1), "aligned"), (dict(param=3 * MB + 1), "aligned"), (dict(momentum=2 * MB + 2), "aligned"),
    (dict(update=4 * MB + 1), "aligned"), (dict(grad_dtype=3), "type"), (dict(param_dtype=-1), "type"),
    (dict(update=4 * MB, update_dtype=9), "type"), (dict(lr_scale=float("nan")), "finite"),
    (dict(lr_scale=float("inf")), "finite"), (dict(param=1 * MB), "overlap"), (dict(momentum=1 * MB + 64), "overlap"),
    (dict(momentum=3 * MB), "overlap"), (dict(update=3 * MB + 16), "overlap"),
    (dict(update=1 * MB, update_dtype=F16), "overlap"), (dict(update=1 * MB, ldu=17), "overlap"),
    (dict(rows=1000000, cols=1000000, ldg=1000000, ldp=1000000), "too large"),
])
def test_muon_refused(kw, match):
    with pytest.raises(B.PsgdError, match=match) as e:
        B.psgd_muon_step(table(matrix(**kw)), opts(), WS, 1 << 44)
    assert e.value.status == B.PSGD_ERR_INVALID_ARG


@pytest.mark.parametrize("kw,match", [
    (dict(lr=float("nan")), "finite"), (dict(momentum=float("inf")), "finite"), (dict(weight_decay=float("nan")), "finite"),
    (dict(a=float("inf")), "finite"), (dict(eps=-1e-9), "eps"), (dict(eps=float("nan")), "finite"), (dict(steps=0), "steps"),
    (dict(steps=101), "steps"), (dict(pieces=3), "pieces"), (dict(pieces=-1), "pieces"),
    (dict(a=20.0), "singular values"), (dict(a=1e30), "singular values"), (dict(c=3e4), "singular values"),
])
def test_muon_options_refused(kw, match):
    refused(B.psgd_muon_workspace, table(matrix()), opts(**kw), match=match)
    refused(B.psgd_muon_step, table(matrix()), opts(**kw), WS, 1 << 40, match=match)


def test_muon_list_refused():
    two = table(matrix(), matrix(grad=11 * MB, momentum=12 * MB, param=3 * MB + 64))
    refused(B.psgd_muon_step, two, opts(), WS, 1 << 40, match="overlap")
    # an output over another matrix's gradient
    two = table(matrix(), matrix(grad=11 * MB, momentum=12 * MB, param=1 * MB + 128))
    refused(B.psgd_muon_step, two, opts(), WS, 1 << 40, match="overlap")
    # in place is a matrix's own gradient only
    two = table(matrix(), matrix(grad=11 * MB, momentum=0, param=0, update=1 * MB))
    refused(B.psgd_muon_step, two, opts(), WS, 1 << 40, match="overlap")
    lib = B.lib
    out = ctypes.c_size_t()
    assert lib.psgd_muon_step(-1, None, ctypes.byref(opts()), None, 0, None) == B.PSGD_ERR_INVALID_ARG
    assert lib.psgd_muon_step(1, None, ctypes.byref(opts()), None, 0, None) == B.PSGD_ERR_INVALID_ARG
    assert lib.psgd_muon_step(1, table(matrix()), None, None, 0, None) == B.PSGD_ERR_INVALID_ARG
    assert lib.psgd_muon_workspace(1, table(matrix()), ctypes.byref(opts()), None) == B.PSGD_ERR_INVALID_ARG
    assert lib.psgd_muon_workspace(0, None, ctypes.byref(opts()), ctypes.byref(out)) == B.PSGD_OK


def test_muon_workspace():
    need = B.psgd_muon_workspace(table(matrix()), opts())
    for ws, n in ((0, need), (WS + 64, need), (WS, need - 1)):
        refused(B.psgd_muon_step, table(matrix()), opts(), ws, n, status=B.PSGD_ERR_WORKSPACE, match="workspace")
    refused(B.psgd_muon_step, table(matrix()), opts(), 1 * MB, 1 << 40, match="overlap")
    # two pieces need more; matrices that a workgroup each takes whole need nothing;
    # a long list is worked off in groups
    wide = matrix(rows=80, cols=300, ldg=300, ldp=300)
    one = B.psgd_muon_workspace(table(wide), opts(pieces=1))
    assert need == 256 < one < B.psgd_muon_workspace(table(wide), opts(pieces=2))
    big = matrix(rows=4096, cols=4096, ldg=4096, ldp=4096)
    ten, ninety = (B.psgd_muon_workspace(table(*[big] * n), opts()) for n in (16, 90))
    assert ninety == ten


def test_muon_empty_matrices_need_nothing():
    B.psgd_muon_step(table(matrix(rows=0), matrix(cols=0, grad=0, param=0)), opts(), WS, 256)
    B.psgd_muon_step((B.psgd_muon_tensor_t * 0)(), opts(), WS, 256)

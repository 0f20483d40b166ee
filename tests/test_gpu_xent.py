"""Vocabulary cross entropy on the GPU against the definition in 64 bits.

Bounds, entry by entry, before any run (u = 2^-24, half-steps h: bf16 2^-8, fp16
2^-11, e the rounding of E in fp16, 2^-11, or of nothing for fp32 tensors):
  logit    S_tv = sum_d |x||w|:  dl = ((D / 16 + 16) u + r) S + 2u|l|, r = 0 for 16-bit tensors, whose products
           are exact, and 2^-20 for fp32 ones (three roundings to 22 bits in each product, one product left out)
           and the values below 2^-39 of their tensor's largest: D 2^-38 max|x| max|w|
  lse      max over the words of dl, the exponentials' and logarithm's roundings: 2^-20 (1 + |lse|)
  loss     both, and 2u of either
  G        |u| (p (dl + dlse + e + 2^-20) + 2^-24 max_v p) + h |G|;  the target's entry from the loss's error
  dx       sum_v dG |w| s + (V / 16 + 160) u s sum |G||w| + half a step;  dw, db alike, and dw of fp32 and fp16
           tensors what x loses under the weights' powers of two: T 2^-38 (fp16: 2^-24) max|u| max|x| for G of 1
"""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a GPU", allow_module_level=True)

from gpu_util import say  # noqa: E402
from rank_gradient_compression_amd import binding as B  # noqa: E402
from rank_gradient_compression_amd import torch_api as T  # noqa: E402

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16
HALF = {F32: 2.0 ** -22, BF16: 2.0 ** -8, F16: 2.0 ** -11}   # of G as the products take it
OUT = {F32: 2.0 ** -23, BF16: 2.0 ** -8, F16: 2.0 ** -11}    # of what is stored (fp32: the scale's rounding as well)
TINY = {F32: 1e-37, BF16: 1e-37, F16: 2.0 ** -24}
U = 2.0 ** -24


def inputs(t, v, d, dtype, bias, seed=0, ignored=0.2):
    g = torch.Generator(device=DEV)
    g.manual_seed(1000 * t + 10 * v + d + seed)
    x = torch.randn(t, d, generator=g, device=DEV)
    w = torch.randn(v, d, generator=g, device=DEV) * (2.0 / d ** 0.5)
    y = torch.randint(0, v, (t,), generator=g, device=DEV)
    x += (torch.rand(t, 1, generator=g, device=DEV) < 0.5) * w[y] * 1.5
    y[torch.rand(t, generator=g, device=DEV) < ignored] = -100
    b = torch.randn(v, generator=g, device=DEV).to(dtype) if bias else None
    return x.to(dtype), w.to(dtype), y, b


class Reference:
    """The definition in float64 and the bounds above."""

    def __init__(self, x, w, y, b=None, weights=None, scale=1.0, mean=False, ignore=-100):
        dtype = x.dtype
        f32 = dtype == F32
        xd, wd = x.double(), w.double()
        v, d = w.shape
        self.keep = (y >= 0) & (y != ignore)
        good = self.keep & (y < v)
        l = xd @ wd.t()
        if b is not None:
            l = l + b.double()
        self.lse = torch.logsumexp(l, 1)
        at = y.clamp(0, v - 1).view(-1, 1)
        self.loss = torch.where(self.keep, self.lse - l.gather(1, at).view(-1), torch.zeros_like(self.lse))
        self.loss = torch.where(self.keep & (y >= v), torch.full_like(self.loss, float("nan")), self.loss)
        size = xd.abs() @ wd.abs().t()
        dl = ((d / 16 + 16) * U + (2.0 ** -20 if f32 else 0.0)) * size + 2 * U * l.abs().nan_to_num(posinf=0.0, neginf=0.0)
        if f32:
            dl = dl + d * 2.0 ** -38 * float(xd.abs().max()) * float(wd.abs().max())
        dl = torch.where(torch.isinf(l), torch.zeros_like(dl), dl)
        self.dlse = dl.max(1).values + 2.0 ** -20 * (1 + self.lse.abs())
        self.dloss = self.dlse + dl.gather(1, at).view(-1) + 2 * U * (self.lse.abs() + l.gather(1, at).view(-1).abs())
        s = scale / max(1, int(self.keep.sum())) if mean else scale
        u = torch.ones_like(self.lse) if weights is None else weights.double()
        u = torch.where(good, u, torch.zeros_like(u))[:, None]
        p = torch.exp(l - self.lse[:, None])
        hot = torch.zeros_like(p).scatter_(1, at, 1.0)
        e = 0.0 if f32 else 2.0 ** -11
        g = torch.where(u != 0, (p - hot) * u, torch.zeros_like(p))
        dg = u.abs() * (p * (dl + self.dlse[:, None] + e + 2.0 ** -20) + 2.0 ** -24 * p.max(1, keepdim=True).values)
        dg = torch.where(hot > 0, u.abs() * p * self.dloss[:, None] + 2.0 ** -20 * g.abs(), dg)
        dg = torch.where(u != 0, dg, torch.zeros_like(dg)) + HALF[dtype] * g.abs()
        xz = torch.where(good[:, None], xd, torch.zeros_like(xd))
        a = abs(s)
        self.dx, self.dw, self.db = s * (g @ wd), s * (g.t() @ xz), s * g.sum(0)
        xe = 2.0 ** -20 if f32 else 0.0  # (the other operand's pieces)
        self.tol_dx = a * (dg @ wd.abs()) + a * ((v / 16 + 160) * U + xe) * (g.abs() @ wd.abs())
        t = x.shape[0]
        self.tol_dw = a * (dg.t() @ xz.abs()) + a * ((t / 16 + 160) * U + xe) * (g.abs().t() @ xz.abs())
        if weights is not None and dtype != BF16:
            size = float(u.abs().max()) * (float(xz.abs().max()) * 2.0 ** -38 if f32 else 2.0 ** -24)
            self.tol_dw = self.tol_dw + a * t * size
        self.tol_db = a * dg.sum(0) + a * (t + 64) * U * g.abs().sum(0)


def close(name, got, want, tol, dtype=None):
    got = got.double()
    if dtype is not None:
        tol = tol + OUT[dtype] * (want.abs() + tol) + TINY[dtype]
    bad = ~((got - want).abs() <= tol)
    bad &= ~(torch.isnan(got) & torch.isnan(want))
    if bad.any():
        i = int(bad.flatten().nonzero()[0])
        raise AssertionError(f"{name}: {int(bad.sum())} of {bad.numel()} entries off; entry {i}: "
                             f"{float(got.flatten()[i])} for {float(want.flatten()[i])}, "
                             f"bound {float(tol.expand_as(want).flatten()[i])}")


def check(ref, loss, lse, dx=None, dw=None, db=None):
    close("lse", lse, ref.lse, ref.dlse)
    close("loss", loss, ref.loss, torch.where(ref.keep, ref.dloss, torch.zeros_like(ref.dloss)))
    if dx is not None:
        close("dx", dx, ref.dx, ref.tol_dx, dx.dtype)
    if dw is not None:
        close("dw", dw, ref.dw, ref.tol_dw, dw.dtype)
    if db is not None:
        close("dbias", db, ref.db, ref.tol_db, db.dtype)


SIZES = [(1, 1, 1), (1, 2, 8), (3, 5, 7), (1, 333, 64), (16, 64, 64), (17, 65, 130), (32, 97, 33), (33, 64, 72), (20, 1000, 650),
         (64, 640, 256), (100, 129, 65), (129, 513, 200), (257, 300, 1000), (700, 1111, 96), (300, 4000, 64)]


@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("t,v,d", SIZES)
def test_forward_and_gradients(t, v, d, dtype):
    bias = (t + v) % 2 == 0
    x, w, y, b = inputs(t, v, d, dtype, bias)
    say(f"[xent] {t} x {v} x {d} {dtype} bias={bias}")
    ref = Reference(x, w, y, b, mean=True)
    loss, lse = T.cross_entropy(x, w, y, b)
    check(ref, loss, lse)
    loss2, lse2, dx, dw, db = T.cross_entropy_train(x, w, y, b)
    check(ref, loss2, lse2, dx, dw, db)
    assert torch.equal(loss, loss2) and torch.equal(lse, lse2)
    assert (db is None) == (not bias) and dx.dtype == dw.dtype == dtype


@pytest.mark.parametrize("dtype,t,v,d", [(BF16, 600, 33278 // 2, 128), (BF16, 2100, 8200, 64), (F32, 520, 16700, 96)])
def test_large_tiles(dtype, t, v, d):
    """Enough tiles of 256 x 256 to be taken, last ones cut on both sides."""
    x, w, y, b = inputs(t, v, d, dtype, True, seed=3)
    say(f"[xent] large {t} x {v} x {d} {dtype}")
    loss, lse, dx, dw, db = T.cross_entropy_train(x, w, y, b)
    check(Reference(x, w, y, b, mean=True), loss, lse, dx, dw, db)


@pytest.mark.parametrize("dtype", [BF16, F16, F32])
def test_weights_scale_and_accumulation(dtype):
    t, v, d = 90, 210, 48
    x, w, y, b = inputs(t, v, d, dtype, True, seed=5)
    g = torch.Generator(device=DEV)
    g.manual_seed(1)
    u = torch.randn(t, generator=g, device=DEV) * torch.logspace(-6, 3, t, device=DEV)
    u[7] = 0.0
    for scale, reduction in ((-2.5, "sum"), (1024.0, "mean")):
        ref = Reference(x, w, y, b, u, scale, reduction == "mean")
        loss, lse, dx, dw, db = T.cross_entropy_train(x, w, y, b, weights=u, reduction=reduction, scale=scale)
        check(ref, loss, lse, dx, dw, db)
        # fp32 dw, then the same again on top: twice, exactly
        out = torch.zeros(v, d, device=DEV)
        db32 = torch.zeros(v, dtype=dtype, device=DEV)
        T.cross_entropy_train(x, w, y, b, weights=u, reduction=reduction, scale=scale, dw=out, dbias=db32)
        one = out.clone()
        close("dw in fp32", one, ref.dw, ref.tol_dw, F32)
        T.cross_entropy_train(x, w, y, b, weights=u, reduction=reduction, scale=scale, dw=out, dbias=db32, accumulate=True)
        assert torch.equal(out, 2 * one)


def test_accumulation_in_16_bits():
    x, w, y, b = inputs(200, 300, 64, BF16, True, seed=6)
    ref = Reference(x, w, y, b, mean=True)
    old = torch.randn(300, 64, device=DEV).to(BF16)
    oldb = torch.randn(300, device=DEV).to(BF16)
    dw, db = old.clone(), oldb.clone()
    T.cross_entropy_train(x, w, y, b, dw=dw, dbias=db, accumulate=True)
    close("dw", dw, old.double() + ref.dw, ref.tol_dw, BF16)
    close("dbias", db, oldb.double() + ref.db, ref.tol_db, BF16)


def test_views_and_strides():
    """Rows with gaps, addresses off 16 bytes, results in views of a flat buffer;
    what lies between and behind stays as it was."""
    t, v, d = 70, 150, 40
    for dtype in (BF16, F16, F32):
        x, w, y, b = inputs(t, v, d, dtype, False, seed=7)
        ref = Reference(x, w, y, mean=True)
        for off, gap in ((0, 0), (0, 8), (1, 3), (8, 0), (2, 1)):
            xs = torch.full((t, d + off + gap), float("nan"), dtype=dtype, device=DEV)
            ws = torch.full((v, d + off + gap), float("nan"), dtype=dtype, device=DEV)
            xv, wv = xs[:, off:off + d], ws[:, off:off + d]
            xv.copy_(x), wv.copy_(w)
            flat = torch.full((off + v * (d + gap) + 5,), 7.0, device=DEV)
            dwv = flat[off:off + v * (d + gap)].view(v, d + gap)[:, :d]
            loss, lse, dx, dw, _ = T.cross_entropy_train(xv, wv, y, dw=dwv)
            say(f"[xent] views {dtype} off {off} gap {gap}")
            check(ref, loss, lse, dx)
            close("dw", dwv, ref.dw, ref.tol_dw, F32)
            rest = flat.clone()
            rest[off:off + v * (d + gap)].view(v, d + gap)[:, :d] = 7.0
            assert torch.equal(rest, torch.full_like(rest, 7.0))


def test_only_what_is_wanted():
    x, w, y, b = inputs(50, 80, 32, BF16, True, seed=8)
    full = T.cross_entropy_train(x, w, y, b)
    for need in ((True, False, False), (False, True, False), (False, False, True), (False, False, False)):
        got = T.cross_entropy_train(x, w, y, b, need_dx=need[0], need_dw=need[1], need_dbias=need[2])
        for n, a, c in zip((True, True) + need, got, full):
            assert (a is not None) == n and (not n or torch.equal(a, c))


@pytest.mark.parametrize("dtype", [BF16, F16, F32])
def test_ignored_tokens_may_hold_anything(dtype):
    t, v, d = 140, 200, 40
    x, w, y, b = inputs(t, v, d, dtype, True, seed=9, ignored=0.0)
    gone = torch.arange(t, device=DEV) % 3 == 0
    y[gone] = torch.where(torch.arange(t, device=DEV) % 2 == 0, 11, -7)[gone]
    y[~gone & (y == 11)] = 12
    clean = T.cross_entropy_train(x, w, y, b, ignore_index=11)
    bad = x.clone()
    bad[gone] = float("nan")
    bad[0] = float("inf")
    u = torch.ones(t, device=DEV)
    u[gone] = float("nan")
    got = T.cross_entropy_train(bad, w, y, b, ignore_index=11, weights=u)
    if dtype == F32:  # (the scale of x's pieces goes by what is finite, here the other rows)
        check(Reference(torch.where(gone[:, None], torch.zeros_like(x), x), w, y, b, mean=True, ignore=11),
              got[0], torch.where(gone, torch.logsumexp(b.double(), 0), got[1].double()), got[2], got[3], got[4])
    else:
        for a, c in zip((got[0], got[2], got[3], got[4]), (clean[0], clean[2], clean[3], clean[4])):
            assert torch.equal(a, c)
        assert torch.equal(got[1][~gone], clean[1][~gone])
    assert not got[0][gone].any() and not got[2][gone].any() and torch.isnan(got[1][gone]).all()


def test_every_token_ignored():
    x, w, y, b = inputs(40, 90, 24, BF16, True, seed=10)
    y[:] = -100
    loss, lse, dx, dw, db = T.cross_entropy_train(x, w, y, b)
    assert not any(v.any() for v in (loss, dx, dw, db)) and torch.isfinite(lse).all()
    xl = x.clone().requires_grad_(True)
    total = T.linear_cross_entropy(xl, w, y)
    total.backward()
    assert float(total.detach()) == 0.0 and not xl.grad.any()


def test_targets_past_the_vocabulary():
    x, w, y, b = inputs(40, 90, 24, BF16, False, seed=11, ignored=0.0)
    y[3], y[39] = 90, 1 << 40
    loss, lse, dx, dw, _ = T.cross_entropy_train(x, w, y)
    assert torch.isnan(loss[[3, 39]]).all() and torch.isfinite(lse).all() and not dx[[3, 39]].any()
    check(Reference(x, w, y, mean=True), loss, lse, dx, dw)


@pytest.mark.parametrize("t", [5, 200])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_masked_words(t, dtype):
    """A bias of -infinity, or of the type's lowest value, takes words out: a whole
    tile of them, the first and the last."""
    v, d = 600, 40
    x, w, y, b = inputs(t, v, d, dtype, True, seed=12, ignored=0.0)
    y.clamp_(min=300, max=500)
    b[:280], b[-3:] = -float("inf"), torch.finfo(dtype).min
    ref = Reference(x, w, y, b, mean=True)
    loss, lse, dx, dw, db = T.cross_entropy_train(x, w, y, b)
    check(ref, loss, lse, dx, dw, db)
    assert not dw[:280].any() and not dw[-3:].any() and not db[:280].any()


def test_no_word_left_and_not_finite():
    x, w, y, b = inputs(40, 100, 24, BF16, True, seed=13, ignored=0.0)
    _, lse = T.cross_entropy(x, w, y, torch.full_like(b, -float("inf")))
    assert torch.isinf(lse).all() and (lse < 0).all()
    x[5] = float("nan")
    loss, lse, dx, _, _ = T.cross_entropy_train(x, w, y, b)
    ok = torch.arange(40, device=DEV) != 5
    assert torch.isnan(loss[5]) and torch.isnan(lse[5]) and torch.isnan(dx[5]).all()
    assert torch.isfinite(loss[ok]).all() and torch.isfinite(lse[ok]).all() and torch.isfinite(dx[ok]).all()


def test_confident_and_far_logits():
    """Probabilities next to 1 and to 0: the target's entry of G does not cancel."""
    t, v, d = 60, 128, 64
    for dtype in (BF16, F16, F32):
        w = torch.zeros(v, d, dtype=dtype, device=DEV)
        w[torch.arange(v, device=DEV), torch.arange(v, device=DEV) % d] = 1.0
        x = torch.zeros(t, d, dtype=dtype, device=DEV)
        y = torch.arange(t, device=DEV) % d
        x[torch.arange(t, device=DEV), y] = torch.linspace(4.0, 60.0, t, device=DEV).to(dtype)
        say(f"[xent] confident {dtype}")
        loss, lse, dx, dw, _ = T.cross_entropy_train(x, w, y, reduction="sum")
        check(Reference(x, w, y), loss, lse, dx, dw)


@pytest.mark.parametrize("scale", [2.0 ** -60, 2.0 ** 60])
def test_fp32_of_any_size(scale):
    """Tiny hidden states and huge weights, and the other way round."""
    x, w, y, _ = inputs(50, 120, 32, F32, False, seed=14)
    x, w = x * scale, w / scale
    loss, lse, dx, dw, _ = T.cross_entropy_train(x, w, y, scale=4.0)
    check(Reference(x, w, y, scale=4.0, mean=True), loss, lse, dx, dw)


def test_no_token():
    w, b = torch.randn(30, 8, device=DEV).to(BF16), torch.randn(30, device=DEV).to(BF16)
    x, y = torch.empty(0, 8, dtype=BF16, device=DEV), torch.empty(0, dtype=torch.int64, device=DEV)
    loss, lse = T.cross_entropy(x, w, y, b)
    assert loss.shape == lse.shape == (0,)
    loss, lse, dx, dw, db = T.cross_entropy_train(x, w, y, b)
    assert dx.shape == (0, 8) and not dw.any() and not db.any()
    old = torch.ones(30, 8, dtype=BF16, device=DEV)
    T.cross_entropy_train(x, w, y, b, dw=old, dbias=b.clone(), accumulate=True)
    assert torch.equal(old, torch.ones_like(old))


def test_equal_calls_give_equal_bits():
    for dtype, t in ((BF16, 700), (F32, 300), (F16, 9)):
        x, w, y, b = inputs(t, 2000, 96, dtype, True, seed=15)
        first = T.cross_entropy_train(x, w, y, b)
        torch.full((1 << 26,), float("nan"), device=DEV)  # (what the next workspace finds)
        again = T.cross_entropy_train(x, w, y, b)
        assert all(torch.equal(a, c) for a, c in zip(first, again))


def test_blocks_of_tokens():
    """More tokens than a block holds: dw adds up over the blocks, in fp32 where it
    is 16-bit itself."""
    v, d = 128, 16
    t = (1 << 30) // (v * 2) + 300
    x, w, y, b = inputs(t, v, d, BF16, True, seed=16)
    say(f"[xent] {t} tokens in two blocks")
    loss, lse, dx, dw, db = T.cross_entropy_train(x, w, y, b, scale=4096.0, need_dx=True)
    out = torch.zeros(v, d, device=DEV)
    T.cross_entropy_train(x, w, y, b, scale=4096.0, need_dx=False, need_dbias=False, dw=out)
    assert torch.equal(out.to(BF16), dw)
    n = int((y >= 0).sum())
    want_w, want_b = torch.zeros(v, d, dtype=torch.float64, device=DEV), torch.zeros(v, dtype=torch.float64, device=DEV)
    tol_w, tol_b = torch.zeros_like(want_w), torch.zeros_like(want_b)
    step = 1 << 19
    for a in range(0, t, step):
        ref = Reference(x[a:a + step], w, y[a:a + step], b, scale=4096.0 / n)
        check(ref, loss[a:a + step], lse[a:a + step], dx[a:a + step])
        want_w += ref.dw
        want_b += ref.db
        tol_w += ref.tol_dw
        tol_b += ref.tol_db
    close("dw", dw, want_w, tol_w, BF16)
    close("dbias", db, want_b, tol_b, BF16)


def test_offsets_beyond_32_bits():
    """Hidden states of more than 2^31 values."""
    d, v = 4096, 40
    t = (1 << 31) // d + 500
    g = torch.Generator(device=DEV)
    g.manual_seed(2)
    x = torch.zeros(t, d, dtype=BF16, device=DEV)
    x[-700:] = torch.randn(700, d, generator=g, device=DEV).to(BF16)
    w = (torch.randn(v, d, generator=g, device=DEV) / 32).to(BF16)
    y = torch.full((t,), -100, device=DEV)
    y[-700:] = torch.randint(0, v, (700,), generator=g, device=DEV)
    say("[xent] hidden states past 2^31 values")
    loss, lse, dx, dw, _ = T.cross_entropy_train(x, w, y)
    ref = Reference(x[-700:], w, y[-700:], mean=True)
    check(ref, loss[-700:], lse[-700:], dx[-700:], dw)
    assert not loss[:-700].any() and not dx[:1000].any()


# ------------------------------------------------------------------- autograd
@pytest.mark.parametrize("reduction", ["mean", "sum", "none"])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_autograd(reduction, dtype):
    x, w, y, b = inputs(60, 140, 40, dtype, True, seed=17)
    x3, y3 = x.view(4, 15, 40), y.view(4, 15)
    leaves = [v.clone().requires_grad_(True) for v in (x3, w, b)]
    out = T.linear_cross_entropy(leaves[0], leaves[1], y3, leaves[2], reduction=reduction)
    up = torch.randn(out.shape, device=DEV) if reduction == "none" else torch.tensor(0.3, device=DEV)
    out.backward(up)
    # (an incoming 0.3 is a factor behind the rounding to the type: one more half-step)
    ref = Reference(x, w, y, b, up.reshape(-1) if reduction == "none" else None, 1.0 if reduction == "none" else float(up),
                    reduction == "mean")
    for name, leaf, want, tol in (("dx", leaves[0], ref.dx, ref.tol_dx), ("dw", leaves[1], ref.dw, ref.tol_dw),
                                  ("db", leaves[2], ref.db, ref.tol_db)):
        assert leaf.grad.dtype == dtype and leaf.grad.shape == leaf.shape
        close(name, leaf.grad.reshape(want.shape), want, tol + 2 * OUT[dtype] * want.abs(), dtype)
    keep = torch.where(ref.keep, ref.dloss, torch.zeros_like(ref.dloss))
    if reduction == "none":
        close("loss", out.reshape(-1), ref.loss, keep)
    else:
        n = int(ref.keep.sum()) if reduction == "mean" else 1
        close("total", out, ref.loss.sum() / n, (keep.sum() + 60 * U * ref.loss.abs().sum()) / n + U)


@pytest.mark.parametrize("dtype,up", [(F16, 65536.0), (F16, 2.0 ** -10), (BF16, 0.3), (F32, 1e30)])
def test_autograd_incoming_scale(dtype, up):
    """An incoming scale beyond the type's own range or digits: the bounds are those
    of gradients of a loss times that scale, and one more rounding of the product."""
    x, w, y, b = inputs(70, 500, 40, dtype, True, seed=23)
    leaves = [v.clone().requires_grad_(True) for v in (x, w, b)]
    T.linear_cross_entropy(leaves[0], leaves[1], y, leaves[2]).backward(torch.tensor(up, device=DEV))
    # (float16 takes the scale as a weight of every token, with the bound of weights)
    weights = torch.full((70,), up, device=DEV) if dtype == F16 else None
    ref = Reference(x, w, y, b, weights, 1.0 if dtype == F16 else up, True)
    for name, leaf, want, tol in (("dx", leaves[0], ref.dx, ref.tol_dx), ("dw", leaves[1], ref.dw, ref.tol_dw),
                                  ("db", leaves[2], ref.db, ref.tol_db)):
        assert torch.isfinite(leaf.grad).all(), name
        close(name, leaf.grad, want, tol + OUT[dtype] * want.abs(), dtype)


@pytest.mark.parametrize("reduction", ["mean", "sum"])
def test_autograd_captured(reduction):
    """Loss and gradients of 20,000 tokens in a graph, replayed between eager work."""
    x, w, y, b = inputs(20000, 60, 24, BF16, True, seed=24)

    def step(*leaves):
        out = T.linear_cross_entropy(leaves[0], leaves[1], y, leaves[2], reduction=reduction)
        return (out.detach(),) + torch.autograd.grad(out, leaves)

    fixed = [v.clone().requires_grad_(True) for v in (x, w, b)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(*fixed)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step(*fixed)
    for k in range(4):
        with torch.no_grad():
            fixed[0].copy_(x.roll(k, 0) * (1 + k))
        graph.replay()
        torch.cuda.synchronize()
        want = step(*[v.detach().clone().requires_grad_(True) for v in fixed])
        for name, a, e in zip(("total", "dx", "dw", "db"), got, want):
            assert torch.equal(a, e), (name, k)


def test_autograd_parts_and_strides():
    x, w, y, b = inputs(30, 50, 24, F32, True, seed=18)
    wt = w.t().contiguous().requires_grad_(True)  # (a transposed weight is copied)
    T.linear_cross_entropy(x, wt.t(), y, b).backward()
    close("dw", wt.grad.t(), Reference(x, w, y, b, mean=True).dw, Reference(x, w, y, b, mean=True).tol_dw, F32)
    xe = torch.randn(1, 24, device=DEV, requires_grad=True)  # expanded: its gradients add up
    T.linear_cross_entropy(xe.expand(30, 24), w, y, reduction="sum").backward()
    ref = Reference(xe.detach().expand(30, 24), w, y)
    close("dx", xe.grad[0], ref.dx.sum(0), ref.tol_dx.sum(0) + 30 * U * ref.dx.abs().sum(0), F32)
    bl = b.clone().requires_grad_(True)
    T.linear_cross_entropy(x, w, y, bl, reduction="none").sum().backward()
    assert bl.grad.shape == b.shape
    with torch.no_grad():
        assert not T.linear_cross_entropy(x.requires_grad_(True), w, y).requires_grad


def test_autograd_gradient_is_the_difference():
    x, w, y, b = inputs(12, 30, 16, F32, True, seed=19, ignored=0.1)
    leaf = w.clone().requires_grad_(True)
    T.linear_cross_entropy(x, leaf, y, b, reduction="sum").backward()
    g = torch.Generator(device=DEV)
    g.manual_seed(3)
    for _ in range(3):
        step = torch.randn(w.shape, generator=g, device=DEV)
        h = 1e-2
        f = [float(T.cross_entropy(x, w + s * h * step, y, b)[0].double().sum()) for s in (1, -1)]
        want = float((leaf.grad.double() * step.double()).sum())
        # the third derivative of a log-sum of exponentials along a direction of logits of size q is at most q^3 / 4
        q = float((x.double() @ step.double().t()).abs().max()) * 2
        bound = len(y) * q ** 3 / 24 * h ** 2 + len(y) * 2.0 ** -18 * 10 / h
        assert abs((f[0] - f[1]) / (2 * h) - want) <= bound


# --------------------------------------------------------- streams and graphs
def test_another_stream_and_two_calls_at_once():
    x, w, y, b = inputs(500, 3000, 128, BF16, True, seed=20)
    want = T.cross_entropy_train(x, w, y, b)
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    got = []
    for _ in range(4):
        for s in (s1, s2):
            with torch.cuda.stream(s):
                got.append(T.cross_entropy_train(x, w, y, b))
    torch.cuda.synchronize()
    for g in got:
        assert all(torch.equal(a, c) for a, c in zip(g, want))


@pytest.mark.parametrize("t,dtype", [(6, BF16), (300, F32)])
def test_captured_and_replayed(t, dtype):
    x, w, y, b = inputs(t, 900, 72, dtype, True, seed=21)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        T.cross_entropy_train(x, w, y, b)
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = T.cross_entropy_train(x, w, y, b)
    for k in range(4):
        x2, _, y2, _ = inputs(t, 900, 72, dtype, True, seed=30 + k)
        x.copy_(x2), y.copy_(y2)
        want = T.cross_entropy_train(x, w, y, b)  # (eager work between the replays)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, c) for a, c in zip(out, want)), f"replay {k}"


# ------------------------------------------------------------------- refusals
def test_torch_layer_refuses():
    x, w, y, b = inputs(20, 30, 16, BF16, True)
    cpu = torch.zeros(20, 16, dtype=BF16)
    for bad in (lambda: T.cross_entropy(cpu, w, y), lambda: T.cross_entropy(x, w.float(), y),
                lambda: T.cross_entropy(x, w[:, :8], y), lambda: T.cross_entropy(x, w, y[:5]),
                lambda: T.cross_entropy(x, w, y.int()), lambda: T.cross_entropy(x, w, y, b.float()),
                lambda: T.cross_entropy(x, w, y, b[:3]), lambda: T.cross_entropy(x.t(), w, y),
                lambda: T.cross_entropy(x.double(), w.double(), y), lambda: T.cross_entropy(x[0], w, y),
                lambda: T.cross_entropy_train(x, w, y, reduction="none"),
                lambda: T.cross_entropy_train(x, w, y, weights=torch.ones(20, dtype=BF16, device=DEV)),
                lambda: T.cross_entropy_train(x, w, y, weights=torch.ones(19, device=DEV)),
                lambda: T.cross_entropy_train(x, w, y, accumulate=True),
                lambda: T.cross_entropy_train(x, w, y, b, dw=torch.zeros(30, 16, device=DEV), accumulate=True),
                lambda: T.cross_entropy_train(x, w, y, dw=torch.zeros(30, 15, device=DEV)),
                lambda: T.cross_entropy_train(x, w, y, b, dbias=torch.zeros(30, device=DEV)),
                lambda: T.linear_cross_entropy(x, w, y, reduction="max"), lambda: T.linear_cross_entropy(x, w, y[:4])):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(B.PsgdError, match="overlap"):
        T.cross_entropy_train(x, w, y, dw=w)
    with pytest.raises(B.PsgdError, match="vocab"):
        T.cross_entropy(x, w[:0], y)
    with pytest.raises(B.PsgdError, match="dim"):
        T.cross_entropy(x[:, :0], w[:, :0], y)
    with pytest.raises(B.PsgdError, match="scale"):
        T.cross_entropy_train(x, w, y, scale=float("nan"))

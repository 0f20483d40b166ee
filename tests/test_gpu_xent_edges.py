"""Edges of the vocabulary cross entropy on the GPU, against the definition in 64
bits: masks, offsets that all logits share, rows and weights of very different
sizes, many blocks of tokens, many tokens.

Bounds as in test_gpu_xent.py where nothing else is said (u = 2^-24)."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a GPU", allow_module_level=True)

from gpu_util import say  # noqa: E402
from test_gpu_xent import BF16, DEV, F16, F32, OUT, Reference, U, check, close, inputs  # noqa: E402
from rank_gradient_compression_amd import binding as B  # noqa: E402
from rank_gradient_compression_amd import torch_api as T  # noqa: E402
from rank_gradient_compression_amd import torch_xent as X  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("mask", [-1e9, -1e10, None])
@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("t", [5, 200])
def test_finite_masks_of_whole_segments(t, dtype, mask):
    """A large negative bias (None: the type's lowest value) over whole segments of
    words and over the padded end of the vocabulary: the words' probabilities are
    exp of less than -60000, zero, so all is as over the words that are left."""
    v, d = 600, 40
    x, w, y, b = inputs(t, v, d, dtype, True, seed=40, ignored=0.1)
    lowest = torch.finfo(dtype).min
    gone = torch.zeros(v, dtype=torch.bool, device=DEV)
    gone[64:192] = gone[320:352] = gone[576:] = True
    b[gone] = max(mask or lowest, lowest)
    live = (~gone).nonzero().flatten()
    y = torch.where(y >= 0, live[y.clamp(min=0) % len(live)], y)
    place = torch.cumsum((~gone).long(), 0) - 1
    say(f"[xent] masks {t} {dtype} {mask}")
    loss, lse, dx, dw, db = T.cross_entropy_train(x, w, y, b)
    ref = Reference(x, w[live], torch.where(y >= 0, place[y.clamp(min=0)], y), b[live], mean=True)
    check(ref, loss, lse, dx, dw[live], db[live])
    assert not dw[gone].any() and not db[gone].any()
    again = T.cross_entropy(x, w, y, b)
    assert torch.equal(again[0], loss) and torch.equal(again[1], lse)


@pytest.mark.parametrize("t", [20, 130])
@pytest.mark.parametrize("top", [100.0, 1000.0])
@pytest.mark.parametrize("dtype", [BF16, F16, F32])
def test_an_offset_of_all_logits_cancels(t, top, dtype):
    """Logits of 100 or 1000 and some that every type holds exactly, as does fp32 the
    sums: what is lost is relative to the distances from a token's largest logit
    (at most 20 here), not to the logits.
      loss  the sum of 90 exponentials 2^-19, logf 2^-22, a difference and a rounding of at most 25: 2^-17 in all
      G     E (fp16: 2^-11 p and 2^-25 of the largest p; fp32 tensors: exact), exponentials and sums 2^-18 p (the
            target's entry: p times the loss's error, and expm1f's 2^-22), and half a step of the type"""
    v, d = 90, 8
    g = torch.Generator(device=DEV)
    g.manual_seed(41)
    near = torch.randint(0, 81, (v,), generator=g, device=DEV) * 0.25 - 20.0
    w = torch.zeros(v, d, dtype=dtype, device=DEV)
    w[:, 0], w[:, 1], w[:, 2] = 1.0, near.to(dtype), 1.0
    x = torch.zeros(t, d, dtype=dtype, device=DEV)
    x[:, 0], x[:, 1] = top, torch.exp2(-(torch.arange(t, device=DEV) % 4).double()).to(dtype)
    x[torch.arange(t, device=DEV), 2 + torch.arange(t, device=DEV) % 6] = 0.5
    y = torch.randint(0, v, (t,), generator=g, device=DEV)
    y[0] = int(near.argmax())
    l = x.double() @ w.double().t()
    assert torch.equal(l.float().double(), l)
    l = l - top
    want = torch.logsumexp(l, 1) - l.gather(1, y[:, None])[:, 0]
    say(f"[xent] offset {top} {t} {dtype}")
    out = torch.zeros(v, d, device=DEV)
    loss, lse, dx, dw, _ = T.cross_entropy_train(x, w, y, reduction="sum", dw=out)
    close("loss", loss, want, torch.full_like(want, 2.0 ** -17))
    p = torch.softmax(l, 1)
    hot = torch.nn.functional.one_hot(y, v).bool()
    G = torch.where(hot, torch.expm1(-want)[:, None].expand_as(p), p)
    half = {F32: 2.0 ** -22, BF16: 2.0 ** -8, F16: 2.0 ** -11}[dtype]
    e = 0.0 if dtype == F32 else 2.0 ** -11
    dg = torch.where(hot, p * 2.0 ** -17 + 2.0 ** -22 * G.abs(), p * (e + 2.0 ** -18) + 2.0 ** -25 * p.max(1, keepdim=True).values)
    dg = dg + half * G.abs()
    xd, wd = x.double(), w.double()
    close("dx", dx, G @ wd, dg @ wd.abs() + 200 * U * (G.abs() @ wd.abs()), dtype)
    # (by column: the one that all share is 100 or 1000, the others 1)
    close("dw", dw, G.t() @ xd, dg.t() @ xd.abs() + (200 * U) * (G.abs().t() @ xd.abs()), F32)


@pytest.mark.parametrize("t", [3, 100])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_every_word_at_the_lowest_value(t, dtype):
    """Logits that fp32 cannot tell apart: the words are equally likely."""
    v, d = 200, 16
    x, w, y, b = inputs(t, v, d, dtype, True, seed=42, ignored=0.0)
    b[:] = torch.finfo(dtype).min
    loss, lse, dx, dw, db = T.cross_entropy_train(x, w, y, b, reduction="sum", dw=torch.zeros(v, d, device=DEV))
    want = torch.full_like(loss, float(np.log(v))).double()
    close("loss", loss, want, torch.full_like(want, 2.0 ** -20))
    n = torch.bincount(y, minlength=v).double()
    e = {F32: 2.0 ** -18, BF16: 2.0 ** -10}[dtype]
    close("dbias", db, t / v - n, t / v * e + n * 2.0 ** -18, dtype)


@pytest.mark.parametrize("size", [1e9, 1e12, 3e38])
@pytest.mark.parametrize("t", [12, 140])
def test_large_values_in_ignored_rows(t, size):
    """fp32 padding of any finite size: bounds of the other rows alone."""
    v, d = 200, 40
    x, w, y, b = inputs(t, v, d, F32, True, seed=43, ignored=0.0)
    gone = torch.arange(t, device=DEV) % 3 == 0
    x[gone] = size
    x[gone, ::2] *= -1
    y[gone] = -100
    pad = gone.clone()
    y[1] = v + 5  # (past the vocabulary: no part of the gradients either)
    x[1] = size
    gone[1] = True
    say(f"[xent] padding of {size} beside {t} tokens")
    loss, lse, dx, dw, db = T.cross_entropy_train(x, w, y, b, reduction="sum", scale=0.25)
    ref = Reference(x[~gone], w, y[~gone], b, scale=0.25)
    check(ref, loss[~gone], lse[~gone], dx[~gone], dw, db)
    assert not loss[pad].any() and torch.isnan(loss[1]) and not dx[gone].any()
    again = T.cross_entropy(x, w, y, b)
    assert torch.equal(again[0][~gone], loss[~gone]) and torch.equal(again[1][~gone], lse[~gone])
    # a weight of zero takes a row out just so
    y[gone] = 3
    u = torch.where(gone, 0.0, 1.0)
    dx, dw = T.cross_entropy_train(x, w, y, b, reduction="sum", scale=0.25, weights=u)[2:4]
    close("dw", dw, ref.dw, ref.tol_dw, F32)
    close("dx", dx[~gone], ref.dx, ref.tol_dx, F32)


@pytest.mark.parametrize("t", [12, 140])
def test_one_token_far_larger_than_the_others(t):
    """Loss, lse and dx of a token go by its own row."""
    v, d = 200, 40
    x, w, y, b = inputs(t, v, d, F32, True, seed=44, ignored=0.0)
    x[5] *= 1e12
    rest = torch.arange(t, device=DEV) != 5
    loss, lse, dx, _, _ = T.cross_entropy_train(x, w, y, b, reduction="sum")
    check(Reference(x[rest], w, y[rest], b), loss[rest], lse[rest], dx[rest])
    check(Reference(x[5:6], w, y[5:6], b), loss[5:6], lse[5:6])


def half_step(want, dtype):
    """Half of the distance between the type's numbers around a value."""
    bits = {BF16: 8, F16: 11, F32: 24}[dtype]
    return torch.exp2(torch.floor(torch.log2(want.abs().clamp(min=1e-30))) - bits)


@pytest.mark.parametrize("dtype", [BF16, F16])
def test_bias_gradient_of_many_blocks(dtype):
    """Eight blocks of 4096 tokens: dbias is rounded once, at the end (what comes
    before: E's 2^-11 of every probability, sums of 32768 in fp32)."""
    t, v, d = 8 * 4096, 1 << 17, 8
    g = torch.Generator(device=DEV)
    g.manual_seed(45)
    x = torch.randn(t, d, generator=g, device=DEV).to(dtype)
    w = torch.randn(v, d, generator=g, device=DEV).to(dtype) * 0.5
    b = torch.randn(v, generator=g, device=DEV).to(dtype)
    y = torch.randint(0, 64, (t,), generator=g, device=DEV)
    scale = 1024.0 if dtype == BF16 else 64.0  # (512 hits of a target, times 1024, are no fp16 number)
    old = (torch.randn(v, generator=g, device=DEV) * 300).to(dtype)
    say(f"[xent] eight blocks {dtype}")
    _, lse, _, _, db = T.cross_entropy_train(x, w, y, b, reduction="sum", scale=scale, need_dx=False, need_dw=False)
    more = old.clone()
    T.cross_entropy_train(x, w, y, b, reduction="sum", scale=scale, need_dx=False, need_dw=False, dbias=more, accumulate=True)
    total = torch.zeros(v, dtype=torch.float64, device=DEV)
    for a in range(0, t, 1024):
        l = x[a:a + 1024].double() @ w.double().t() + b.double()
        total += torch.softmax(l, 1).sum(0)
    hits = torch.bincount(y, minlength=v).double()
    want = scale * (total - hits)
    # (logits of at most 30, in error by 20 u of the sizes that add up to them)
    tol = scale * (total * (2.0 ** -11 + 2.0 ** -16) + hits * 2.0 ** -16 + 2.0 ** -24)
    got = db.double()
    assert ((got - want).abs() <= tol + half_step(want, dtype) * 1.0001).all()
    want = want + old.double()
    assert ((more.double() - want).abs() <= tol + half_step(want, dtype) * 1.0001).all()


def test_bias_gradient_whose_blocks_cancel():
    """fp16: a partial sum beyond the type's range whose total is within it."""
    t, v, d = 4096, 1 << 17, 8
    x = torch.zeros(2 * t, d, dtype=F16, device=DEV)
    w = torch.zeros(v, d, dtype=F16, device=DEV)
    b = torch.zeros(v, dtype=F16, device=DEV)
    b[7] = 12.0
    y = torch.full((2 * t,), 9, device=DEV)
    u = torch.ones(2 * t, device=DEV) * 64.0
    u[t:] *= -1
    db = T.cross_entropy_train(x, w, y, b, weights=u, reduction="sum", need_dx=False, need_dw=False)[4]
    assert not db.any()


@pytest.mark.parametrize("dtype,scale", [(BF16, 1.0), (F32, 1.0), (F16, 1e-28)])
@pytest.mark.parametrize("t", [12, 70])
def test_weights_very_far_apart(t, dtype, scale):
    """The smallest weight 2^-200 of the largest."""
    v, d = 150, 24
    x, w, y, b = inputs(t, v, d, dtype, True, seed=46, ignored=0.2)
    u = torch.ones(t, device=DEV)
    u[0::4], u[1::4], u[2::4] = 1e30, -1e-30, 1e-5
    say(f"[xent] weights far apart {t} {dtype}")
    loss, lse, dx, dw, db = T.cross_entropy_train(x, w, y, b, weights=u, reduction="sum", scale=scale,
                                                  dw=torch.zeros(v, d, device=DEV))
    check(Reference(x, w, y, b, u, scale), loss, lse, dx, dw, db)


def test_factors_beyond_fp32():
    """The powers of two of G and w together are no fp32 number, dx is one.  (G: 2^-25 of
    a third; w: 2^-39 of 2^-16 of its largest; p 4.5e-5 to 2^-18: 2^-16 in all.)"""
    t, v, d = 40, 64, 16
    x = torch.zeros(t, d, device=DEV)
    x[:, 0] = 2.0 ** -60
    w = torch.zeros(v, d, device=DEV)
    w[:, 0], w[5, 1] = 2.0 ** 60, 2.0 ** 44
    b = torch.full((v,), -10.0, device=DEV)
    b[3] = 0.0
    y = torch.full((t,), 3, device=DEV)
    u = torch.full((t,), 2.0 ** 97, device=DEV)
    dx, dw = T.cross_entropy_train(x, w, y, b, weights=u, reduction="sum")[2:4]
    p = float(np.exp(-10.0) / (1 + 63 * np.exp(-10.0)))
    want = torch.full((t,), 2.0 ** (97 + 44) * p, dtype=torch.float64, device=DEV)
    close("dx", dx[:, 1], want, want * 2.0 ** -16)
    assert not dx[:, 2:].any()
    want = torch.full((60,), t * 2.0 ** (97 - 60) * p, dtype=torch.float64, device=DEV)
    close("dw", dw[4:, 0], want, want * 2.0 ** -16)


@pytest.mark.parametrize("t", [4, 100])
@pytest.mark.parametrize("dtype", [BF16, F16])
def test_small_probabilities_of_16_bit_tensors(t, dtype):
    """20 nats under a segment's largest, 2e-9: E holds it with its 11 bits, and the
    gradient's own type is what it is rounded to (fp16: half a step of 2^-24 under a
    row's weight at 2^13)."""
    v, d = 64, 8
    w = torch.zeros(v, d, dtype=dtype, device=DEV)
    w[1:, 0] = -20.0
    x = torch.zeros(t, d, dtype=dtype, device=DEV)
    x[:, 0] = 1.0
    y = torch.zeros(t, dtype=torch.int64, device=DEV)
    dw = T.cross_entropy_train(x, w, y, reduction="sum", dw=torch.zeros(v, d, device=DEV))[3]
    p = np.exp(-20.0) / (1 + 63 * np.exp(-20.0))
    want = torch.full((v - 1,), t * p, dtype=torch.float64, device=DEV)
    tol = want * (2.0 ** -11 + (2.0 ** -8 if dtype == BF16 else 0.0) + 2.0 ** -18) + (t * 2.0 ** -25 * 2.0 ** -13 if dtype == F16 else 0.0)
    close("dw", dw[1:, 0], want, tol)


@pytest.mark.parametrize("t", [9, 90])
def test_words_without_a_place_may_hold_anything(t):
    """fp32: a bias of -infinity takes a word out, whatever finite values its row of
    weights holds (a vocabulary's unused end)."""
    v, d = 300, 24
    x, w, y, b = inputs(t, v, d, F32, True, seed=47, ignored=0.1)
    y.clamp_(max=279)
    live = torch.arange(v, device=DEV) < 280
    b[~live] = -float("inf")
    for size in (1e12, 1e30):
        big = w.clone()
        big[~live] = size
        big[~live, ::2] *= -1
        loss, lse, dx, dw, db = T.cross_entropy_train(x, big, y, b)
        check(Reference(x, w[live], y, b[live], mean=True), loss, lse, dx, dw[live], db[live])
        assert not dw[~live].any() and not db[~live].any()


def test_tokens_beyond_2_24():
    """More tokens than one launch has workgroups for."""
    t, v, d = (1 << 24) + 777, 5, 8
    g = torch.Generator(device=DEV)
    g.manual_seed(48)
    x = torch.randn(t, d, generator=g, device=DEV).to(BF16)
    w = torch.randn(v, d, generator=g, device=DEV).to(BF16)
    y = torch.full((t,), -100, device=DEV)
    at = torch.cat([torch.arange(0, t, 4099, device=DEV), torch.arange(t - 500, t, device=DEV)]).unique()
    y[at] = torch.randint(0, v, (len(at),), generator=g, device=DEV)
    say("[xent] 2^24 tokens and some")
    loss, lse = T.cross_entropy(x, w, y)
    ref = Reference(x[at], w, y[at], mean=True)
    check(ref, loss[at], lse[at])
    assert int((loss != 0).sum()) == len(at) and torch.isfinite(lse).all()
    loss2, lse2, dx, dw, _ = T.cross_entropy_train(x, w, y, dw=torch.zeros(v, d, device=DEV))
    check(ref, loss2[at], lse2[at], dx[at], dw)
    assert torch.equal(loss, loss2) and torch.equal(lse, lse2)


def test_operands_beyond_2_31_threads():
    """Rows whose copy, eight values a thread, is more than one launch holds."""
    t, v = (1 << 28) + 1001, 3
    x = (torch.arange(t, device=DEV, dtype=torch.int32) % 251).to(BF16).view(t, 1) / 64
    w = torch.tensor([[0.5], [-1.0], [2.0]], dtype=BF16, device=DEV)
    y = torch.full((t,), -100, device=DEV)
    at = torch.cat([torch.arange(0, t, 65537, device=DEV), torch.arange(t - 500, t, device=DEV),
                    torch.arange(t // 2 - 300, t // 2 + 300, device=DEV)]).unique()
    y[at] = at % v
    say("[xent] 2^28 tokens of one value")
    loss, lse = T.cross_entropy(x, w, y)
    check(Reference(x[at], w, y[at]), loss[at], lse[at])
    assert torch.equal(lse[:251].repeat(4), lse[251 * 1000000:251 * 1000004])


@pytest.mark.parametrize("dtype", [BF16, F16, F32])
def test_only_what_is_wanted_under_weights(dtype):
    t, v, d = 75, 130, 40
    x, w, y, b = inputs(t, v, d, dtype, True, seed=49)
    u = torch.logspace(-5, 5, t, device=DEV)
    full = T.cross_entropy_train(x, w, y, b, weights=u)
    for need in ((True, False, False), (False, True, False), (False, False, True), (True, False, True)):
        got = T.cross_entropy_train(x, w, y, b, weights=u, need_dx=need[0], need_dw=need[1], need_dbias=need[2])
        for n, a, c in zip((True, True) + need, got, full):
            assert (a is not None) == n and (not n or torch.equal(a, c))


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_backward_multiplies_in_place_of_fp32_copies(dtype):
    """One product in fp32 and one rounding; beside the gradients themselves the
    backward pass takes no memory of their size."""
    x, w, y, b = inputs(64, 8192, 1024, dtype, True, seed=50)
    want = T.cross_entropy_train(x, w, y, b)[2:]
    for up in (1.0, 0.3, -1e-30, float("inf")):
        leaves = [v.clone().requires_grad_(True) for v in (x, w, b)]
        out = T.linear_cross_entropy(leaves[0], leaves[1], y, leaves[2])
        torch.cuda.synchronize()
        torch.cuda.reset_peak_memory_stats()
        before = torch.cuda.memory_allocated()
        out.backward(torch.tensor(up, device=DEV), retain_graph=True)
        extra = torch.cuda.max_memory_allocated() - before
        assert extra <= sum(v.numel() * v.element_size() for v in leaves) + (1 << 20)
        for leaf, g in zip(leaves, want):
            assert torch.equal(leaf.grad.nan_to_num(7.0), (g.float() * up).to(dtype).nan_to_num(7.0))
        out.backward(torch.tensor(up, device=DEV))  # (again, from the same saved gradients)
        for leaf, g in zip(leaves, want):
            one = (g.float() * up).to(dtype)
            assert torch.equal(leaf.grad.nan_to_num(7.0), (one + one).nan_to_num(7.0))


@pytest.mark.parametrize("dtype", [BF16, F16, F32])
def test_scale_of_any_length_and_address(dtype):
    """Half a step of the type, and what the product's rounding to fp32 may add where it
    brings it to a tie (the compiler rounds some products to fp16 at once, some so)."""
    flat = torch.randn(5000, device=DEV).to(dtype)
    f = torch.tensor([3.0, -0.7], device=DEV)[1:]
    half = torch.finfo(dtype).eps / 2 + 2.0 ** -23
    for at, n, to in ((0, 0, 0), (0, 1, 0), (1, 7, 0), (8, 4096, 16), (3, 4097, 3), (0, 5000, 0)):
        out = torch.full((5100,), 9.0, dtype=dtype, device=DEV)
        v, o = flat[at:at + n], out[to:to + n]
        X._call(DEV, B.psgd_xent_scale, v.data_ptr(), X._dtype(v), n, f.data_ptr(), o.data_ptr())
        want = v.double() * f.double()
        assert ((o.double() - want).abs() <= half * want.abs() + (2.0 ** -25 if dtype == F16 else 0.0)).all()
        assert (out[:to] == 9.0).all() and (out[to + n:] == 9.0).all()
        v = v.clone()
        X._call(DEV, B.psgd_xent_scale, v.data_ptr(), X._dtype(v), n, f.data_ptr(), v.data_ptr())
        assert ((v.double() - want).abs() <= half * want.abs() + (2.0 ** -25 if dtype == F16 else 0.0)).all()


@pytest.mark.parametrize("t", [0, 1, 63, 1025, 65536, 65537, 300003])
def test_total(t):
    """fp64 sums of the losses as they are, rounded once."""
    g = torch.Generator(device=DEV)
    g.manual_seed(51)
    loss = torch.rand(t, generator=g, device=DEV) * 20
    y = torch.randint(-2, 6, (t,), generator=g, device=DEV)
    n = int(((y >= 0) & (y != 4)).sum())
    want = float(loss.double().sum())
    for mean, value in ((True, want / max(1, n)), (False, want)):
        got = X._total(loss, y, mean, 4)
        assert got.shape == () and abs(float(got) - value) <= (2.0 ** -24 + t * 2.0 ** -53) * abs(value)
    if t > 1:
        assert torch.equal(X._total(loss, y.repeat_interleave(2)[::2], True, 4), X._total(loss, y, True, 4))
        loss[t // 2] = float("nan")
        assert torch.isnan(X._total(loss, y, False, 4))


@pytest.mark.parametrize("low", [BF16, F16])
def test_autocast(low):
    """Under autocast the inputs are taken in its type, as by a linear layer: 16-bit
    hidden states with a float32 head, gradients in each input's own type."""
    x, w, y, b = inputs(60, 140, 40, F32, True, seed=52)
    leaves = [x.to(low).requires_grad_(True), w.clone().requires_grad_(True), b.clone().requires_grad_(True)]
    with torch.autocast("cuda", dtype=low):
        out = T.linear_cross_entropy(leaves[0], leaves[1], y, leaves[2])
    out.backward()
    same = [v.detach().to(low).requires_grad_(True) for v in leaves]
    want = T.linear_cross_entropy(same[0], same[1], y, same[2])
    want.backward()
    assert torch.equal(out, want)
    for a, c in zip(leaves, same):
        assert a.grad.dtype == a.dtype and torch.equal(a.grad, c.grad.to(a.dtype))
    with torch.autocast("cuda", enabled=False), pytest.raises(ValueError):
        T.linear_cross_entropy(leaves[0], leaves[1], y)


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("t", [1, 2, 15, 16, 17, 32])
@pytest.mark.parametrize("v,d", [(300, 40), (1000, 650), (90, 64), (70, 50001), (66, 49160)])
def test_gradients_of_few_tokens_are_rounded_once(t, v, d, dtype):
    """Up to 32 tokens of a 16-bit type: half a step of dx, dw and dbias, and before it
    fp32's roundings and G's as two values of the type (bf16 2^-16; fp16 2^-21, and
    2^-38 of the token's weight)."""
    x, w, y, b = inputs(t, v, d, dtype, True, seed=53, ignored=0.0)
    u = torch.linspace(0.3, 3.0, t, device=DEV)
    xd, wd = x.double(), w.double()
    l = xd @ wd.t() + b.double()
    size = xd.abs() @ wd.abs().t() + b.double().abs()
    p = torch.softmax(l, 1)
    g = u.double()[:, None] * (p - torch.nn.functional.one_hot(y, v))
    dl = ((d / 16 + 16) * U) * size
    e = u.double()[:, None] * p * (dl + dl.max(1, keepdim=True).values + 2.0 ** -18)
    e = e + g.abs() * (2.0 ** -16 if dtype == BF16 else 2.0 ** -21) + (u.double()[:, None] * 2.0 ** -38 if dtype == F16 else 0.0)
    # (dw: a token's row of x under its weight's power of two, up to 2^-4 here, in fp16)
    small = 2.0 ** -25 * 16 * float(u.max()) * t if dtype == F16 else 0.0
    say(f"[xent] {t} tokens once rounded, {v} x {d} {dtype}")
    for weights in (u, None):
        if weights is None:
            g, e, small = g / u.double()[:, None], e / u.double()[:, None], 0.0
        dx, dw, db = T.cross_entropy_train(x, w, y, b, weights=weights, reduction="sum")[2:]
        many = (v / 16 + 160) * U
        for name, got, want, tol in (("dx", dx, g @ wd, e @ wd.abs() + many * (g.abs() @ wd.abs())),
                                     ("dw", dw, g.t() @ xd, e.t() @ xd.abs() + many * (g.abs().t() @ xd.abs()) + small),
                                     ("db", db, g.sum(0), e.sum(0) + many * g.abs().sum(0))):
            close(name, got, want, tol + half_step(want.abs() + tol, dtype) + (2.0 ** -25 if dtype == F16 else 0.0))
        half = T.cross_entropy_train(x, w, y, b, weights=weights, reduction="sum", dw=torch.ones(v, d, device=DEV), accumulate=True,
                                     dbias=torch.zeros_like(b))[3]
        close("dw on top", half, 1 + g.t() @ xd, e.t() @ xd.abs() + many * (g.abs().t() @ xd.abs()) + small + 2.0 ** -23)


@pytest.mark.parametrize("t", [6, 60])
@pytest.mark.parametrize("dtype", [BF16, F16, F32])
def test_an_infinite_logit_is_not_a_number(t, dtype):
    """exp(inf - inf): the token's loss, lse and gradients, and no other token's loss."""
    x, w, y, b = inputs(t, 100, 24, dtype, True, seed=54, ignored=0.0)
    x[3, 5] = float("inf")
    w[:, 5] = w[:, 5].abs() + 0.25
    loss, lse, dx, _, _ = T.cross_entropy_train(x, w, y, b)
    others = torch.arange(t, device=DEV) != 3
    assert torch.isnan(loss[3]) and torch.isnan(lse[3]) and torch.isnan(dx[3]).all()
    check(Reference(x[others], w, y[others], b), loss[others], lse[others])
    assert torch.isfinite(dx[others]).all()
    b[9] = float("inf")
    loss, lse = T.cross_entropy(x, w, y, b)
    assert torch.isnan(loss).all() and torch.isnan(lse).all()


@pytest.mark.parametrize("dtype,t", [(F16, 20), (F16, 90), (BF16, 5), (F32, 40)])
@pytest.mark.parametrize("reduction", ["none", "mean"])
def test_autograd_of_every_kind_captured(dtype, t, reduction):
    """Loss and gradients in a graph, replayed between eager work on other inputs."""
    x, w, y, b = inputs(t, 210, 40, dtype, True, seed=55)
    up = torch.linspace(0.1, 2.0, t, device=DEV) if reduction == "none" else torch.tensor(0.7, device=DEV)

    def step(*leaves):
        out = T.linear_cross_entropy(leaves[0], leaves[1], y, leaves[2], reduction=reduction)
        return (out.detach(),) + torch.autograd.grad(out, leaves, up)

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
        for name, a, e in zip(("loss", "dx", "dw", "db"), got, want):
            assert torch.equal(a, e), (name, k)

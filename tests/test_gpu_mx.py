"""Microscaled 4-bit operands on the GPU against the float64 oracle: codes and
scales bit for bit, products within a bound derived from the sums' lengths.

Tolerance of a product: the 4-bit values' products are exact and summed in
fp32, at most 64 to a matrix-core step, so an entry's error is at most
(steps + partial sums + a few) * 2^-24 * sum |a||b|; BOUND(k) = (k / 16 + 32)
* 2^-24 leaves four roundings for every step of 64.  Results of 16 bits add one
rounding: 2^-8 (bfloat16) or 2^-11 (float16) of the entry, at least the type's
smallest step.
"""
import warnings

import numpy as np
import pytest

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a GPU", allow_module_level=True)

from gpu_util import say  # noqa: E402
from oracle import microscaling as MX  # noqa: E402
from rank_gradient_compression_amd import binding as B  # noqa: E402
from rank_gradient_compression_amd import torch_api as T  # noqa: E402

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16
HALF_STEP = {F32: 0.0, BF16: 2.0 ** -8, F16: 2.0 ** -11}


def matrix(rows, cols, dtype, seed=0):
    """Rows of different scales, a few entries far out, a zero block, -0."""
    g = np.random.default_rng([seed, rows, cols])
    x = g.standard_normal((rows, cols)) * np.exp(g.standard_normal((rows, 1)))
    x[g.random((rows, cols)) < 0.01] *= 30.0
    x[0, : min(cols, 40)] = 0.0
    x[-1, -1] = -0.0
    return torch.from_numpy(x).to(dtype).to(DEV)


def rand_bytes(rows, cols, seed=0):
    g = np.random.default_rng([7, seed, rows, cols])
    return torch.from_numpy(g.integers(0, 256, (rows, cols), dtype=np.uint8)).to(DEV)


def f64(t):
    return t.detach().cpu().double().numpy()


def check_operand(q, x64, rand=None, what=""):
    codes, scales = MX.quantize(x64, rand)
    rows, cols = x64.shape
    assert q.shape == (rows, cols)
    got = q.codes.cpu().numpy()
    assert np.array_equal(got, MX.pack_codes(codes)), f"{what}: codes differ"
    want, known = MX.pack_scales(scales, cols)
    s = q.scales.cpu().numpy()
    assert s.size == want.size and np.array_equal(s[known], want[known]), f"{what}: scales differ"


SHAPES = [(1, 1), (1, 31), (2, 32), (3, 33), (31, 255), (32, 256), (33, 257), (129, 127), (128, 128), (130, 650), (4, 1100),
          (300, 5)]


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("stochastic", [False, True])
def test_quantize_bit_for_bit(dtype, stochastic):
    for rows, cols in SHAPES:
        say(f"[mx] quantize {rows}x{cols} {dtype} stochastic={stochastic}")
        x = matrix(rows, cols, dtype)
        r = rand_bytes(rows, cols) if stochastic else None
        rn = None if r is None else r.cpu().numpy()
        v = torch.full_like(x, 7.0)
        check_operand(T.mx_quantize(x, rand=r, values=v), f64(x), rn, "rows")
        assert np.array_equal(f64(v), MX.round_values(f64(x), rn)), "values differ"
        a, t = T.mx_quantize_both(x, rand=r)
        check_operand(a, f64(x), rn, "both, rows")
        check_operand(t, f64(x).T, None if rn is None else rn.T, "both, columns")
        check_operand(T.mx_quantize_t(x, rand=r), f64(x).T, None if rn is None else rn.T, "columns")
        assert torch.equal(T.mx_dequantize(a, dtype=F32).double().cpu(), torch.from_numpy(MX.round_values(f64(x), rn)))


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_every_width_of_a_last_tile(dtype):
    for cols in [*range(1, 40), *range(250, 272)]:
        x, r = matrix(3, cols, dtype, seed=21), rand_bytes(3, cols)
        rn = r.cpu().numpy()
        say(f"[mx] width {cols} {dtype}")
        v = x.clone()
        check_operand(T.mx_quantize(v, rand=r, values=v), f64(x), rn, "rows, in place")
        assert np.array_equal(f64(v), MX.round_values(f64(x), rn)), "values differ"
        check_operand(T.mx_quantize_t(x, rand=r), f64(x).T, rn.T, "columns")


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_strided_and_unaligned_rows(dtype):
    for off, ld in [(0, 700), (1, 701), (3, 650 + 3), (2, 652)]:
        rows, cols = 37, 649
        buf = torch.zeros(off + rows * ld + 8, dtype=dtype, device=DEV)
        x = buf[off:off + rows * ld].view(rows, ld)[:, :cols]
        x.copy_(matrix(rows, cols, dtype, seed=ld))
        say(f"[mx] strided {dtype} offset {off} stride {ld}")
        a, t = T.mx_quantize_both(x)
        check_operand(a, f64(x))
        check_operand(t, f64(x).T)
        out = torch.zeros_like(buf)
        v = out[off:off + rows * ld].view(rows, ld)[:, :cols]
        check_operand(T.mx_quantize(x, values=v), f64(x))
        assert np.array_equal(f64(v), MX.round_values(f64(x)))
        assert float(out[off:off + rows * ld].view(rows, ld)[:, cols:].abs().sum()) == 0.0, "wrote past the rows"
        T.mx_dequantize(a, out=v.zero_())
        assert np.array_equal(f64(v), MX.round_values(f64(x)))
        want = MX.round_values(f64(x))
        T.mx_quantize(x, values=x)  # in place
        assert np.array_equal(f64(x), want)


def test_edge_values():
    tiny, big = 2.0 ** -149, float(np.finfo(np.float32).max)
    rows = []
    for top in (6.0, np.nextafter(np.float32(6), np.float32(7)), 3.0, np.nextafter(np.float32(3), np.float32(4)), 1.0,
                tiny, 6 * 2.0 ** -127, 7 * 2.0 ** -127, big, big / 2):
        r = np.zeros(64, np.float32)
        r[:7] = np.float32(top) * np.array([1, -0.9, 0.5, 0.25, -0.125, 0.04, 0.0], np.float32)
        r[32:36] = [tiny, -tiny, 2.0 ** -130, 0.0]
        rows.append(r)
    x = torch.from_numpy(np.stack(rows)).to(DEV)
    for col in (False, True):
        v = x.t().contiguous() if col else x
        a, t = T.mx_quantize_both(v)
        check_operand(a, f64(v))
        check_operand(t, f64(v).T)
    w = torch.empty_like(x)
    T.mx_quantize(x, values=w)
    # (the largest fp32 value and -0.9 of it round to +-2^128, infinite in fp32)
    with np.errstate(over="ignore"):
        want = MX.round_values(f64(x)).astype(np.float32)
    assert np.isinf(want).sum() == 2 and np.array_equal(w.cpu().numpy(), want)


def test_infinities_and_nan_stay_in_their_blocks():
    x = matrix(70, 300, F32)
    x[3, 5], x[40, 299], x[69, 64] = float("inf"), float("nan"), float("-inf")
    a, t = T.mx_quantize_both(x)
    check_operand(a, f64(x))
    check_operand(t, f64(x).T)
    v = torch.empty_like(x)
    T.mx_quantize(x, values=v)
    want = MX.round_values(f64(x))
    assert np.array_equal(f64(v), want, equal_nan=True)
    # a product's rows with such a block are NaN, the others are not touched
    b = T.mx_quantize(matrix(50, 300, F32, seed=3))
    c = f64(T.mx_product(a, b))
    bad = np.isnan(want).any(axis=1)
    assert np.isnan(c[bad]).all() and np.isfinite(c[~bad]).all()


def within(got, want, tol, dtype):
    """Entries within tol; float16 entries beyond its range are infinite (its
    largest value is 65504, and 65520 is the first that rounds up)."""
    ok = np.abs(got - want) <= tol
    if dtype == F16:
        ok |= (np.abs(want) + tol >= 65520) & np.isinf(got) & (np.sign(got) == np.sign(want))
    return bool(np.all(ok))


def product_bound(a64, b64, dtype):
    k = a64.shape[1]
    want = a64 @ b64.T
    return want, (k / 16 + 32) * 2.0 ** -24 * (np.abs(a64) @ np.abs(b64).T) + HALF_STEP[dtype] * np.abs(want) + 1e-300


# every way the product is computed: few rows on either side, small tiles that
# share the summed axis, the three large tiles, a single chunk of columns
PRODUCTS = [(1, 1, 1), (1, 33, 300), (5, 70, 4096), (24, 500, 2600), (33, 129, 513), (64, 257, 1024), (100, 90, 2049),
            (128, 1000, 257), (300, 20, 700), (1000, 1, 640), (200, 200, 256), (161, 130, 64), (257, 260, 1000),
            (130, 4000, 290), (700, 650, 2600), (1100, 1300, 300), (1030, 2100, 520), (4100, 2050, 770), (650, 33278, 4)]


@pytest.mark.parametrize("m,n,k", PRODUCTS)
def test_product(m, n, k):
    x, w = matrix(m, k, F32, seed=1), matrix(n, k, F32, seed=2)
    a, b = T.mx_quantize(x), T.mx_quantize(w)
    a64, b64 = f64(T.mx_dequantize(a)), f64(T.mx_dequantize(b))
    for dtype in (F32, BF16, F16):
        say(f"[mx] product {m}x{n}x{k} {dtype}")
        want, tol = product_bound(a64, b64, dtype)
        c = T.mx_product(a, b, dtype=dtype)
        assert within(f64(c), want, tol, dtype), (m, n, k, dtype, float(np.max(np.abs(f64(c) - want) / tol)))
        assert torch.equal(T.mx_product(a, b, dtype=dtype), c), "a repeated call differs"
        # accumulation, into a strided, unaligned matrix whose neighbours stay
        for off, ld in [(0, n + 8 - n % 8), (1, n + 3)]:
            buf = torch.full((off + m * ld + 8,), 0.5, dtype=dtype, device=DEV)
            out = buf[off:off + m * ld].view(m, ld)
            T.mx_product(a, b, out=out[:, :n], accumulate=True)
            got = f64(out[:, :n])
            assert within(got, want + 0.5, tol + HALF_STEP[dtype] * (np.abs(want) + 0.5) + 2.0 ** -24, dtype)
            assert bool((out[:, n:] == 0.5).all()) and bool((buf[:off] == 0.5).all())
            T.mx_product(a, b, out=out[:, :n])
            assert torch.equal(out[:, :n], c), "a strided result differs"
            assert bool((out[:, n:] == 0.5).all()) and bool((buf[off + m * ld:] == 0.5).all())


def test_product_without_columns_or_rows():
    e = lambda r, c: T.mx_quantize(torch.zeros(r, c, device=DEV))  # noqa: E731
    c = T.mx_product(e(5, 0), e(7, 0), out=torch.full((5, 7), 3.0, device=DEV))
    assert float(c.abs().sum()) == 0.0
    c = T.mx_product(e(5, 0), e(7, 0), out=torch.full((5, 7), 3.0, device=DEV), accumulate=True)
    assert bool((c == 3.0).all())
    assert T.mx_product(e(0, 64), e(7, 64)).shape == (0, 7)
    assert T.mx_linear(torch.zeros(0, 64, device=DEV), e(7, 64)).shape == (0, 7)
    assert float(T.mx_linear(torch.zeros(3, 0, device=DEV), e(7, 0)).abs().sum()) == 0.0


def test_product_of_extreme_scales():
    # 2^-120 against 2^120: every block's scales cancel
    for m, n, k in [(3, 40, 300), (200, 140, 300), (300, 300, 600)]:
        x, w = matrix(m, k, F32, seed=4).clamp(-8, 8), matrix(n, k, F32, seed=5).clamp(-8, 8)
        c = T.mx_product(T.mx_quantize(x), T.mx_quantize(w))
        d = T.mx_product(T.mx_quantize(x * 2.0 ** -110), T.mx_quantize(w * 2.0 ** 110))
        assert torch.equal(c, d)


def test_padding_is_never_read_as_data():
    # operands whose memory around the used bytes holds NaN scales and codes
    m, n, k = 70, 45, 290
    x, w = matrix(m, k, F32, seed=6), matrix(n, k, F32, seed=7)
    want = T.mx_product(T.mx_quantize(x), T.mx_quantize(w))

    def dirty(src, rows):
        cb, sb = B.psgd_mx_sizes(rows, k)
        big = torch.full((cb + sb + 4096,), 255, dtype=torch.uint8, device=DEV)
        base = (cb + 255) // 256 * 256 + 512
        q = T.MxTensor(rows, k, DEV)
        q.buf, q.codes_ptr, q.scales_ptr = big, big.data_ptr() + 256, big.data_ptr() + base
        B.psgd_mx_quantize(src.data_ptr(), B.PSGD_DTYPE_F32, rows, k, k, 0, q.codes_ptr, q.scales_ptr, 0, 0, 0, 0,
                           torch.cuda.current_stream().cuda_stream)
        return q

    assert torch.equal(T.mx_product(dirty(x, m), dirty(w, n)), want)


@pytest.mark.parametrize("m,n,k", [(1, 500, 4096), (3, 77, 650), (4, 100, 8000), (16, 64, 300), (24, 96, 1100), (40, 64, 333),
                                   (300, 200, 650), (7, 1, 32), (32, 40, 2500), (28, 33, 4000), (9, 8300, 2600)])
@pytest.mark.parametrize("dtype", [F32, BF16, F16])
def test_linear(m, n, k, dtype):
    x, w = matrix(m, k, dtype, seed=8), matrix(n, k, dtype, seed=9)
    wq = T.mx_quantize(w)
    a64, b64 = MX.round_values(f64(x)), MX.round_values(f64(w))
    for out in (F32, dtype):
        want, tol = product_bound(a64, b64, out)
        say(f"[mx] linear {m}x{n}x{k} {dtype} -> {out}")
        y = T.mx_linear(x, wq, dtype=out)
        assert y.dtype == out and within(f64(y), want, tol, out)
    ld = k + 5
    xs = torch.zeros(m * ld + 1, dtype=dtype, device=DEV)[1:].view(m, ld)[:, :k]
    xs.copy_(x)
    assert torch.equal(T.mx_linear(xs, wq, dtype=dtype), y), "strided activations differ"


@pytest.mark.parametrize("m,k,n", [(40, 65, 33), (300, 130, 257)])
@pytest.mark.parametrize("stochastic", [False, True])
def test_linear_gradients(m, k, n, stochastic):
    x, w, dy = matrix(m, k, F32, 1), matrix(n, k, F32, 2), matrix(m, n, F32, 3)
    rand = rand_bytes(m, n) if stochastic else None
    rn = None if rand is None else rand.cpu().numpy()
    y, saved = T.mx_linear_forward(x, w)
    dx, dw = T.mx_linear_backward(dy, saved, rand=rand)
    q = MX.round_values
    xr, wr, xt, wt = q(f64(x)), q(f64(w)), q(f64(x).T), q(f64(w).T)
    dyr, dyt = q(f64(dy), rn), q(f64(dy).T, None if rn is None else rn.T)
    for got, a64, b64 in ((y, xr, wr), (dx, dyr, wt), (dw, dyt, xt)):
        want, tol = product_bound(a64, b64, F32)
        assert np.all(np.abs(f64(got) - want) <= tol)
    # against differences: y is linear in the rounded operands, so for the
    # gradient of <dy, y> a change of one rounded entry by h moves it by h times
    # the formula's gradient, exactly up to fp64 rounding
    loss = lambda a, b: float(np.sum(dyr * (a @ b.T)))  # noqa: E731
    g = np.random.default_rng(5)
    wrong_axis = q(f64(w))
    for _ in range(5):
        i, j = int(g.integers(m)), int(g.integers(k))
        a = wt.T.copy()  # the weights that dx's formula uses
        hi, lo = xr.copy(), xr.copy()
        hi[i, j] += 0.5
        lo[i, j] -= 0.5
        diff = loss(hi, a) - loss(lo, a)
        assert abs(diff - f64(dx)[i, j]) <= 1e-4 * np.sum(np.abs(dyr[i]) * np.abs(wt[j])) + 1e-9
    if k > 64:
        assert not np.array_equal(wrong_axis, wt.T)
    # accumulation into a given matrix
    acc = torch.ones(n, k, device=DEV)
    T.mx_linear_backward(dy, saved, rand=rand, dw=acc, accumulate=True)
    want, tol = product_bound(dyt, xt, F32)
    assert np.all(np.abs(f64(acc) - want - 1.0) <= tol + 2.0 ** -23 * (np.abs(want) + 1))


def test_linear_under_autograd():
    x = matrix(6 * 7, 96, BF16, 1).view(6, 7, 96).requires_grad_(True)
    w = matrix(50, 96, F32, 2).to(BF16).requires_grad_(True)
    y = T.mx_linear_train(x, w, stochastic=False)
    dy = matrix(42, 50, BF16, 3).view(6, 7, 50)
    y.backward(dy)
    yy, saved = T.mx_linear_forward(x.detach().reshape(42, 96), w.detach())
    dx, dw = T.mx_linear_backward(dy.reshape(42, 50), saved)
    assert y.shape == (6, 7, 50) and torch.equal(y.detach().reshape(42, 50), yy)
    assert torch.equal(x.grad.reshape(42, 96), dx) and torch.equal(w.grad, dw.to(BF16))


@pytest.mark.parametrize("m,k,n,xd,wd", [(1, 33, 5, F32, F32), (130, 70, 300, BF16, BF16), (70, 257, 129, BF16, F32),
                                         (300, 650, 260, F16, F16)])
@pytest.mark.parametrize("stochastic", [False, True])
def test_training_pass_is_the_single_calls(m, k, n, xd, wd, stochastic):
    """One launch for two matrices, gradients left out, rows with a stride: the
    same bytes as the quantiser and the product called one by one."""
    say(f"[mx] training pass {m}x{k}x{n} {xd} {wd} {stochastic}")
    x, w, dy = matrix(m, k + 3, xd, 1)[:, :k], matrix(n, k, wd, 2), matrix(m, n + 5, xd, 3)[:, 2: n + 2]
    rand = rand_bytes(m, n) if stochastic else None
    y, (xt, wt) = T.mx_linear_forward(x, w)
    dx, dw = T.mx_linear_backward(dy, (xt, wt), rand=rand)
    xr, xt1 = T.mx_quantize_both(x)
    wr, wt1 = T.mx_quantize_both(w)
    dyr, dyt = T.mx_quantize_both(dy, rand)
    for got, want in ((xt, xt1), (wt, wt1)):
        assert torch.equal(T.mx_dequantize(got), T.mx_dequantize(want)) and torch.equal(got.codes, want.codes)
    assert torch.equal(y, T.mx_product(xr, wr, dtype=xd))
    assert torch.equal(dx, T.mx_product(dyr, wt1, dtype=xd))
    assert torch.equal(dw, T.mx_product(dyt, xt1))
    only_x, none = T.mx_linear_backward(dy, (xt, wt), rand=rand, need_dw=False)
    assert none is None and torch.equal(only_x, dx)
    none, only_w = T.mx_linear_backward(dy, (xt, wt), rand=rand, need_dx=False)
    assert none is None and torch.equal(only_w, dw)
    assert T.mx_linear_backward(dy, (xt, wt), need_dx=False, need_dw=False) == (None, None)


@pytest.mark.parametrize("m,k,n", [(0, 5, 7), (5, 0, 7), (5, 7, 0), (0, 0, 0)])
def test_training_pass_of_nothing(m, k, n):
    z = lambda r, c: torch.zeros(r, c, device=DEV)  # noqa: E731
    y, saved = T.mx_linear_forward(z(m, k), z(n, k))
    dx, dw = T.mx_linear_backward(z(m, n), saved, dw=torch.ones(n, k, device=DEV))
    for got, shape in ((y, (m, n)), (dx, (m, k)), (dw, (n, k))):
        assert got.shape == shape and not bool(got.any())


def test_frozen_weights_under_autograd():
    x = matrix(40, 96, BF16, 1).requires_grad_(True)
    w = matrix(50, 96, BF16, 2)
    T.mx_linear_train(x, w, stochastic=False).sum().backward()
    assert w.grad is None and x.grad.shape == x.shape
    x, w = x.detach(), w.requires_grad_(True)
    T.mx_linear_train(x, w, stochastic=False).sum().backward()
    assert x.grad is None and w.grad.shape == w.shape


def test_training_pass_refuses():
    x, w = torch.zeros(4, 64, device=DEV), torch.zeros(8, 64, device=DEV)
    _, saved = T.mx_linear_forward(x, w)
    for bad in (torch.zeros(8, 63, device=DEV), torch.zeros(8, 64), torch.zeros(64, 8, device=DEV).t(), w.double()):
        with pytest.raises(ValueError):
            T.mx_linear_forward(x, bad)
    dy = torch.zeros(4, 8, device=DEV)
    for bad in (dy[:3], torch.zeros(4, 9, device=DEV), dy.cpu(), dy.double()):
        with pytest.raises(ValueError):
            T.mx_linear_backward(bad, saved)
    with pytest.raises(ValueError):
        T.mx_linear_backward(dy, saved, accumulate=True)
    with pytest.raises(ValueError):
        T.mx_linear_backward(dy, saved, dw=torch.zeros(8, 63, device=DEV))
    with pytest.raises(ValueError):
        T.mx_linear_backward(dy, saved, rand=torch.zeros(4, 9, dtype=torch.uint8, device=DEV))


def test_torch_layer_refuses():
    x = torch.zeros(4, 64, device=DEV)
    q = T.mx_quantize(x)
    for bad in (x.double(), x.t(), x[:, ::2], torch.zeros(3, device=DEV), torch.zeros(4, 64), torch.zeros(2, 3, 64, device=DEV)):
        with pytest.raises((ValueError, B.PsgdError)):
            T.mx_quantize(bad)
    for rand in (torch.zeros(4, 64, device=DEV), torch.zeros(4, 63, dtype=torch.uint8, device=DEV),
                 torch.zeros(4, 64, dtype=torch.uint8)):
        with pytest.raises(ValueError):
            T.mx_quantize(x, rand=rand)
    with pytest.raises(ValueError):
        T.mx_quantize(x, values=torch.zeros(4, 63, device=DEV))
    with pytest.raises(ValueError):
        T.mx_product(q, T.mx_quantize(torch.zeros(4, 65, device=DEV)))
    with pytest.raises(ValueError):
        T.mx_product(q, q, accumulate=True)
    with pytest.raises(ValueError):
        T.mx_product(q, q, out=torch.zeros(4, 5, device=DEV))
    with pytest.raises(ValueError):
        T.mx_linear(torch.zeros(2, 63, device=DEV), q)
    with pytest.raises(ValueError):
        T.mx_dequantize(q, out=torch.zeros(4, 63, device=DEV))


def test_another_stream_and_graph_replays():
    x, w, dy = matrix(300, 520, BF16, 1), matrix(400, 520, BF16, 2), matrix(300, 400, BF16, 3)
    wq = T.mx_quantize(w)

    def work():
        y, saved = T.mx_linear_forward(x, w)
        dx, dw = T.mx_linear_backward(dy, saved)
        return [y, dx, dw, T.mx_linear(x[:2], wq), T.mx_linear(x, wq)]

    want = [t.clone() for t in work()]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = work()
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        outs = work()
    for i in range(4):
        x.copy_(matrix(300, 520, BF16, 10 + i))
        eager = [t.clone() for t in work()]
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs, eager)), f"replay {i}"


def test_offsets_beyond_32_bits():
    # 70000 x 65536 bf16: 9.2 GB in, rows past 2^32 bytes of x and past 2^31 codes
    rows, cols = 70000, 65536
    say(f"[mx] quantize {rows}x{cols}")
    x = torch.zeros(rows, cols, dtype=BF16, device=DEV)
    tail = matrix(70, cols, BF16, 11)
    x[-70:] = tail
    q = T.mx_quantize(x)
    want = T.mx_quantize(tail)
    nb = cols // 32 * 16
    assert torch.equal(q.buf[(rows - 70) * nb:rows * nb], want.buf[:70 * nb])
    b = T.mx_quantize(matrix(40, cols, BF16, 12))
    c = T.mx_product(q, b)
    assert torch.equal(c[-70:], T.mx_product(want, b)) and float(c[:-70].abs().sum()) == 0.0
    del x, q, c
    torch.cuda.empty_cache()
    # a result of more than 2^32 bytes
    m, n, k = 40000, 33000, 40
    say(f"[mx] product {m}x{n}x{k}")
    xa, xb = matrix(m, k, F32, 13), matrix(n, k, F32, 14)
    a, b = T.mx_quantize(xa), T.mx_quantize(xb)
    c = T.mx_product(a, b)
    last = T.mx_product(T.mx_quantize(xa[-50:].contiguous()), b)
    assert torch.equal(c[-50:], last)


@pytest.mark.parametrize("rows,cols", [(3, 300), (33, 257), (70, 5), (9, 650)])
def test_equal_inputs_give_equal_bytes_in_place(rows, cols):
    """The whole operand, the scale bytes of rows past the last included."""
    say(f"[mx] bytes in place {rows}x{cols}")
    past = np.ones(-(-rows // 32) * -(-cols // 256) * 256, bool)
    for i in range(rows):
        for b in range(-(-cols // 32)):
            past[MX.scale_index(i, b, cols)] = False
    for dtype in (F32, BF16, F16):
        x = matrix(rows, cols, dtype, seed=31)
        r = rand_bytes(rows, cols)
        want = T.mx_quantize(x, rand=r)
        both, _ = T.mx_quantize_both(x, rand=r)
        v = x.clone()
        got = T.mx_quantize(v, rand=r, values=v)
        for q in (want, both, got):
            assert torch.equal(q.codes, want.codes) and torch.equal(q.scales, want.scales)
            assert not q.scales.cpu().numpy()[past].any(), "scale bytes of rows past the last"


def test_autograd_layer_of_strided_activations_and_weights():
    m, k, n = 40, 96, 50
    base, wb = matrix(m, k, BF16, 1), matrix(n, k, BF16, 2)
    wide, tall = torch.zeros(m, 2 * k, dtype=BF16, device=DEV), torch.zeros(n, 2 * k, dtype=BF16, device=DEV)
    wide[:, ::2], tall[:, ::2] = base, wb
    one = base[:1]
    dy = matrix(n, m, BF16, 3).t()
    for x, w in ((base.t().contiguous().t(), wb), (base, wb.t().contiguous().t()), (wide[:, ::2], tall[:, ::2]),
                 (one.expand(m, k), wb)):
        plain, wp = x.clone(memory_format=torch.contiguous_format), w.clone(memory_format=torch.contiguous_format)
        x, w = x.detach().requires_grad_(True), w.detach().requires_grad_(True)
        y = T.mx_linear_train(x, w, stochastic=False)
        dx, dw = torch.autograd.grad(y, (x, w), dy)
        want, saved = T.mx_linear_forward(plain, wp)
        dx1, dw1 = T.mx_linear_backward(dy.contiguous(), saved)
        assert torch.equal(y.detach(), want) and torch.equal(dx, dx1) and torch.equal(dw, dw1.to(BF16))
    for shape, wshape in (((3, 0, 64), (50, 64)), ((3, 2, 0), (50, 0)), ((3, 2, 64), (0, 64))):
        x, w = torch.ones(shape, device=DEV, requires_grad=True), torch.ones(wshape, device=DEV, requires_grad=True)
        y = T.mx_linear_train(x, w, stochastic=False)
        assert y.shape == (*shape[:-1], wshape[0]) and not bool(y.any())
        y.sum().backward()
        assert x.grad.shape == shape and w.grad.shape == wshape and not bool(x.grad.any()) and not bool(w.grad.any())


def test_autograd_layer_lets_go_of_its_operands():
    x, w = matrix(2048, 1024, BF16, 1).requires_grad_(True), matrix(512, 1024, BF16, 2).requires_grad_(True)
    dy = matrix(2048, 512, BF16, 3)
    T.mx_linear_train(x, w, stochastic=False).backward(dy)
    dx, dw = x.grad.clone(), w.grad.clone()
    x.grad = w.grad = None
    torch.cuda.synchronize()
    before = torch.cuda.memory_allocated()
    y = T.mx_linear_train(x, w, stochastic=False)
    operands = sum(B.psgd_mx_sizes(1024, 2048)) + sum(B.psgd_mx_sizes(1024, 512))
    assert torch.cuda.memory_allocated() - before >= operands + y.numel() * 2
    y.backward(dy)
    x_dx, w_dw, x.grad, w.grad = x.grad, w.grad, None, None
    assert torch.equal(x_dx, dx) and torch.equal(w_dw, dw)
    del x_dx, w_dw
    assert torch.cuda.memory_allocated() - before <= y.numel() * 2 + 4096
    with pytest.raises(RuntimeError, match="second time"):
        y.backward(dy)


def test_linear_warns_where_a_gradient_would_be_lost():
    x, w = matrix(4, 64, BF16, 1), T.mx_quantize(matrix(8, 64, BF16, 2))
    want = T.mx_linear(x, w)
    with pytest.warns(UserWarning, match="mx_linear_train"):
        y = T.mx_linear(x.requires_grad_(True), w)
    assert torch.equal(y, want) and not y.requires_grad
    with warnings.catch_warnings():
        warnings.simplefilter("error")
        with torch.no_grad():
            T.mx_linear(x, w)
        T.mx_linear(x.detach(), w)


def large_tile(m, n, k):
    """Rows and columns of the tile that a product of more than 128 rows on both
    sides and several chunks takes (the library's rule, evaluated here so that
    the shapes below are seen to reach every one of them)."""
    tiles = lambda bm, bn: -(-m // bm) * -(-n // bn)  # noqa: E731
    rounds = lambda bm: -(-tiles(bm, 256) // 256)  # noqa: E731
    assert m > 128 and n > 128 and k > 256
    if tiles(64, 64) <= 256:
        return 64, 64
    if tiles(256, 256) <= 128:
        return 128, 128
    return (192, 256) if 3 * rounds(192) < 4 * rounds(256) else (256, 256)


# both sides off the tile's multiples, a last block that is not full, an odd and
# an even number of chunks of 256
@pytest.mark.parametrize("m,n,k,tile", [(700, 650, 2600, (64, 64)), (1500, 2030, 290, (128, 128)), (4100, 2050, 770, (192, 256)),
                                        (4000, 10900, 290, (256, 256)), (4010, 10999, 570, (256, 256))])
def test_every_large_tile(m, n, k, tile):
    """Sampled rows, and all of the last tile's, against float64; the bytes around the result stay."""
    assert large_tile(m, n, k) == tile
    x, w = matrix(m, k, F32, seed=41), matrix(n, k, F32, seed=42)
    a, b = T.mx_quantize(x), T.mx_quantize(w)
    rows = sorted({0, 15, 16, 63, tile[0] - 1, tile[0], m // 2, *range(m - 1 - (m - 1) % tile[0], m)})
    a64, b64 = f64(T.mx_dequantize(a))[rows], f64(T.mx_dequantize(b))
    for dtype in (F32, BF16, F16):
        say(f"[mx] tile {tile} {m}x{n}x{k} {dtype}")
        want, tol = product_bound(a64, b64, dtype)
        off, ld = 3, n + 5
        buf = torch.full((off + m * ld + 8,), 0.5, dtype=dtype, device=DEV)
        out = buf[off:off + m * ld].view(m, ld)
        T.mx_product(a, b, out=out[:, :n], accumulate=True)
        got = f64(out[rows, :n])
        assert within(got, want + 0.5, tol + HALF_STEP[dtype] * (np.abs(want) + 0.5) + 2.0 ** -24, dtype)
        c = T.mx_product(a, b, dtype=dtype)
        assert within(f64(c[rows]), want, tol, dtype)
        T.mx_product(a, b, out=out[:, :n])
        assert torch.equal(out[:, :n], c), "a strided result differs"
        d = torch.full((m, n), 0.5, dtype=dtype, device=DEV)
        T.mx_product(a, b, out=d, accumulate=True)
        assert within(f64(d[rows]), want + 0.5, tol + HALF_STEP[dtype] * (np.abs(want) + 0.5) + 2.0 ** -24, dtype)
        assert bool((out[:, n:] == 0.5).all()) and bool((buf[:off] == 0.5).all()) and bool((buf[off + m * ld:] == 0.5).all())


def test_stochastic_layer_under_autograd():
    """The default: the incoming gradient's random bytes come from the generator."""
    x, w = matrix(70, 96, BF16, 1), matrix(50, 96, BF16, 2)
    dy = matrix(70, 50, BF16, 3)
    y, saved = T.mx_linear_forward(x, w)
    seeds = []
    for seed in (5, 6):
        g = torch.Generator(device=DEV)
        g.manual_seed(seed)
        rand = torch.randint(0, 256, dy.shape, dtype=torch.uint8, device=DEV, generator=g)
        dx, dw = T.mx_linear_backward(dy, saved, rand=rand)
        # (that pass against the oracle, with the same bytes)
        rn = rand.cpu().numpy()
        for got, a64, b64 in ((dx, MX.round_values(f64(dy), rn), MX.round_values(f64(w).T)),
                              (dw, MX.round_values(f64(dy).T, rn.T), MX.round_values(f64(x).T))):
            want, tol = product_bound(a64, b64, got.dtype)
            assert within(f64(got), want, tol, got.dtype)
        g.manual_seed(seed)
        xl, wl = x.clone().requires_grad_(True), w.clone().requires_grad_(True)
        out = T.mx_linear_train(xl, wl, generator=g)
        assert torch.equal(out.detach(), y)
        out.backward(dy)
        assert torch.equal(xl.grad, dx) and torch.equal(wl.grad, dw.to(BF16))
        seeds.append(dx)
    assert not torch.equal(*seeds)
    torch.manual_seed(9)
    rand = torch.randint(0, 256, dy.shape, dtype=torch.uint8, device=DEV)
    dx, _ = T.mx_linear_backward(dy, saved, rand=rand)
    torch.manual_seed(9)
    xl = x.clone().requires_grad_(True)
    T.mx_linear_train(xl, w).backward(dy)
    assert torch.equal(xl.grad, dx)

"""Orthogonalised updates and the optimiser step around them on the GPU against
the oracle in 64 bits.

Tolerance of an update, relative Frobenius norm, before any run: what the
documented roundings alone do to it in the oracle (newton_schulz_rounded), times
two because the kernel's own choices of powers of two and of the smaller sums'
order move single roundings; what fp32 sums add: plain fp32 steps of the same
matrix differ from 64 bits by about as much (measured in the test, on the CPU,
times four: three products for one); and half a step of the result's type.
An update may leave that by no more than 6 of its root mean square in one entry.
"""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a GPU", allow_module_level=True)

from gpu_util import cpu, say  # noqa: E402
from oracle import ends as E  # noqa: E402
from rank_gradient_compression_amd import binding as B  # noqa: E402
from rank_gradient_compression_amd import torch_api as T  # noqa: E402

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16
HALF = {F32: 2.0 ** -24, BF16: 2.0 ** -8, F16: 2.0 ** -11}
PIECES = {F32: 2, BF16: 1, F16: 2}


def gradient(rows, cols, dtype=F32, seed=0, noise=0.3):
    g = np.random.default_rng([seed, rows, cols])
    k = min(8, rows, cols)
    x = g.standard_normal((rows, k)) / np.arange(1, k + 1) @ g.standard_normal((k, cols))
    x = x / np.linalg.norm(x) + noise * g.standard_normal((rows, cols)) / np.sqrt(rows * cols)
    return torch.from_numpy(x).to(dtype).to(DEV)


def fp32_steps(u, steps=5):
    a, b, c = (np.float32(v) for v in E.COEFFICIENTS)
    x = np.asarray(u, np.float64)
    x = (x / (np.linalg.norm(x) + 1e-7)).astype(np.float32)
    x = x.T if x.shape[0] > x.shape[1] else x
    for _ in range(steps):
        g = x @ x.T
        x = a * x + (b * g + c * (g @ g)) @ x
    return x.T if np.asarray(u).shape[0] > np.asarray(u).shape[1] else x


def norm(x):
    return float(np.linalg.norm(x))


def tolerance(u64, dtype, pieces, exact, steps=5):
    n = norm(exact) or 1.0
    rounded = norm(E.newton_schulz_rounded(u64, pieces, steps) - exact) / n
    sums = norm(fp32_steps(u64, steps) - exact) / n
    return 2 * rounded + 4 * sums + HALF[dtype] + 2.0 ** -22


def check(got, u64, dtype=None, pieces=None, steps=5, what=""):
    dtype = got.dtype if dtype is None else dtype
    exact = E.newton_schulz(u64, steps=steps)
    tol = tolerance(u64, dtype, pieces or PIECES[dtype], exact, steps)
    off = cpu(got) - exact
    rms = norm(exact) / np.sqrt(exact.size)
    say(f"[muon] {what} {exact.shape} {dtype}: off {norm(off) / (norm(exact) or 1.0):.2e}, bound {tol:.2e}")
    assert norm(off) <= tol * norm(exact)
    assert np.abs(off).max() <= 6 * tol * max(rms, np.abs(exact).max() / 6)
    return exact


SHAPES = [(1, 1), (1, 7), (9, 1), (2, 3), (8, 8), (27, 64), (64, 27), (64, 64), (65, 33), (100, 300), (130, 128), (128, 129),
          (257, 256), (300, 650), (650, 300), (512, 64), (31, 2000), (700, 700)]


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("rows,cols", SHAPES)
def test_orthogonalize(rows, cols, dtype):
    x = gradient(rows, cols, dtype)
    say(f"[muon] orthogonalize {rows} x {cols} {dtype}")
    out = T.orthogonalize(x)
    assert out.dtype == dtype and out.shape == x.shape
    check(out, cpu(x))


@pytest.mark.parametrize("pieces", [1, 2])
@pytest.mark.parametrize("rows,cols", [(1100, 1300), (2100, 700), (600, 3000)])
def test_larger_tiles(rows, cols, pieces):
    x = gradient(rows, cols, BF16, seed=2)
    out = torch.empty(rows, cols, device=DEV)
    say(f"[muon] {rows} x {cols}, {pieces} pieces")
    T.orthogonalize(x, out=out, pieces=pieces)
    check(out, cpu(x), F32, pieces)


@pytest.mark.parametrize("steps", [1, 2, 3, 8])
def test_steps(steps):
    x = gradient(90, 140, F32, seed=3)
    check(T.orthogonalize(x, steps=steps), cpu(x), steps=steps, what=f"{steps} steps")


def test_singular_values_come_near_one():
    g = torch.Generator(device=DEV)
    g.manual_seed(0)
    x = torch.randn(300, 500, generator=g, device=DEV)
    s = torch.linalg.svdvals(T.orthogonalize(x).double().cpu())
    assert 0.6 < float(s.min()) and float(s.max()) < 1.25


def test_other_coefficients():
    x = gradient(60, 80, F32, seed=4)
    for co in ((2.0, -1.5, 0.5), (1.875, -1.25, 0.375), (1.5, -0.5, 0.0), (3.0, -3.0, 1.0), (0.5, 0.0, 0.0)):
        exact = E.newton_schulz(cpu(x), steps=6, coefficients=co)
        got = cpu(T.orthogonalize(x, steps=6, coefficients=co))
        assert norm(got - exact) <= 2e-5 * norm(exact), co


@pytest.mark.parametrize("scale", [1e-30, 1e-12, 1e12, 1e30])
def test_any_size_of_gradient(scale):
    x = gradient(40, 70, F32, seed=5) * scale
    exact = E.newton_schulz(cpu(x))
    got = cpu(T.orthogonalize(x))
    # (X is held times 2^14 or more in fp16, whose smallest step is 2^-24: an entry of
    # the first X is off by 2^-39 at most whatever its size, which five steps multiply
    # by 3.4445 each.  A gradient far below eps has entries smaller than that.)
    assert norm(got - exact) <= 1e-5 * norm(exact) + 3.4445 ** 5 * 2.0 ** -39 * x.numel() ** 0.5
    tiny = gradient(40, 70, F32, seed=5) * 1e-30
    unit = cpu(T.orthogonalize(tiny, eps=0.0))
    assert norm(unit - E.newton_schulz(cpu(tiny), eps=0.0)) <= 1e-5 * norm(unit)


@pytest.mark.parametrize("r,c", [(50, 30), (300, 280)])
def test_zero_without_eps(r, c):
    assert not T.orthogonalize(torch.zeros(r, c, device=DEV), eps=0.0).any()


def test_zero_rank_one_and_orthogonal():
    assert not T.orthogonalize(torch.zeros(50, 30, device=DEV)).any()
    u, v = np.random.default_rng(6).standard_normal((2, 60))
    x = torch.from_numpy(np.outer(u, v)).float().to(DEV)
    check(T.orthogonalize(x), cpu(x), what="rank one")
    q = torch.from_numpy(np.linalg.qr(np.random.default_rng(7).standard_normal((64, 64)))[0]).float().to(DEV)
    check(T.orthogonalize(q), cpu(q), what="orthogonal")


def test_views_in_place_and_types():
    x = gradient(70, 90, BF16, seed=8)
    want = T.orthogonalize(x)
    big = torch.full((75, 200), 7.0, dtype=BF16, device=DEV)
    for off in (0, 1, 8):
        view = big[2:72, off:off + 90]
        view.copy_(x)
        assert torch.equal(T.orthogonalize(view), want)
        T.orthogonalize(view, out=view)
        assert torch.equal(view, want)
        rest = big.clone()
        rest[2:72, off:off + 90] = 7.0
        assert torch.equal(rest, torch.full_like(rest, 7.0))
        big.fill_(7.0)
    for dtype in (F32, F16):
        out = torch.empty(70, 90, dtype=dtype, device=DEV)
        T.orthogonalize(x, out=out)
        check(out, cpu(x), what="from bfloat16 to")


def test_empty():
    for shape in ((0, 5), (5, 0), (0, 0)):
        assert T.orthogonalize(torch.empty(shape, device=DEV)).shape == shape
    T.Muon([], []).step()


# ------------------------------------------------------------------- the step
def step_case(shapes, dtype, seed=0, grad_dtype=None):
    params = [gradient(r, c, dtype, seed + 1, noise=1.0) for r, c in shapes]
    grads = [gradient(r, c, grad_dtype or dtype, seed + 2) for r, c in shapes]
    momentum = [gradient(r, c, F32, seed + 3) * 3 for r, c in shapes]
    return params, grads, momentum


def check_step(before, after, grads, m0, m1, lr, mu, nesterov, wd, factors, dtype, pieces):
    for p, q, g, m, n, f in zip(before, after, grads, m0, m1, factors):
        want, wm = E.muon_step(cpu(p), cpu(g), cpu(m), lr, mu, nesterov, wd, f)
        # one fused product and sum, rounded once
        assert np.all(np.abs(cpu(n) - wm) <= 2.0 ** -23 * (np.abs(wm) + np.abs(mu * cpu(m))) + 1e-40)
        u = cpu(g) + mu * wm if nesterov else wm
        x = E.newton_schulz(u)
        tol = tolerance(u, F32, pieces, x) * lr * f * norm(x) + (HALF[dtype] + 2.0 ** -22) * norm(want)
        say(f"[muon] step {want.shape}: off {norm(cpu(q) - want):.2e}, bound {tol:.2e}")
        assert norm(cpu(q) - want) <= tol


LISTS = {
    "one": [(40, 60)],
    "mixed": [(64, 27), (10, 300), (300, 10), (128, 128), (1, 1), (5, 1), (200, 333)],
    "conv": [(64, 27)] + [(64, 576)] * 3 + [(128, 576), (128, 1152), (128, 64), (256, 1152), (256, 128)],
    "long": [(8 + i, 40 - i) for i in range(30)] * 2,
}


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("name", list(LISTS))
def test_step_over_a_list(name, dtype):
    shapes = LISTS[name]
    params, grads, momentum = step_case(shapes, dtype, seed=10)
    before, m0 = [p.clone() for p in params], [m.clone() for m in momentum]
    say(f"[muon] list {name} {dtype}")
    T.Muon(params, grads, lr=0.05, momentum=0.9, weight_decay=0.1, momentum_buffers=momentum).step()
    factors = [max(1.0, r / c) ** 0.5 for r, c in shapes]
    check_step(before, params, grads, m0, momentum, 0.05, 0.9, True, 0.1, factors, dtype, PIECES[dtype])


@pytest.mark.parametrize("nesterov", [True, False])
@pytest.mark.parametrize("scale", ["rms", "spectral", 0.25])
def test_options(nesterov, scale):
    shapes = [(50, 20), (20, 50)]
    params, grads, momentum = step_case(shapes, F32, seed=20)
    before, m0 = [p.clone() for p in params], [m.clone() for m in momentum]
    opt = T.Muon(params, grads, lr=0.1, momentum=0.8, nesterov=nesterov, scale=scale, momentum_buffers=momentum)
    factors = [0.2 * 50 ** 0.5 if scale == "rms" else 0.25 if scale == 0.25 else max(1.0, r / c) ** 0.5 for r, c in shapes]
    opt.step()
    check_step(before, params, grads, m0, momentum, 0.1, 0.8, nesterov, 0.0, factors, F32, 2)
    before, m0 = [p.clone() for p in params], [m.clone() for m in momentum]
    opt.step(lr=0.01)
    check_step(before, params, grads, m0, momentum, 0.01, 0.8, nesterov, 0.0, factors, F32, 2)


def test_mixed_types_and_strides():
    """Gradients of other types than the weights', weights of both precisions in one
    list, rows with gaps and addresses off 16 bytes."""
    shapes = [(60, 100), (100, 60), (33, 47), (47, 33)]
    params, grads, momentum = step_case(shapes, F32, seed=30)
    kinds = [(F32, BF16), (BF16, F32), (F16, F16), (BF16, BF16)]
    holders, ps, gs = [], [], []
    for (pt, gt), p, g, off in zip(kinds, params, grads, (0, 3, 1, 8)):
        for t, dt, to in ((p, pt, ps), (g, gt, gs)):
            h = torch.full((t.shape[0], t.shape[1] + off + 5), 7.0, dtype=dt, device=DEV)
            v = h[:, off:off + t.shape[1]]
            v.copy_(t)
            holders.append((h, off, t.shape[1]))
            to.append(v)
    before, m0 = [p.clone() for p in ps], [m.clone() for m in momentum]
    T.Muon(ps, gs, lr=0.02, momentum=0.95, momentum_buffers=momentum).step()
    for i, ((pt, _), (r, c)) in enumerate(zip(kinds, shapes)):
        check_step(before[i:i + 1], ps[i:i + 1], gs[i:i + 1], m0[i:i + 1], momentum[i:i + 1], 0.02, 0.95, True, 0.0,
                   [max(1.0, r / c) ** 0.5], pt, PIECES[pt])
    for h, off, c in holders:
        rest = h.clone()
        rest[:, off:off + c] = 7.0
        assert torch.equal(rest, torch.full_like(rest, 7.0))


def test_not_finite_stays_in_its_matrix():
    shapes = [(40, 50), (60, 30), (30, 30)]
    params, grads, momentum = step_case(shapes, F32, seed=40)
    clean = [p.clone() for p in params]
    m2 = [m.clone() for m in momentum]
    T.Muon(clean, grads, momentum_buffers=m2).step()
    grads[1][3, 4], grads[2][0, 0] = float("nan"), float("inf")
    T.Muon(params, grads, momentum_buffers=momentum).step()
    assert torch.equal(params[0], clean[0])
    assert torch.isnan(params[1]).all() and torch.isnan(params[2]).all()


def test_bind_and_zero_momentum():
    shapes = [(40, 64), (64, 40)]
    params, grads, _ = step_case(shapes, F32, seed=50)
    opt = T.Muon(params, grads, lr=0.1, momentum=0.9)
    m0 = [torch.zeros(s, device=DEV) for s in shapes]
    before = [p.clone() for p in params]
    opt.step()
    factors = [max(1.0, r / c) ** 0.5 for r, c in shapes]
    check_step(before, params, grads, m0, opt.momentum, 0.1, 0.9, True, 0.0, factors, F32, 2)
    other = [g.to(BF16) for g in step_case(shapes, F32, seed=60)[1]]
    moved = [p.clone() for p in params]
    with pytest.raises(ValueError):
        opt.bind(moved[::-1], other)
    m1, kept = [m.clone() for m in opt.momentum], [p.clone() for p in params]
    opt.bind(moved, other)
    opt.step()
    check_step(kept, moved, other, m1, opt.momentum, 0.1, 0.9, True, 0.0, factors, F32, 2)
    assert all(torch.equal(a, b) for a, b in zip(params, kept))


def test_equal_calls_give_equal_bits():
    for dtype in (F32, BF16):
        x = gradient(500, 700, dtype, seed=70)
        first = T.orthogonalize(x)
        torch.full((1 << 26,), float("nan"), device=DEV)  # (what the next workspace finds)
        assert torch.equal(T.orthogonalize(x), first)


def test_streams_and_two_at_once():
    x = [gradient(600, 400, BF16, seed=80 + i) for i in range(2)]
    want = [T.orthogonalize(v) for v in x]
    params, grads, momentum = step_case([(200, 300), (300, 100)], F32, seed=90)
    clean, m2 = [p.clone() for p in params], [m.clone() for m in momentum]
    one = T.Muon(clean, grads, momentum_buffers=m2)
    for _ in range(6):
        one.step()
    torch.cuda.synchronize()
    s = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = []
    for _ in range(4):
        for i in range(2):
            with torch.cuda.stream(s[i]):
                got.append((i, T.orthogonalize(x[i])))
    # one handle's steps from two streams: each after the one before
    opt = T.Muon(params, grads, momentum_buffers=momentum)
    for k in range(6):
        s[k % 2].wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s[k % 2]):
            opt.step()
    torch.cuda.synchronize()
    assert all(torch.equal(g, want[i]) for i, g in got)
    assert all(torch.equal(a, b) for a, b in zip(params, clean))


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_captured_and_replayed(dtype):
    shapes = [(128, 300), (300, 70), (64, 64)]
    params, grads, momentum = step_case(shapes, dtype, seed=100)
    eager, m2 = [p.clone() for p in params], [m.clone() for m in momentum]
    opt = T.Muon(params, grads, momentum_buffers=momentum)
    ref = T.Muon(eager, grads, momentum_buffers=m2)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        opt.step()
    torch.cuda.current_stream().wait_stream(s)
    ref.step()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        opt.step()
    for k in range(4):
        for g, n in zip(grads, step_case(shapes, dtype, seed=110 + k)[1]):
            g.copy_(n)
        ref.step()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(params, eager)), f"replay {k}"
        assert all(torch.equal(a, b) for a, b in zip(momentum, m2)), f"replay {k}"


def test_offsets_beyond_32_bits():
    """A matrix of more than 2^31 values, against the polynomial of its Gram matrix in
    64 bits on its last rows."""
    r, c = 1000000, 2176
    g = torch.Generator(device=DEV)
    g.manual_seed(5)
    x = torch.empty(r, c, dtype=BF16, device=DEV)
    for i in range(0, r, 100000):
        x[i:i + 100000] = torch.randn(100000, c, generator=g, device=DEV)
    say("[muon] a matrix past 2^31 values")
    out = T.orthogonalize(x)
    s = torch.zeros(c, c, dtype=torch.float64, device=DEV)
    for i in range(0, r, 50000):
        v = x[i:i + 50000].double()
        s += v.t() @ v
    s /= s.diagonal().sum()
    a, b, co = E.COEFFICIENTS
    p = torch.eye(c, dtype=torch.float64, device=DEV)
    for _ in range(5):
        q = p @ s @ p
        p = (a * torch.eye(c, dtype=torch.float64, device=DEV) + b * q + co * q @ q) @ p
    n = 0.0
    for i in range(0, r, 100000):
        n += float(x[i:i + 100000].double().square().sum())
    want = x[-3000:].double() @ p / n ** 0.5
    # (a Gaussian matrix of this shape is near orthogonal: five steps with one fp16
    # piece are off by 2e-3 at most, and bfloat16 by half a step)
    assert float((out[-3000:].double() - want).norm() / want.norm()) <= 4e-3 + HALF[BF16]


def test_refusals():
    x = gradient(20, 30)
    for bad in (lambda: T.orthogonalize(x.cpu()), lambda: T.orthogonalize(x[0]), lambda: T.orthogonalize(x.t()),
                lambda: T.orthogonalize(x.double()), lambda: T.orthogonalize(x, out=x[:, :5]),
                lambda: T.Muon([x], []), lambda: T.Muon([x], [x[:5]]), lambda: T.Muon([x], [x.t()]),
                lambda: T.Muon([x], [x.clone()], momentum_buffers=[x.to(BF16)]),
                lambda: T.Muon([x], [x.clone()], momentum_buffers=[torch.zeros(20, 31, device=DEV)[:, :30]]),
                lambda: T.Muon([x], [x.clone()], scale="other")):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(B.PsgdError, match="overlap"):
        T.Muon([x], [x]).step()
    with pytest.raises(B.PsgdError, match="overlap"):
        T.orthogonalize(x[:, :20], out=x[:, 5:25])
    with pytest.raises(B.PsgdError, match="steps"):
        T.orthogonalize(x, steps=0)

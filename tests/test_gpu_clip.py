"""The gradient clip on the GPU against the float64 oracle.

Tolerances: squares are summed in fp64, so norms and the coefficient carry
one rounding to fp32 (2^-24; the comparison allows 2^-23); an output carries
the coefficient's rounding, the product's and the output type's own: 2^-22 in
fp32, 2^-8 + 2^-22 in bfloat16, 2^-11 + 2^-22 in float16, of its own size, or
half the type's smallest step.
"""
import gc
import weakref

import numpy as np
import pytest

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a GPU", allow_module_level=True)

import workloads as W  # noqa: E402
from gpu_util import say  # noqa: E402
from oracle import microscaling as MX  # noqa: E402
from rank_gradient_compression_amd import binding as B  # noqa: E402
from rank_gradient_compression_amd import torch_api as T  # noqa: E402

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16
REL = {F32: 2.0 ** -22, BF16: 2.0 ** -8 + 2.0 ** -22, F16: 2.0 ** -11 + 2.0 ** -22}
STEP = {F32: 2.0 ** -149, BF16: 2.0 ** -133, F16: 2.0 ** -24}


def grads(sizes, dtypes, seed=0, size=1e-2):
    g = np.random.default_rng([seed, len(sizes)])
    return [torch.from_numpy(size * g.standard_normal(n) * np.exp(g.standard_normal())).to(d).to(DEV)
            for n, d in zip(sizes, dtypes)]


def f64(t):
    return t.detach().cpu().double().numpy()


def check(gs, stats, outs, max_norm, scale=1.0, before=None):
    src = [f64(g) for g in gs] if before is None else before
    norm, coef, per, want = MX.clip(src, max_norm, scale)
    s = f64(stats)
    assert s[0] == pytest.approx(norm, rel=2.0 ** -23) and s[1] == pytest.approx(coef, rel=2.0 ** -23)
    assert np.allclose(s[2:], per, rtol=2.0 ** -23, atol=0)
    if outs is None:
        return
    for o, w in zip(outs, want):
        assert np.all(np.abs(f64(o).reshape(-1) - w.reshape(-1)) <= REL[o.dtype] * np.abs(w.reshape(-1)) + STEP[o.dtype])


SETS = {
    "none": [],
    "one value": [1],
    "one vector": [650],
    "odd": [1, 3, 8191, 8192, 8193, 0, 27, 100001, 0],
    "many": [(i * 37) % 301 for i in range(700)],
    "large and small": [3_000_001, 5, 2_000_000, 1],
}


@pytest.mark.parametrize("name", list(SETS))
@pytest.mark.parametrize("din,dout", [(F32, F32), (F32, BF16), (F32, F16), (BF16, F32), (BF16, BF16), (BF16, F16),
                                      (F16, F32), (F16, BF16), (F16, F16)])
def test_norm_and_clip(name, din, dout):
    sizes = SETS[name]
    gs = grads(sizes, [din] * len(sizes))
    outs = [torch.full((n,), 9.0, dtype=dout, device=DEV) for n in sizes]
    say(f"[clip] {name} {din} -> {dout}")
    c = T.GradientClip(gs, outs)
    total = MX.clip([f64(g) for g in gs], 1.0)[0]
    for max_norm in (0.3 * total, 2.0 * total + 1.0, 0.0, float("inf")):
        stats = c.clip(max_norm)
        check(gs, stats, outs, max_norm)
        again = [o.clone() for o in outs]
        assert torch.equal(c.clip(max_norm), stats) and all(torch.equal(a, b) for a, b in zip(again, outs))
        check(gs, c.norm(max_norm), None, max_norm)
    check(gs, c.clip(0.5 * total, scale=-0.25), outs, 0.5 * total, -0.25)
    c.close()


def test_mixed_types_and_alignments():
    sizes = [1000, 8192, 20000, 77, 8200, 16385]
    kinds = [F32, BF16, F16, BF16, F32, F16]
    for shift_in, shift_out in [(0, 1), (1, 0), (1, 1), (3, 2), (4, 4)]:
        gs, outs, keep = [], [], []
        for i, (n, d) in enumerate(zip(sizes, kinds)):
            src = torch.full((n + 16,), 5.0, dtype=d, device=DEV)
            dst = torch.full((n + 16,), 5.0, dtype=kinds[-1 - i], device=DEV)
            gs.append(src[shift_in:shift_in + n])
            outs.append(dst[shift_out:shift_out + n])
            keep.append(dst)
            gs[-1].copy_(grads([n], [d], seed=i)[0])
        say(f"[clip] mixed types, shifts {shift_in} {shift_out}")
        c = T.GradientClip(gs, outs)
        check(gs, c.clip(0.5), outs, 0.5)
        for dst, n in zip(keep, sizes):
            assert bool((dst[:shift_out] == 5).all()) and bool((dst[shift_out + n:] == 5).all()), "wrote outside"


def test_in_place_and_new_addresses():
    sizes = [3000, 17, 9000]
    gs = grads(sizes, [F32, BF16, BF16])
    before = [f64(g) for g in gs]
    c = T.GradientClip(gs)
    check(gs, c.clip(0.1), gs, 0.1, before=before)
    other = grads(sizes, [F32, BF16, BF16], seed=5)
    outs = [torch.empty_like(g) for g in other]
    c.bind(other, outs)
    check(other, c.clip(0.1), outs, 0.1)
    with pytest.raises(ValueError):
        c.bind(other[:2], outs[:2])
    with pytest.raises(ValueError):
        c.bind([g.float() for g in other], outs)


def test_large_values_do_not_overflow_and_small_ones_do_not_vanish():
    gs = [torch.tensor([1e30, -2e30, 3.0], device=DEV), torch.tensor([1e-30, 2e-25], device=DEV)]
    outs = [torch.empty_like(g) for g in gs]
    c = T.GradientClip(gs, outs)
    check(gs, c.clip(1.0), outs, 1.0)
    tiny = [torch.full((1000,), 1e-30, device=DEV)]
    check(tiny, T.GradientClip(tiny, [torch.empty_like(tiny[0])]).clip(1.0), None, 1.0)


def test_infinities_and_nan():
    gs = grads([5000, 300], [F32, BF16])
    outs = [torch.empty_like(g) for g in gs]
    c = T.GradientClip(gs, outs)
    gs[0][4321] = float("inf")
    s = f64(c.clip(1.0))
    assert np.isinf(s[0]) and s[1] == 0.0 and np.isinf(s[2]) and np.isfinite(s[3])
    o = f64(outs[0])
    assert np.isnan(o[4321]) and np.all(np.delete(o, 4321) == 0) and np.all(f64(outs[1]) == 0)
    gs[1][7] = float("nan")
    s = f64(c.clip(1.0))
    assert np.isnan(s[0]) and np.isnan(s[1]) and np.isinf(s[2]) and np.isnan(s[3])
    assert all(bool(t.isnan().all()) for t in outs)


def test_model_set_into_the_flat_buffer():
    tensors = W.resnet18_cifar_set()
    shapes = [s for _, s in tensors]
    ps = T.PowerSGD(shapes, 2, device=DEV)
    n = [int(np.prod(s)) for s in shapes]
    gs = grads(n, [BF16] * len(n))
    outs = [ps.view(ps.grads, i).view(-1) for i in range(len(n))]
    c = T.GradientClip(gs, outs)
    check(gs, c.clip(0.7), outs, 0.7)
    used = sum(float(o.double().abs().sum()) for o in outs)
    assert used == pytest.approx(float(ps.grads.double().abs().sum()), rel=1e-12), "wrote between the tensors"
    ps.close()


def test_more_than_2_to_the_31_elements():
    n = (1 << 31) + 12345
    say(f"[clip] one tensor of {n} bf16 values")
    g = torch.full((n,), 2.0 ** -10, dtype=BF16, device=DEV)
    g[-1] = 3.0
    c = T.GradientClip([g])
    norm = (((n - 1) * 2.0 ** -20) + 9.0) ** 0.5
    s = f64(c.clip(norm / 2))
    assert s[0] == pytest.approx(norm, rel=2.0 ** -23) and s[1] == pytest.approx(0.5, rel=1e-6)
    assert float(g[-1]) == 1.5 and float(g[-2]) == 2.0 ** -11 and float(g[0]) == 2.0 ** -11


def test_calls_before_and_without_bound_outputs():
    # few sums, which the writing pass adds, and more than it (and LDS) takes
    for count, size in ((1, 5000), (20, 600_000), (2100, 70)):
        g = [torch.full((size,), 0.5, device=DEV) for _ in range(count)]
        o = [torch.full_like(t, 7.0) for t in g]
        h = B.psgd_clip_create([t.numel() for t in g], [B.PSGD_DTYPE_F32] * len(g), [B.PSGD_DTYPE_F32] * len(g))
        nbytes = B.psgd_clip_workspace(h)
        ws, stats = torch.empty(nbytes, dtype=torch.uint8, device=DEV), torch.zeros(2 + len(g), device=DEV)
        s = torch.cuda.current_stream().cuda_stream
        B.psgd_clip_workspace_init(h, ws.data_ptr(), nbytes, s)
        B.psgd_clip_apply(h, 1.0, 1.0, stats.data_ptr(), ws.data_ptr(), nbytes, s)
        assert bool(torch.isnan(stats).all()), "never bound"
        B.psgd_clip_bind(h, [t.data_ptr() for t in g], None, ws.data_ptr(), nbytes, s)
        B.psgd_clip_apply(h, 1.0, 1.0, stats.data_ptr(), ws.data_ptr(), nbytes, s)
        norm = 0.5 * sum(t.numel() for t in g) ** 0.5
        assert abs(float(stats[0]) - norm) <= 2.0 ** -23 * norm and all(bool((t == 7.0).all()) for t in o)
        B.psgd_clip_bind(h, [t.data_ptr() for t in g], [t.data_ptr() for t in o], ws.data_ptr(), nbytes, s)
        B.psgd_clip_apply(h, 1.0, 1.0, stats.data_ptr(), ws.data_ptr(), nbytes, s)
        assert all(bool((t == t[0]).all()) and 0 < float(t[0]) < 0.5 for t in o)
        torch.cuda.synchronize()
        B.psgd_clip_destroy(h)


def test_refusals():
    x = torch.zeros(8, device=DEV)
    for gs, outs in [([x.double()], None), ([x[::2]], None), ([torch.zeros(8)], None), ([x], [torch.zeros(7, device=DEV)]),
                     ([x], []), ([x], [x.int()])]:
        with pytest.raises(ValueError):
            T.GradientClip(gs, outs)
    c = T.GradientClip([x])
    for bad in (-1.0, float("nan")):
        with pytest.raises(T.B.PsgdError):
            c.clip(bad)
    with pytest.raises(T.B.PsgdError):
        c.clip(1.0, scale=float("inf"))
    with pytest.raises(T.B.PsgdError):
        T.GradientClip([x, x])  # both in place: the outputs overlap


def test_another_stream_and_graph_replays():
    sizes = [20000, 5, 9000]
    gs = grads(sizes, [F32, BF16, F32])
    outs = [torch.empty(n, dtype=F32, device=DEV) for n in sizes]
    c = T.GradientClip(gs, outs)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        st = c.clip(0.2)
    s.synchronize()
    check(gs, st, outs, 0.2)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        stats = c.clip(0.2)
    for i in range(4):
        for a, b in zip(gs, grads(sizes, [F32, BF16, F32], seed=20 + i)):
            a.copy_(b)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        check(gs, stats, outs, 0.2)
        replayed = [o.clone() for o in outs] + [stats.clone()]
        eager = c.clip(0.2)
        assert all(torch.equal(a, b) for a, b in zip(replayed, outs + [eager]))


def test_refused_bind_keeps_the_binding():
    sizes = [3000, 500]
    gs = grads(sizes, [F32, F32])
    outs = [torch.empty_like(g) for g in gs]
    before, refs = [f64(g) for g in gs], [weakref.ref(t) for t in (*gs, *outs)]
    c = T.GradientClip(gs, outs)
    others = grads(sizes, [F32, F32], seed=8)
    for bad in ([others[0], others[0][:500]], [others[1].new_empty(3000), others[0][:500]]):
        with pytest.raises(B.PsgdError, match="overlap"):
            c.bind(others, bad)
    del gs, outs
    gc.collect()
    assert all(r() is not None for r in refs)
    check(None, c.clip(0.1), [r() for r in refs[2:]], 0.1, before=before)


@pytest.mark.parametrize("count", [1, 2100])  # sums added by the writing pass, and by a launch of their own
def test_infinite_limit_clips_nothing(count):
    gs = grads([700] * count, [F32] * count)
    gs[-1][5], gs[0][6] = float("inf"), float("-inf")
    outs = [torch.empty_like(g) for g in gs]
    c = T.GradientClip(gs, outs)
    for stats in (c.clip(float("inf")), c.norm()):
        s = f64(stats)
        assert np.isinf(s[0]) and s[1] == 1.0 and np.isinf(s[[2, -1]]).all() and np.isfinite(s[3:-1]).all()
    assert all(torch.equal(o, g) for o, g in zip(outs, gs))
    gs[0][7] = float("nan")
    for stats in (c.clip(float("inf")), c.norm()):
        s = f64(stats)
        assert np.isnan(s[:3]).all()
    assert all(bool(o.isnan().all()) for o in outs)


def test_calls_of_one_handle_on_several_streams():
    """Construction, binding and clips in turn on two streams, the first of
    them behind work that takes a while, without a host synchronisation."""
    sizes = [30000, 7]
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    sets = [grads(sizes, [F32, BF16], seed=i) for i in range(4)]
    outs = [[torch.empty(n, device=DEV) for n in sizes] for _ in sets]
    busy = torch.ones(4096, 4096, device=DEV)
    torch.cuda.synchronize()
    stats = []
    with torch.cuda.stream(a):
        for _ in range(20):
            torch.mm(busy, busy)
        c = T.GradientClip(sets[0], outs[0])
    with torch.cuda.stream(b):
        stats.append(c.clip(0.1))
    for i, s in ((1, a), (2, b), (3, a)):
        with torch.cuda.stream(s):
            for _ in range(20):
                torch.mm(busy, busy)
            c.bind(sets[i], outs[i])
        with torch.cuda.stream(b if s is a else a):
            stats.append(c.clip(0.1))
    torch.cuda.synchronize()
    for g, o, s in zip(sets, outs, stats):
        check(g, s, o, 0.1)


# bytes beyond which the outputs are stored past the cache, sums and chunks of
# 8192 values up to which the writing pass adds the sums (the library's limits)
STREAM_BYTES, INLINE_CHUNKS = 192 << 20, 8192


@pytest.mark.parametrize("dtype,out,sizes,inline", [
    (F32, F32, [30_000_001, 1_000_000], True), (BF16, F32, [40_000_003], True),
    (F32, F32, [70_000_001, 13], False), (F32, BF16, [20_000_000, 49_999_999], False)])
def test_lists_larger_than_the_cache(dtype, out, sizes, inline):
    """Streaming stores, with the sums added by the writing pass and by a launch
    of their own; the outputs in float64 on the device."""
    size = lambda d: torch.empty(0, dtype=d).element_size()  # noqa: E731
    total, chunks = sum(sizes), sum(-(-n // 8192) for n in sizes)
    assert total * (size(dtype) + size(out)) > STREAM_BYTES and total * size(dtype) < 1 << 30
    assert (chunks <= INLINE_CHUNKS) == inline
    g = torch.Generator(device=DEV)
    g.manual_seed(total)
    gs = [(1e-3 * torch.randn(n, generator=g, device=DEV)).to(dtype) for n in sizes]
    outs = [torch.full((n,), 9.0, dtype=out, device=DEV) for n in sizes]
    say(f"[clip] {sizes} {dtype} -> {out}")
    per = [float((t.double() ** 2).sum()) ** 0.5 for t in gs]
    norm = sum(p * p for p in per) ** 0.5
    limit = 0.4 * norm
    s = f64(T.GradientClip(gs, outs).clip(limit))
    coef = limit / (norm + 1e-6)
    # (the norms of the reference are float64 sums in another order: 2^-40 is far above their error)
    assert np.allclose(s, [norm, coef, *per], rtol=2.0 ** -23 + 2.0 ** -40, atol=0)
    for t, o in zip(gs, outs):
        want = t.double() * coef
        assert bool(((o.double() - want).abs() <= REL[out] * want.abs() + STEP[out]).all())

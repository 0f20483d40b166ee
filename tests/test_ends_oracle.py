"""CPU pins of the oracle of the cross entropy and of the orthogonalised step:
other formulas, differences, closed forms, and planted mistakes."""
import numpy as np
import pytest

from oracle import ends as E

torch = pytest.importorskip("torch")


def case(t=7, v=11, d=5, seed=0, bias=True):
    g = np.random.default_rng(seed)
    x, w = g.standard_normal((t, d)), g.standard_normal((v, d))
    y = g.integers(0, v, t)
    y[2] = -100
    return x, w, y, g.standard_normal(v) if bias else None


@pytest.mark.parametrize("bias", [True, False])
@pytest.mark.parametrize("mean", [True, False])
def test_cross_entropy_is_torchs(bias, mean):
    x, w, y, b = case(bias=bias)
    loss, lse, dx, dw, db = E.cross_entropy(x, w, y, b, mean=mean)
    xt, wt = torch.tensor(x, requires_grad=True), torch.tensor(w, requires_grad=True)
    bt = torch.tensor(b if bias else np.zeros(len(w)), requires_grad=True)
    l = xt @ wt.t() + bt
    total = torch.nn.functional.cross_entropy(l, torch.tensor(y), reduction="mean" if mean else "sum")
    total.backward()
    each = torch.nn.functional.cross_entropy(l, torch.tensor(y), reduction="none").detach().numpy()
    np.testing.assert_allclose(loss, each, rtol=1e-12, atol=1e-14)
    np.testing.assert_allclose(lse, torch.logsumexp(l, 1).detach().numpy(), rtol=1e-12)
    for mine, theirs in ((dx, xt.grad), (dw, wt.grad), (db, bt.grad)):
        np.testing.assert_allclose(mine, theirs.numpy(), rtol=1e-10, atol=1e-13)


def test_cross_entropy_gradients_are_differences():
    x, w, y, b = case(seed=3)
    u = np.random.default_rng(4).standard_normal(len(x))
    _, _, dx, dw, db = E.cross_entropy(x, w, y, b, weights=u, scale=0.5)

    def f(x, w, b):
        return 0.5 * float((u * E.cross_entropy(x, w, y, b)[0]).sum())

    h = 1e-6
    for which, grad in ((0, dx), (1, dw), (2, db)):
        for i in list(np.ndindex(grad.shape))[::7]:
            at = [x.copy(), w.copy(), b.copy()]
            at[which][i] += h
            up = f(*at)
            at[which][i] -= 2 * h
            assert (up - f(*at)) / (2 * h) == pytest.approx(grad[i], abs=1e-8)


def test_ignored_and_impossible_targets():
    x, w, y, b = case()
    y[0], y[1], y[3] = -1, 4, 99
    loss, lse, dx, dw, _ = E.cross_entropy(x, w, y, b, ignore_index=4, mean=True)
    assert loss[0] == loss[1] == loss[2] == 0.0 and np.isnan(loss[3]) and np.isfinite(lse).all()
    assert not dx[:4].any() and dx[4:].any()
    assert not any(v.any() for v in E.cross_entropy(x, w, np.full(7, -100), b, mean=True)[2:])


def test_a_masked_word_has_no_gradient():
    x, w, y, b = case()
    y[:], b[6] = 1, -np.inf
    _, lse, dx, dw, db = E.cross_entropy(x, w, y, b)
    assert not dw[6].any() and db[6] == 0.0 and np.isfinite(lse).all() and np.isfinite(dx).all()


@pytest.mark.parametrize("shape", [(4, 9), (9, 4), (6, 6), (1, 5), (5, 1), (1, 1)])
def test_newton_schulz_maps_singular_values(shape):
    u = np.random.default_rng(5).standard_normal(shape)
    p, s, q = np.linalg.svd(u, full_matrices=False)
    s = s / np.sqrt((s * s).sum())
    a, b, c = E.COEFFICIENTS
    for _ in range(5):
        s = a * s + b * s ** 3 + c * s ** 5
    np.testing.assert_allclose(E.newton_schulz(u, eps=0.0), (p * s) @ q, rtol=1e-9, atol=1e-12)
    assert shape != (6, 6) or np.all((0.6 < s) & (s < 1.3))


def test_newton_schulz_of_zero_and_of_any_scale():
    u = np.random.default_rng(6).standard_normal((3, 8))
    assert not E.newton_schulz(np.zeros((3, 8))).any()
    np.testing.assert_allclose(E.newton_schulz(u * 1e20), E.newton_schulz(u * 1e3), rtol=1e-8, atol=1e-10)


@pytest.mark.parametrize("nesterov", [True, False])
def test_muon_step_by_hand(nesterov):
    g = np.random.default_rng(7)
    p, grad, m = g.standard_normal((3, 4)), g.standard_normal((3, 4)), g.standard_normal((3, 4))
    new_p, new_m = E.muon_step(p, grad, m, 0.1, 0.9, nesterov, 0.5, 2.0)
    np.testing.assert_allclose(new_m, 0.9 * m + grad)
    u = grad + 0.9 * new_m if nesterov else new_m
    np.testing.assert_allclose(new_p, p * 0.95 - 0.2 * E.newton_schulz(u))


def test_rounded_steps_stay_near():
    g = np.random.default_rng(8)
    u = g.standard_normal((48, 96)) + 5.0 * np.outer(g.standard_normal(48), g.standard_normal(96))
    exact = E.newton_schulz(u)
    off = [np.linalg.norm(E.newton_schulz_rounded(u, n) - exact) / np.linalg.norm(exact) for n in (1, 2)]
    assert 1e-5 < off[0] < 4e-3 and off[1] < 2e-6


@pytest.mark.parametrize("mistake", ["sign", "transposed", "square", "no one-hot", "no lse"])
def test_planted_mistakes_show(mistake):
    x, w, y, b = case(seed=9)
    _, lse, dx, _, _ = E.cross_entropy(x, w, y, b)
    u = np.random.default_rng(10).standard_normal((4, 9))
    a, bb, c = E.COEFFICIENTS
    x0 = u / np.linalg.norm(u)
    g = x0 @ x0.T
    right = a * x0 + (bb * g + c * g @ g) @ x0
    np.testing.assert_allclose(right, E.newton_schulz(u, steps=1, eps=0.0), rtol=1e-12)
    l = x @ w.T + b
    p = np.exp(l - lse[:, None])
    hot = np.eye(len(w))[np.maximum(y, 0)]
    keep = (y >= 0)[:, None]
    np.testing.assert_allclose((p - hot) * keep @ w, dx, rtol=1e-10, atol=1e-13)
    wrong = {"sign": a * x0 - (bb * g + c * g @ g) @ x0, "transposed": a * x0 + x0 @ (bb * x0.T @ x0),
             "square": a * x0 + (bb * g + c * g) @ x0}.get(mistake)
    if wrong is not None:
        assert np.linalg.norm(wrong - right) > 1e-2
    else:
        bad = (p * keep) @ w if mistake == "no one-hot" else ((np.exp(l) - hot) * keep) @ w
        assert np.linalg.norm(bad - dx) > 1e-2

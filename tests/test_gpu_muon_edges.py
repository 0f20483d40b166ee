"""Edges of the orthogonalised step's handle on the GPU: refused options, weights
that a saved graph still needs, values that are not finite in large matrices."""
import pytest

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a GPU", allow_module_level=True)

from gpu_util import cpu, say  # noqa: E402
from oracle import ends as E  # noqa: E402
from test_gpu_muon import BF16, DEV, F32, check_step, gradient, step_case  # noqa: E402
from rank_gradient_compression_amd import binding as B  # noqa: E402
from rank_gradient_compression_amd import torch_api as T  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("lr", [float("nan"), float("inf"), 3e38])
def test_a_refused_learning_rate_is_not_kept(lr):
    """(3e38 times the matrix's sqrt(40 / 20) is no number.)"""
    shapes = [(40, 20)]
    params, grads, momentum = step_case(shapes, F32, seed=100)
    clean, m2 = [p.clone() for p in params], [m.clone() for m in momentum]
    opt, other = (T.Muon(p, grads, lr=0.1, momentum_buffers=m) for p, m in ((params, momentum), (clean, m2)))
    with pytest.raises(B.PsgdError):
        opt.step(lr=lr)
    assert all(torch.equal(a, b) for a, b in zip(params + momentum, clean + m2))
    opt.step()
    other.step()
    assert all(torch.equal(a, b) for a, b in zip(params + momentum, clean + m2))


@pytest.mark.parametrize("shape", [(30, 16), (300, 64)])
def test_a_step_between_forward_and_backward_is_noticed(shape):
    """The loss "none" keeps the weights for its backward pass: with other weights than
    it saw it would be of no loss at all."""
    w = torch.randn(shape, device=DEV, requires_grad=True)
    x, y = torch.randn(8, shape[1], device=DEV), torch.randint(0, shape[0], (8,), device=DEV)
    opt = T.Muon([w.detach()], [torch.randn(shape, device=DEV)])
    out = T.linear_cross_entropy(x, w, y, reduction="none")
    opt.step()
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        out.sum().backward()
    out = T.linear_cross_entropy(x, w, y, reduction="none")
    T.orthogonalize(w.detach(), out=w.detach())
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        out.sum().backward()
    T.linear_cross_entropy(x, w, y, reduction="none").sum().backward()
    with torch.inference_mode():
        p, g = torch.randn(shape, device=DEV), torch.randn(shape, device=DEV)
        T.Muon([p], [g]).step()


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_not_finite_stays_in_its_large_matrix(dtype):
    """One value that is not finite, in matrices of several tiles: all of its matrix's
    update is NaN and nothing of the others'."""
    shapes = [(200, 330), (330, 200), (70, 300), (300, 70)]
    params, grads, momentum = step_case(shapes, dtype, seed=110)
    clean, m2 = [p.clone() for p in params], [m.clone() for m in momentum]
    T.Muon(clean, grads, momentum_buffers=m2).step()
    grads[1][329, 0], grads[2][3, 4] = float("nan"), float("-inf")
    T.Muon(params, grads, momentum_buffers=momentum).step()
    assert torch.equal(params[0], clean[0]) and torch.equal(params[3], clean[3])
    assert torch.isnan(params[1]).all() and torch.isnan(params[2]).all()


@pytest.mark.parametrize("rows,cols", [(13, 650), (2600, 17), (27, 4096), (31, 900), (48, 700)])
def test_thin_matrices_keep_bfloat16s_digits(rows, cols):
    """Few singular values share a piece's roundings: two pieces, so that what is left
    is bfloat16's own rounding (half a step of each entry) and 1e-5 of the update."""
    x = gradient(rows, cols, BF16, seed=120)
    out = T.orthogonalize(x)
    exact = torch.from_numpy(E.newton_schulz(cpu(x))).to(DEV)
    rounded = exact.to(BF16).double()
    own = float((rounded - exact).norm() / exact.norm())
    off = float((out.double() - exact).norm() / exact.norm())
    say(f"[muon] thin {rows} x {cols}: off {off:.2e}, rounding alone {own:.2e}")
    # (an entry next to a tie may go to the other side of it: the distances add)
    assert off <= 1.02 * own + 1e-5


@pytest.mark.parametrize("shapes", [[(27, 64), (300, 500), (40, 30)], [(27, 64)] * 3 + [(700, 900)] * 3 + [(20, 800)],
                                    [(64, 27)] * 30 + [(1100, 1300)] * 3 + [(1300, 1100)]])
def test_lists_of_thin_and_large_matrices(shapes):
    """bfloat16 weights of both kinds in one list, joined or in groups of their own, one of
    small matrices only among them."""
    params, grads, momentum = step_case(shapes, BF16, seed=130)
    before, m0 = [p.clone() for p in params], [m.clone() for m in momentum]
    T.Muon(params, grads, lr=0.05, momentum=0.9, weight_decay=0.1, momentum_buffers=momentum).step()
    factors = [max(1.0, r / c) ** 0.5 for r, c in shapes]
    check_step(before, params, grads, m0, momentum, 0.05, 0.9, True, 0.1, factors, BF16, 1)

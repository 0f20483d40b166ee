"""Edges of the orthogonalised step's handle on the GPU: refused options, weights
that a saved graph still needs, values that are not finite in large matrices."""
import pytest

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a GPU", allow_module_level=True)

from test_gpu_muon import BF16, DEV, F32, gradient, step_case  # noqa: E402
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

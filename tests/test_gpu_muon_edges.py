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

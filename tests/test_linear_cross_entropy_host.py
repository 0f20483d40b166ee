"""What linear_cross_entropy asks of the library, with the library's calls
replaced on the host: these run without a GPU."""
import pytest

torch = pytest.importorskip("torch")
pytest.importorskip("rank_gradient_compression_amd")
from rank_gradient_compression_amd import torch_xent as X  # noqa: E402


@pytest.fixture
def calls(monkeypatch):
    made = []

    def loss_only(x, w, y, b=None, ignore_index=-100):
        made.append("loss")
        return torch.ones(len(x)), torch.ones(len(x))

    def train(x, w, y, b=None, **kw):
        made.append("gradients")
        return torch.ones(len(x)), torch.ones(len(x)), torch.zeros_like(x), torch.zeros_like(w), None

    monkeypatch.setattr(X, "cross_entropy", loss_only)
    monkeypatch.setattr(X, "cross_entropy_train", train)
    monkeypatch.setattr(X, "_total", lambda loss, y, mean, ignore_index: loss.sum())
    return made


@pytest.mark.parametrize("mode", [torch.no_grad, torch.inference_mode])
@pytest.mark.parametrize("reduction", ["mean", "sum", "none"])
def test_evaluation_forms_no_gradients(calls, mode, reduction):
    """Parameters ask for gradients under no_grad too; the call need not form them."""
    x, w, y = torch.ones(4, 3, requires_grad=True), torch.ones(5, 3, requires_grad=True), torch.zeros(4, dtype=torch.int64)
    with mode():
        out = X.linear_cross_entropy(x, w, y, reduction=reduction)
    assert calls == ["loss"] and not out.requires_grad
    X.linear_cross_entropy(x, w, y, reduction=reduction)
    assert calls == ["loss", "loss" if reduction == "none" else "gradients"]

"""The example that runs the vocabulary loss, the clip, the compression and the
orthogonalised step together: it runs, its gradients are the definition's, and
every step's weights follow from what the stages before it left."""
import importlib.util
import os

import numpy as np
import pytest

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a GPU", allow_module_level=True)

from gpu_util import cpu, say  # noqa: E402
from oracle import ends as E  # noqa: E402

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def example():
    spec = importlib.util.spec_from_file_location("compressed_language_step",
                                                  os.path.join(ROOT, "examples", "compressed_language_step.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_example_runs_and_its_gradients_are_right(dtype):
    tokens, dim, hidden, vocab, lr = 60, 24, 32, 90, 0.02
    f32 = dtype == torch.float32
    half = 2.0 ** -24 if f32 else 2.0 ** -8
    state = {}

    def seen(step, leaves, ps):
        w1, w2, b = (cpu(p) for p in leaves)
        if step:  # the weights that the step before left
            for i, now in ((0, w1), (1, w2)):
                want, m = E.muon_step(state["w"][i], state["mhat"][i], state["m"][i], lr, 0.9, True, 0.0,
                                      max(1.0, now.shape[0] / now.shape[1]) ** 0.5)
                state["m"][i] = m
                # (one fp16 piece: 4e-3 of an update at most on these sizes; the weights' rounding)
                off = np.linalg.norm(now - want)
                assert off <= (1e-5 if f32 else 4e-3) * np.linalg.norm(want - state["w"][i]) + 2 * half * np.linalg.norm(want)
        else:
            state["m"] = [np.zeros_like(w1), np.zeros_like(w2)]
        state["w"], state["mhat"] = [w1, w2], [cpu(ps.view(ps.mhat, i)).copy() for i in range(2)]
        if step > 1:
            return
        g = torch.Generator(device="cuda:0")
        g.manual_seed(0)
        x = torch.randn(tokens, dim, generator=g, device="cuda:0").to(dtype)
        y = torch.randint(0, vocab, (tokens,), generator=g, device="cuda:0").cpu().numpy()
        y[::10] = -100
        # the head's gradients from the hidden states as the type holds them
        h = cpu(torch.relu(x @ leaves[0].detach().t()))
        _, _, dh, dw, db = E.cross_entropy(h, w2, y, b, mean=True)
        for name, got, want in (("dw", leaves[1].grad, dw), ("db", leaves[2].grad, db)):
            # (E's, G's and the result's roundings, and the factor of the incoming 1; fp32: its sums)
            tol = 2e-5 if f32 else 3 * half
            off = np.linalg.norm(cpu(got) - want) / np.linalg.norm(want)
            say(f"[example] step {step} {dtype} {name}: off {off:.2e}")
            assert off <= tol
        dw1 = (dh * (h > 0)).T @ cpu(x)
        off = np.linalg.norm(cpu(leaves[0].grad) - dw1) / np.linalg.norm(dw1)
        assert off <= (2e-5 if f32 else 6 * half)

    losses = example().train(steps=4, tokens=tokens, dim=dim, hidden=hidden, vocab=vocab, lr=lr, dtype=dtype, seen=seen)
    assert len(losses) == 4 and all(np.isfinite(losses))

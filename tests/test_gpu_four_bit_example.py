"""The example that runs the 4-bit products, the clip and the compression
together: its loss falls."""
import importlib.util
import os

import pytest

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a GPU", allow_module_level=True)

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_training_steps_lower_the_loss():
    spec = importlib.util.spec_from_file_location("four_bit_training_step",
                                                  os.path.join(ROOT, "examples", "four_bit_training_step.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    losses = mod.train(steps=60)
    assert all(l == l for l in losses)
    assert sum(losses[-5:]) / 5 < 0.5 * losses[0], losses

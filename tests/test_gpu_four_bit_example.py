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


def test_hook_rounds_the_factors_columns_and_nothing_else():
    import numpy as np

    from oracle import microscaling as MX
    from rank_gradient_compression_amd import torch_api as T

    spec = importlib.util.spec_from_file_location("four_bit_training_step",
                                                  os.path.join(ROOT, "examples", "four_bit_training_step.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    ps = T.PowerSGD([(70, 45), (33,), (130, 97), (5,)], 3, device="cuda:0")
    hook = mod.four_bit_hook(ps)
    g = torch.Generator(device="cuda:0")
    g.manual_seed(4)
    for buf, factor in ((ps.p, ps.p_hat), (ps.q, ps.q_of)):
        buf.copy_(torch.randn(buf.shape, generator=g, device="cuda:0"))
        want = buf.clone()
        for i in ps.compressed():
            f = factor(i)  # a view of buf, a column contiguous
            at = f.storage_offset()
            cols = MX.round_values(f.t().cpu().double().numpy())
            want[at:at + cols.size] = torch.from_numpy(cols.astype(np.float32)).reshape(-1).to("cuda:0")
        assert hook(buf.data_ptr(), buf.numel(), torch.cuda.current_stream().cuda_stream) == 0
        assert torch.equal(buf, want)
    assert len(ps.compressed()) == 2
    ps.close()

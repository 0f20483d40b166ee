"""Edges of the vocabulary cross entropy on the GPU, against the definition in 64
bits: masks, offsets that all logits share, rows and weights of very different
sizes, many blocks of tokens, many tokens.

Bounds as in test_gpu_xent.py where nothing else is said (u = 2^-24)."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a GPU", allow_module_level=True)

from gpu_util import say  # noqa: E402
from test_gpu_xent import BF16, DEV, F16, F32, OUT, Reference, U, check, close, inputs  # noqa: E402
from rank_gradient_compression_amd import torch_api as T  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("mask", [-1e9, -1e10, None])
@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("t", [5, 200])
def test_finite_masks_of_whole_segments(t, dtype, mask):
    """A large negative bias (None: the type's lowest value) over whole segments of
    words and over the padded end of the vocabulary: the words' probabilities are
    exp of less than -60000, zero, so all is as over the words that are left."""
    v, d = 600, 40
    x, w, y, b = inputs(t, v, d, dtype, True, seed=40, ignored=0.1)
    lowest = torch.finfo(dtype).min
    gone = torch.zeros(v, dtype=torch.bool, device=DEV)
    gone[64:192] = gone[320:352] = gone[576:] = True
    b[gone] = max(mask or lowest, lowest)
    live = (~gone).nonzero().flatten()
    y = torch.where(y >= 0, live[y.clamp(min=0) % len(live)], y)
    place = torch.cumsum((~gone).long(), 0) - 1
    say(f"[xent] masks {t} {dtype} {mask}")
    loss, lse, dx, dw, db = T.cross_entropy_train(x, w, y, b)
    ref = Reference(x, w[live], torch.where(y >= 0, place[y.clamp(min=0)], y), b[live], mean=True)
    check(ref, loss, lse, dx, dw[live], db[live])
    assert not dw[gone].any() and not db[gone].any()
    again = T.cross_entropy(x, w, y, b)
    assert torch.equal(again[0], loss) and torch.equal(again[1], lse)

"""One worker's training steps of a small two-layer network whose matrix
products run on microscaled 4-bit operands, and whose gradients are clipped by
their global norm and compressed with PowerSGD:

  forward / backward   mx_linear_train: y = Q(x) Q(w)^T, both gradients from
                       4-bit operands quantised along the axes they sum over,
                       the incoming gradient rounded stochastically
  clip                 GradientClip: the norm over all gradients, and the
                       clipped gradients written into the flat buffer
  compress             PowerSGD.compress at rank 4, error feedback, SGD with
                       momentum fused into the residual pass; the factors are
                       sent as 4-bit codes: the hook rounds P and Q in place
                       (values of the codes) before an all-reduce would sum them

Run on the GPU:  python examples/four_bit_training_step.py [--steps N]
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from rank_gradient_compression_amd import binding as B  # noqa: E402
from rank_gradient_compression_amd import torch_api as T  # noqa: E402


def train(steps: int = 60, tokens: int = 700, d_in: int = 650, hidden: int = 512, d_out: int = 64, rank: int = 4,
          max_norm: float = 1.0, lr: float = 0.05, device="cuda:0", seed: int = 0):
    """Losses of every step on a fixed regression target."""
    g = torch.Generator(device=device)
    g.manual_seed(seed)
    x = torch.randn(tokens, d_in, generator=g, device=device)
    target = torch.tanh(x @ torch.randn(d_in, d_out, generator=g, device=device) / d_in ** 0.5)
    shapes = [(hidden, d_in), (hidden,), (d_out, hidden), (d_out,)]
    ps = T.PowerSGD(shapes, rank, device=device)
    ps.init_q(seed)
    params = torch.zeros_like(ps.grads)
    momentum = torch.zeros_like(ps.grads)
    w1, b1, w2, b2 = (ps.view(params, i) for i in range(4))
    for w in (w1, w2):
        w.copy_(torch.randn(w.shape, generator=g, device=device) / w.shape[1] ** 0.5)
    leaves = [t.view(s).detach().requires_grad_(True) for t, s in zip((w1, b1, w2, b2), shapes)]
    flat = [ps.view(ps.grads, i).view(-1) for i in range(4)]
    clip = None

    def send_as_four_bits(buf: int, count: int, stream: int) -> int:
        """Aggregation hook: the buffer as rows of 32-value blocks, rounded in
        place; a multi-worker hook would exchange the codes and average."""
        whole = count // 32 * 32
        B.psgd_mx_quantize(buf, B.PSGD_DTYPE_F32, 1, whole, whole, 0, 0, 0, 0, 0, buf, whole, stream)
        return 0

    hook = B.make_hook(send_as_four_bits)
    losses = []
    for _ in range(steps):
        for p in leaves:
            p.grad = None
        h = torch.relu(T.mx_linear_train(x, leaves[0], generator=g) + leaves[1])
        y = T.mx_linear_train(h, leaves[2], generator=g) + leaves[3]
        loss = torch.nn.functional.mse_loss(y, target, reduction="sum") / tokens
        loss.backward()
        grads = [p.grad.contiguous().view(-1) for p in leaves]
        if clip is None:
            clip = T.GradientClip(grads, flat)
        else:
            clip.bind(grads, flat)
        clip.clip(max_norm)
        ps.compress(mhat=True, hook=hook, params=params, sgd_buf=momentum, sgd_lr=lr, sgd_momentum=0.9)
        losses.append(float(loss.detach()))
    ps.close()
    return losses


def main() -> None:
    ap = argparse.ArgumentParser()
    ap.add_argument("--steps", type=int, default=60)
    args = ap.parse_args()
    losses = train(args.steps)
    print(f"loss {losses[0]:.4f} -> {losses[-1]:.4f} in {len(losses)} steps")


if __name__ == "__main__":
    main()

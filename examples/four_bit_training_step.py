"""One worker's training steps of a small two-layer network whose matrix
products run on microscaled 4-bit operands, and whose gradients are clipped by
their global norm and compressed with PowerSGD:

  forward / backward   mx_linear_train: y = Q(x) Q(w)^T, both gradients from
                       4-bit operands quantised along the axes they sum over,
                       the incoming gradient rounded stochastically
  clip                 GradientClip: the norm over all gradients, and the
                       clipped gradients written into the flat buffer
  compress             PowerSGD.compress at rank 4, error feedback, SGD with
                       momentum fused into the residual pass; the hook rounds
                       every column of P and Q to 4-bit codes' values before
                       an all-reduce would sum them

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


def four_bit_hook(ps):
    """Aggregation hook that rounds each column of each factor, in place, to the
    values of 4-bit codes with blocks of 32 along the column; a multi-worker
    hook would exchange the codes and average.  Whatever error this makes stays
    in the error memory.  The pass-through values behind P's factors have none,
    so they are left as they are."""

    def hook(buf: int, count: int, stream: int) -> int:
        is_p = buf == ps.p.data_ptr()
        for i in ps.compressed():
            _, _, p_off, q_off = ps.tensors[i]
            at, n = buf + 4 * (p_off if is_p else q_off), ps.views[i][0 if is_p else 1]
            B.psgd_mx_quantize(at, B.PSGD_DTYPE_F32, ps.rank, n, n, 0, 0, 0, 0, 0, at, n, stream)
        return 0

    return hook


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

    hook = B.make_hook(four_bit_hook(ps))
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

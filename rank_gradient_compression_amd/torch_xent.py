"""Softmax cross entropy over a large vocabulary, over PyTorch tensors.

Buffers and pointers only, like the other convenience layers: the computation
runs in libpsgd.so, on the current stream of the tensors' device.
"""
from __future__ import annotations

from typing import Optional

import torch

from . import binding as B
from .torch_ops import _as_matrix, _call, _dtype, _matrix, _result, _scratch, _written


def _arguments(x, w, targets, bias, ignore_index: int):
    """(the call's arguments, loss, lse), checked."""
    t, d, ldx = _matrix(x, "x")
    v, dw, ldw = _matrix(w, "w")
    device = x.device
    if d != dw or device != w.device or x.dtype != w.dtype:
        raise ValueError(f"x has {d} columns of {x.dtype} on {device}, the weights {dw} of {w.dtype} on {w.device}")
    if targets.dtype != torch.int64 or targets.shape != (t,) or targets.device != device:
        raise ValueError(f"targets must be {t} int64 values on {device}")
    if bias is not None and (bias.shape != (v,) or bias.dtype != x.dtype or bias.device != device
                             or not bias.is_contiguous()):
        raise ValueError(f"bias must be {v} contiguous values of {x.dtype} on {device}")
    targets = targets.contiguous()
    stats = torch.empty(2, t, dtype=torch.float32, device=device)
    a = B.psgd_xent_t()
    a.tokens, a.vocab, a.dim, a.dtype = t, v, d, _dtype(x)
    a.x, a.ldx, a.w, a.ldw = x.data_ptr(), ldx, w.data_ptr(), ldw
    a.bias = 0 if bias is None else bias.data_ptr()
    a.targets, a.ignore_index = targets.data_ptr(), ignore_index
    loss, lse = stats[0], stats[1]
    a.loss, a.lse, a.scale = loss.data_ptr(), lse.data_ptr(), 1.0
    return a, loss, lse, targets


def _run(fn, a, train: bool, device) -> None:
    need = B.psgd_xent_workspace(a, train)
    ws, ptr = _scratch(need, device)
    _call(device, fn, a, ptr, need)


def cross_entropy(x: torch.Tensor, w: torch.Tensor, targets: torch.Tensor, bias: Optional[torch.Tensor] = None,
                  ignore_index: int = -100):
    """(loss, lse), float32 per token: lse = log sum exp(x w^T + bias) over the
    vocabulary and loss = lse - the target's logit (psgd_xent_forward).  x:
    tokens x dim, w: vocab x dim, targets: int64; a token whose target is
    negative or `ignore_index` has loss 0.  For scoring and evaluation, from
    single tokens on: no gradient flows (linear_cross_entropy has one)."""
    a, loss, lse, targets = _arguments(x, w, targets, bias, ignore_index)
    if a.tokens:
        _run(B.psgd_xent_forward, a, False, x.device)
    return loss, lse


def cross_entropy_train(x: torch.Tensor, w: torch.Tensor, targets: torch.Tensor, bias: Optional[torch.Tensor] = None,
                        weights: Optional[torch.Tensor] = None, reduction: str = "mean", scale: float = 1.0,
                        ignore_index: int = -100, dw: Optional[torch.Tensor] = None,
                        dbias: Optional[torch.Tensor] = None, accumulate: bool = False, need_dx: bool = True,
                        need_dw: bool = True, need_dbias: bool = True):
    """(loss, lse, dx, dw, dbias): cross_entropy and the gradients of
    scale * sum_t weights_t loss_t, divided by the number of tokens that are not
    ignored for reduction "mean" ("sum": not divided) (psgd_xent_train).

    weights  float32 per token (None: ones), for example incoming gradients
    dw       the matrix to write, of any of the three types (None: a new one of
             w's type), for example a view of PowerSGD.grads; dbias alike, of
             x's type; accumulate: both are added to what they hold
    A gradient that is not needed is None and costs nothing."""
    a, loss, lse, targets = _arguments(x, w, targets, bias, ignore_index)
    device = x.device
    if reduction not in ("mean", "sum"):
        raise ValueError('reduction must be "mean" or "sum"')
    if weights is not None:
        if weights.dtype != torch.float32 or weights.shape != (a.tokens,) or weights.device != device:
            raise ValueError(f"weights must be {a.tokens} float32 values on {device}")
        weights = weights.contiguous()
        a.weights = weights.data_ptr()
    if accumulate and ((need_dw and dw is None) or (need_dbias and bias is not None and dbias is None)):
        raise ValueError("accumulate needs dw, and dbias where there is a bias")
    a.scale, a.mean, a.accumulate = scale, reduction == "mean", accumulate
    dx = None
    if need_dx:
        dx = torch.empty(a.tokens, a.dim, dtype=x.dtype, device=device)
        a.dx, a.lddx = dx.data_ptr(), a.dim
    if need_dw:
        dw, a.lddw = _result(dw, a.vocab, a.dim, w.dtype, device)
        a.dw, a.dw_dtype = dw.data_ptr(), _dtype(dw)
    else:
        dw = None
    if need_dbias and bias is not None:
        if dbias is None:
            dbias = torch.empty(a.vocab, dtype=x.dtype, device=device)
        elif dbias.shape != (a.vocab,) or dbias.dtype != x.dtype or dbias.device != device or not dbias.is_contiguous():
            raise ValueError(f"dbias must be {a.vocab} contiguous values of {x.dtype} on {device}")
        a.dbias = dbias.data_ptr()
    else:
        dbias = None
    _run(B.psgd_xent_train, a, True, device)
    _written([g for g in (dw, dbias) if g is not None])
    return loss, lse, dx, dw, dbias


def _total(loss: torch.Tensor, targets: torch.Tensor, mean: bool, ignore_index: int) -> torch.Tensor:
    """The losses' sum or mean (psgd_xent_total)."""
    out = torch.empty((), dtype=torch.float32, device=loss.device)
    targets = targets.contiguous()
    ws, ptr = _scratch(B.PSGD_XENT_TOTAL_BYTES, loss.device)
    _call(loss.device, B.psgd_xent_total, loss.data_ptr(), targets.data_ptr(), loss.numel(), ignore_index, mean,
          out.data_ptr(), ptr, B.PSGD_XENT_TOTAL_BYTES)
    return out


def _times(g: torch.Tensor, factor: torch.Tensor) -> torch.Tensor:
    """A gradient times one float32 value on its device (psgd_xent_scale)."""
    out = torch.empty_like(g)
    _call(g.device, B.psgd_xent_scale, g.data_ptr(), _dtype(g), g.numel(), factor.data_ptr(), out.data_ptr())
    return out


class _CrossEntropyFunction(torch.autograd.Function):
    """mean and sum: the gradients are formed with the loss, from the same
    logits, and the backward pass multiplies them by the one incoming value.
    none: the incoming gradient has a value per token, so the backward pass forms
    the logits again.  float16 too, whatever the reduction: its gradients may be
    too small or too large for the type until the incoming value (a loss scale of
    65536, say) is part of them."""

    @staticmethod
    def forward(ctx, x, w, bias, targets, reduction, ignore_index, grad):
        xm, wm, y = _as_matrix(x), _as_matrix(w), targets.reshape(-1)
        b = None if bias is None else bias.contiguous()
        ctx.x_shape, ctx.reduction, ctx.ignore_index = x.shape, reduction, ignore_index
        # (needs_input_grad goes by the inputs alone, under no_grad too)
        need = tuple(grad and n for n in ctx.needs_input_grad[:3])
        ctx.late = reduction == "none" or x.dtype == torch.float16
        if ctx.late or not any(need):
            loss, _ = cross_entropy(xm, wm, y, b, ignore_index)
            if any(need):
                ctx.save_for_backward(x, w, bias, y)  # (the inputs themselves: what is written to them is noticed)
            if reduction == "none":
                return loss.view(targets.shape)
        else:
            loss, _, dx, dw, db = cross_entropy_train(xm, wm, y, b, reduction=reduction, ignore_index=ignore_index,
                                                      need_dx=need[0], need_dw=need[1], need_dbias=need[2])
            ctx.save_for_backward(dx, dw, db)
        return _total(loss, y, reduction == "mean", ignore_index)

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, grad):
        need = ctx.needs_input_grad[:3]
        if ctx.late:
            x, w, bias, y = ctx.saved_tensors
            b = None if bias is None else bias.contiguous()
            reduction = "mean" if ctx.reduction == "mean" else "sum"
            weights = grad.float().reshape(-1).expand(y.numel())
            _, _, dx, dw, db = cross_entropy_train(_as_matrix(x), _as_matrix(w), y, b, weights=weights, reduction=reduction,
                                                   ignore_index=ctx.ignore_index, need_dx=need[0], need_dw=need[1],
                                                   need_dbias=need[2])
        else:
            dx, dw, db = (None if g is None else _times(g, grad.float()) for g in ctx.saved_tensors)
        return None if dx is None else dx.view(ctx.x_shape), dw, db, None, None, None, None


def linear_cross_entropy(x: torch.Tensor, w: torch.Tensor, targets: torch.Tensor, bias: Optional[torch.Tensor] = None,
                         reduction: str = "mean", ignore_index: int = -100) -> torch.Tensor:
    """The loss of x w^T + bias under autograd: x of any leading shape, targets of
    that shape, w vocab x dim, any strides (copied where their rows are not
    contiguous), one type; under autocast all are taken in autocast's.  reduction:
    "mean" over the tokens that are not ignored (0 where all are), "sum", or "none" (a
    value per token)."""
    if reduction not in ("mean", "sum", "none"):
        raise ValueError('reduction must be "mean", "sum" or "none"')
    if targets.shape != x.shape[:-1]:
        raise ValueError(f"targets of shape {tuple(targets.shape)} for x of shape {tuple(x.shape)}")
    if torch.is_autocast_enabled(x.device.type):
        dtype = torch.get_autocast_dtype(x.device.type)
        x, w, bias = x.to(dtype), w.to(dtype), None if bias is None else bias.to(dtype)
    return _CrossEntropyFunction.apply(x, w, bias, targets, reduction, ignore_index, torch.is_grad_enabled())

"""Orthogonalised updates over PyTorch tensors: one matrix, or the optimiser step
around a list of them.

Buffers and pointers only, like the other convenience layers: the computation
runs in libpsgd.so, on the current stream of the tensors' device.
"""
from __future__ import annotations

import math
from typing import Optional, Sequence, Tuple

import torch

from . import binding as B
from .torch_ops import _call, _dtype, _matrix, _raw_stream, _result, _scratch, _written

_COEFFICIENTS = (3.4445, -4.7750, 2.0315)


def _opts(lr, momentum, weight_decay, coefficients, eps, steps, nesterov, pieces) -> B.psgd_muon_opts_t:
    a, b, c = coefficients
    return B.psgd_muon_opts_t(lr, momentum, weight_decay, a, b, c, eps, steps, nesterov, pieces)


def orthogonalize(x: torch.Tensor, out: Optional[torch.Tensor] = None, steps: int = 5,
                  coefficients: Tuple[float, float, float] = _COEFFICIENTS, eps: float = 1e-7,
                  pieces: int = 0) -> torch.Tensor:
    """x with its singular values brought to about 1 by Newton-Schulz steps
    (psgd_muon_step on one matrix): X = x / (||x|| + eps), then X <- a X +
    (b A + c A^2) X with A = X X^T.  out: of x's shape and any of the three types
    (None: a new one of x's type; x itself: in place).  pieces: 1 for bfloat16's
    precision, 2 for float32's, 0 goes by out's type (a bfloat16 matrix with a side of
    at most 48 takes 2)."""
    rows, cols, ld = _matrix(x, "x")
    out, ldo = _result(out, rows, cols, x.dtype, x.device)
    t = (B.psgd_muon_tensor_t * 1)()
    t[0].grad, t[0].ldg, t[0].grad_dtype = x.data_ptr(), ld, _dtype(x)
    t[0].update, t[0].ldu, t[0].update_dtype = out.data_ptr(), ldo, _dtype(out)
    t[0].rows, t[0].cols = rows, cols
    opts = _opts(0.0, 0.0, 0.0, coefficients, eps, steps, False, pieces)
    need = B.psgd_muon_workspace(t, opts)
    ws, ptr = _scratch(need, x.device)
    _call(x.device, B.psgd_muon_step, t, opts, ptr, need)
    _written([out])
    return out


class Muon:
    """The optimiser step over a list of matrices: momentum, orthogonalised
    update, decay, new weights, in place.

    params   matrices (float32, bfloat16 or float16, rows contiguous)
    grads    one matrix per parameter and of its shape, of any of the three
             types, for example the matrices' views of PowerSGD.mhat
    scale    what a matrix's learning rate is multiplied by: "spectral",
             sqrt(max(1, rows / cols)); "rms", 0.2 sqrt(max(rows, cols)), which
             gives every update an element's size of about 0.2; or a number
    momentum_buffers  contiguous float32 matrices to start from (None: zeros)

    The handle keeps the tensors' addresses; bind() replaces them when they
    move.  Its calls share its momentum and workspace and take effect in the order
    in which they are made: a step on another stream than the one before it waits
    for that stream.  (Not while a graph is captured: there the caller orders the
    replays.)"""

    def __init__(self, params: Sequence[torch.Tensor], grads: Sequence[torch.Tensor], lr: float = 0.02,
                 momentum: float = 0.95, nesterov: bool = True, weight_decay: float = 0.0, steps: int = 5,
                 coefficients: Tuple[float, float, float] = _COEFFICIENTS, eps: float = 1e-7, scale="spectral",
                 momentum_buffers: Optional[Sequence[torch.Tensor]] = None, pieces: int = 0):
        params, grads = list(params), list(grads)
        self.scale = scale
        self.device = params[0].device if params else torch.device("cuda", torch.cuda.current_device())
        self.opts = _opts(lr, momentum, weight_decay, coefficients, eps, steps, nesterov, pieces)
        if momentum_buffers is None:
            momentum_buffers = [torch.zeros(p.shape, dtype=torch.float32, device=p.device) for p in params]
        self.momentum = list(momentum_buffers)
        table = self._table(params, grads)
        self.ws_bytes = B.psgd_muon_workspace(table, self.opts)
        self._last = torch.cuda.current_stream(self.device)  # the stream of the last call
        self.workspace, self._ws = _scratch(self.ws_bytes, self.device)
        self.params, self.grads, self.table = params, grads, table

    def _factor(self, rows: int, cols: int) -> float:
        if self.scale == "spectral":
            return math.sqrt(max(1.0, rows / max(1, cols)))
        if self.scale == "rms":
            return 0.2 * math.sqrt(max(rows, cols))
        return float(self.scale)

    def _table(self, params, grads):
        if not len(params) == len(grads) == len(self.momentum):
            raise ValueError(f"{len(params)} parameters, {len(grads)} gradients, {len(self.momentum)} momentum buffers")
        table = (B.psgd_muon_tensor_t * len(params))()
        for t, p, g, m in zip(table, params, grads, self.momentum):
            t.rows, t.cols, t.ldp = _matrix(p, "a parameter")
            rows, cols, t.ldg = _matrix(g, "a gradient")
            if (rows, cols) != (t.rows, t.cols) or not self.device == p.device == g.device == m.device:
                raise ValueError(f"a parameter of {t.rows} x {t.cols} on {p.device} and a gradient of {rows} x {cols} "
                                 f"on {g.device}")
            if m.shape != p.shape or m.dtype != torch.float32 or not m.is_contiguous():
                raise ValueError(f"a momentum buffer must be a contiguous float32 matrix of {t.rows} x {t.cols}")
            t.param, t.grad, t.momentum = p.data_ptr(), g.data_ptr(), m.data_ptr()
            t.param_dtype, t.grad_dtype = _dtype(p), _dtype(g)
            t.lr_scale = self._factor(t.rows, t.cols)
        return table

    def bind(self, params: Sequence[torch.Tensor], grads: Sequence[torch.Tensor]) -> None:
        """New tensors of the same shapes (and the parameters' types).  Where it
        raises, the handle keeps the tensors that it had."""
        params, grads = list(params), list(grads)
        if [(p.shape, p.dtype) for p in params] != [(p.shape, p.dtype) for p in self.params]:
            raise ValueError("the parameters differ in shape or type from the handle's")
        table = self._table(params, grads)
        self.params, self.grads, self.table = params, grads, table

    def _order(self) -> None:
        """What follows on the current stream comes after the handle's last call."""
        if _raw_stream is not None and _raw_stream(self.device.index) == self._last.cuda_stream:
            return
        stream = torch.cuda.current_stream(self.device)
        if stream == self._last:
            return
        with torch.cuda.device(self.device):
            if torch.cuda.is_current_stream_capturing():
                return
        stream.wait_stream(self._last)
        for t in (self.workspace, *self.momentum):
            t.record_stream(stream)
        self._last = stream

    def step(self, lr: Optional[float] = None) -> None:
        """One step (psgd_muon_step) with the gradients' present values; lr: from
        this step on (where it raises, the handle keeps the one that it had)."""
        kept = self.opts.lr
        if lr is not None:
            self.opts.lr = lr
        self._order()
        try:
            _call(self.device, B.psgd_muon_step, self.table, self.opts, self._ws, self.ws_bytes)
        except B.PsgdError:
            self.opts.lr = kept
            raise
        _written(self.params)

"""The gradient clip and the microscaled 4-bit operands over PyTorch tensors.

Like the PowerSGD class it allocates buffers and marshals pointers; the
computation runs in libpsgd.so, on the current stream of the tensors' device.
"""
from __future__ import annotations

import functools
import math
import warnings
from typing import Optional, Sequence, Tuple

import torch

from . import binding as B

_DTYPES = {torch.float32: B.PSGD_DTYPE_F32, torch.bfloat16: B.PSGD_DTYPE_BF16, torch.float16: B.PSGD_DTYPE_F16}


def _dtype(t: torch.Tensor) -> int:
    d = _DTYPES.get(t.dtype)
    if d is None:
        raise ValueError(f"expected float32, bfloat16 or float16, got {t.dtype}")
    return d


def _stream(device: torch.device) -> int:
    return torch.cuda.current_stream(device).cuda_stream


# Small calls are bound by the host, so the common path (the tensors' device is
# the current one) asks PyTorch's C layer for the device and the raw stream
# where it offers them, instead of building Stream objects and contexts.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


def _call(device: torch.device, fn, *args) -> None:
    """fn(*args, stream) with `device` current, on its current stream."""
    index = device.index
    if _raw_stream is not None and index == _current_device():
        fn(*args, _raw_stream(index))
    else:
        with torch.cuda.device(device):
            fn(*args, _stream(device))


@functools.lru_cache(maxsize=4096)
def _linear_workspace(m: int, n: int, k: int, x_dtype: int) -> int:
    return B.psgd_mx_linear_workspace(m, n, k, x_dtype)


@functools.lru_cache(maxsize=4096)
def _train_workspace(m: int, n: int, k: int) -> int:
    return B.psgd_mx_train_workspace(m, n, k)


def _written(tensors) -> None:
    """Tensors of the caller's that a call of the library has written: a backward
    pass that saved one of them raises, as behind an operation of PyTorch's."""
    torch.autograd.graph.increment_version([t for t in tensors if not t.is_inference()])


def _scratch(nbytes: int, device: torch.device):
    """(tensor, address) of nbytes of scratch; (None, 0) for none."""
    if nbytes == 0:
        return None, 0
    ws = torch.empty(nbytes, dtype=torch.uint8, device=device)
    return ws, ws.data_ptr()


def _matrix(x: torch.Tensor, name: str):
    """(rows, columns, row stride) of a row-major matrix on the GPU."""
    st = x.stride()
    if len(st) != 2:
        raise ValueError(f"{name} must be a matrix, got {len(st)} dimensions")
    if not x.is_cuda:
        raise ValueError(f"{name} must be on the GPU")
    rows, cols = x.shape
    if st[1] != 1 and cols > 1:
        raise ValueError(f"{name} must have contiguous rows")
    return rows, cols, (st[0] if rows > 1 else max(1, cols))


# ------------------------------------------------------------------- the clip
class GradientClip:
    """Global norm of a list of gradients, and the clipped gradients.

    grads  contiguous tensors (float32, bfloat16 or float16, any mixture)
    outs   where the clipped gradients go: one contiguous tensor per gradient
           and of its size, of any of the three types -- for example the
           tensor's view of PowerSGD.grads, so that clipping also packs the
           gradients for the compression; None clips in place

    The handle keeps the addresses; bind() replaces them when the tensors move.

    A handle's calls share its workspace and take effect in the order in which
    they are made: a call on another stream than the one before it waits for
    that stream.  (Not while a graph is captured: there the caller orders the
    replays.)  The gradients themselves are read and the outputs written on the
    current stream, like any tensors.
    """

    def __init__(self, grads: Sequence[torch.Tensor], outs: Optional[Sequence[torch.Tensor]] = None):
        self.handle = 0
        grads = list(grads)
        outs = grads if outs is None else list(outs)
        self._check(grads, outs)
        self.device = grads[0].device if grads else torch.device("cuda", torch.cuda.current_device())
        self._numel = [g.numel() for g in grads]
        self._in, self._out = [_dtype(g) for g in grads], [_dtype(o) for o in outs]
        self.handle = B.psgd_clip_create(self._numel, self._in, self._out)
        self.ws_bytes = B.psgd_clip_workspace(self.handle)
        self._last = torch.cuda.current_stream(self.device)  # the stream of the last call
        with torch.cuda.device(self.device):
            self.workspace = torch.empty(self.ws_bytes, dtype=torch.uint8, device=self.device)
            B.psgd_clip_workspace_init(self.handle, self.workspace.data_ptr(), self.ws_bytes, _stream(self.device))
            self._bind(grads, outs)

    @staticmethod
    def _check(grads, outs) -> None:
        if len(grads) != len(outs):
            raise ValueError(f"{len(grads)} gradients but {len(outs)} outputs")
        for t in (*grads, *outs):
            if not t.is_cuda or not t.is_contiguous() or t.device != grads[0].device:
                raise ValueError("gradients and outputs must be contiguous tensors on one GPU")
        for g, o in zip(grads, outs):
            if g.numel() != o.numel():
                raise ValueError(f"an output of {o.numel()} elements for a gradient of {g.numel()}")

    def _order(self) -> None:
        """What follows on the current stream comes after the handle's last call."""
        index = self.device.index
        if _raw_stream is not None and _raw_stream(index) == self._last.cuda_stream:
            return
        stream = torch.cuda.current_stream(self.device)
        if stream == self._last:
            return
        with torch.cuda.device(self.device):
            if torch.cuda.is_current_stream_capturing():
                return
        stream.wait_stream(self._last)
        self.workspace.record_stream(stream)
        self._last = stream

    def _bind(self, grads, outs) -> None:
        self._order()
        B.psgd_clip_bind(self.handle, [g.data_ptr() for g in grads], [o.data_ptr() for o in outs],
                         self.workspace.data_ptr(), self.ws_bytes, _stream(self.device))
        # Kept alive: the workspace holds their addresses.  After the call, since
        # a refused one leaves the old addresses there.
        self.grads, self.outs = grads, outs

    def bind(self, grads: Sequence[torch.Tensor], outs: Optional[Sequence[torch.Tensor]] = None) -> None:
        """New tensors of the same sizes and types (psgd_clip_bind).  Where it
        raises, the handle keeps the tensors that it had."""
        grads = list(grads)
        outs = grads if outs is None else list(outs)
        self._check(grads, outs)
        if ([g.numel() for g in grads] != self._numel or [_dtype(g) for g in grads] != self._in
                or [_dtype(o) for o in outs] != self._out):
            raise ValueError("the tensors differ in size or type from the handle's")
        if grads and grads[0].device != self.device:
            raise ValueError("the tensors are on another GPU than the handle's workspace")
        with torch.cuda.device(self.device):
            self._bind(grads, outs)

    def _run(self, fn, max_norm: float, scale: float) -> torch.Tensor:
        stats = torch.empty(2 + len(self._numel), dtype=torch.float32, device=self.device)
        self._order()
        _call(self.device, fn, self.handle, max_norm, scale, stats.data_ptr(), self.workspace.data_ptr(),
              self.ws_bytes)
        return stats

    def norm(self, max_norm: float = float("inf"), scale: float = 1.0) -> torch.Tensor:
        """float32 (2 + n) on the device: the global norm of scale * grads, the
        coefficient that max_norm asks for, then every tensor's norm."""
        return self._run(B.psgd_clip_norm, max_norm, scale)

    def clip(self, max_norm: float, scale: float = 1.0) -> torch.Tensor:
        """The same, and outs = scale * coefficient * grads."""
        return self._run(B.psgd_clip_apply, max_norm, scale)

    def close(self) -> None:
        if self.handle:
            B.psgd_clip_destroy(self.handle)
            self.handle = 0

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


# ------------------------------------------------ microscaled 4-bit operands
class MxTensor:
    """A rows x cols operand: codes and scales as psgd.h lays them out."""

    __slots__ = ("rows", "cols", "buf", "device", "codes_ptr", "scales_ptr")

    def __init__(self, rows: int, cols: int, device, buf: Optional[torch.Tensor] = None):
        """Uninitialised operand: one allocation, the scales behind the codes
        at a multiple of 256 bytes.  buf: the buffer of an operand of this size
        instead."""
        off = (rows * ((cols + 31) >> 5) * 16 + 255) & ~255
        self.rows, self.cols = rows, cols
        if buf is None:
            buf = torch.empty(off + ((rows + 31) >> 5) * ((cols + 255) >> 8) * 256, dtype=torch.uint8, device=device)
        self.buf = buf
        self.device = buf.device
        self.codes_ptr = ptr = buf.data_ptr()
        self.scales_ptr = ptr + off

    @staticmethod
    def _scales_at(rows: int, cols: int) -> int:
        return (rows * ((cols + 31) // 32) * 16 + 255) & ~255

    @property
    def shape(self) -> Tuple[int, int]:
        return self.rows, self.cols

    @property
    def codes(self) -> torch.Tensor:
        """The codes' bytes, rows x (16 per block)."""
        n = (self.cols + 31) // 32 * 16
        return self.buf[:self.rows * n].view(self.rows, n)

    @property
    def scales(self) -> torch.Tensor:
        """The scales' bytes, in the tiles of psgd.h."""
        return self.buf[self._scales_at(self.rows, self.cols):]


def _rand(rand: torch.Tensor, x: torch.Tensor) -> int:
    if rand.dtype != torch.uint8 or rand.shape != x.shape or not rand.is_contiguous() or rand.device != x.device:
        raise ValueError("rand must be a contiguous uint8 matrix of x's shape on x's device")
    return rand.data_ptr()


def _quantize(x, rand, want_row: bool, want_col: bool, values):
    rows, cols, ld = _matrix(x, "x")
    dtype, device = _dtype(x), x.device
    ptr, ldv = 0, 0
    if values is not None:
        vr, vc, ldv = _matrix(values, "values")
        if vr != rows or vc != cols or values.dtype != x.dtype or values.device != device:
            raise ValueError("values must have x's shape, type and device")
        ptr = values.data_ptr()
    r = 0 if rand is None else _rand(rand, x)
    q = t = None
    rc = rs = cc = cs = 0
    if want_row:
        q = MxTensor(rows, cols, device)
        rc, rs = q.codes_ptr, q.scales_ptr
    if want_col:
        t = MxTensor(cols, rows, device)
        cc, cs = t.codes_ptr, t.scales_ptr
    _call(device, B.psgd_mx_quantize, x.data_ptr(), dtype, rows, cols, ld, r, rc, rs, cc, cs, ptr, ldv)
    return q, t


def mx_quantize(x: torch.Tensor, rand: Optional[torch.Tensor] = None,
                values: Optional[torch.Tensor] = None) -> MxTensor:
    """The operand of x: blocks of 32 along its rows.  rand: uint8 of x's shape
    for stochastic rounding (None: nearest).  values: receives the values that
    the codes stand for (x's shape and type; may be x itself)."""
    return _quantize(x, rand, True, False, values)[0]


def mx_quantize_both(x: torch.Tensor, rand: Optional[torch.Tensor] = None) -> Tuple[MxTensor, MxTensor]:
    """The operands of x and of x^T (blocks along x's rows and along its
    columns), from one reading of x."""
    return _quantize(x, rand, True, True, None)


def mx_quantize_t(x: torch.Tensor, rand: Optional[torch.Tensor] = None) -> MxTensor:
    """The operand of x^T: blocks of 32 along x's columns."""
    return _quantize(x, rand, False, True, None)[1]


def mx_dequantize(q: MxTensor, dtype: torch.dtype = torch.float32, out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """The values of an operand."""
    if out is None:
        out = torch.empty(q.rows, q.cols, dtype=dtype, device=q.device)
    elif out.shape != q.shape or out.device != q.device:
        raise ValueError("out must have the operand's shape and device")
    _, _, ld = _matrix(out, "out")
    _call(q.device, B.psgd_mx_dequantize, q.codes_ptr, q.scales_ptr, q.rows, q.cols, out.data_ptr(), _dtype(out), ld)
    return out


def _result(out, m: int, n: int, dtype, device):
    """(the result's matrix, its row stride)."""
    if out is None:
        return torch.empty(m, n, dtype=dtype, device=device), max(1, n)
    rows, cols, ld = _matrix(out, "out")
    if rows != m or cols != n or out.device != device:
        raise ValueError(f"out must be a {m} x {n} matrix on {device}")
    return out, ld


def mx_product(a: MxTensor, b: MxTensor, out: Optional[torch.Tensor] = None, dtype: torch.dtype = torch.float32,
               accumulate: bool = False) -> torch.Tensor:
    """a b^T (accumulate: added to out), summed in fp32 and rounded once."""
    m, n, k, device = a.rows, b.rows, a.cols, a.device
    if k != b.cols or device != b.device:
        raise ValueError(f"operands of {k} and {b.cols} columns, on {device} and {b.device}")
    if accumulate and out is None:
        raise ValueError("accumulate needs out")
    c, ldc = _result(out, m, n, dtype, device)
    _call(device, B.psgd_mx_product, m, n, k, a.codes_ptr, a.scales_ptr, b.codes_ptr, b.scales_ptr, c.data_ptr(),
          _dtype(c), ldc, accumulate)
    return c


def mx_linear(x: torch.Tensor, w: MxTensor, out: Optional[torch.Tensor] = None,
              dtype: Optional[torch.dtype] = None) -> torch.Tensor:
    """y = Q(x) w^T for weights that were quantised once (psgd_mx_linear); y
    has x's type unless dtype or out says otherwise.  For serving: no gradient
    flows through it (mx_linear_train has one), and an x that asks for one
    draws a warning."""
    if x.requires_grad and torch.is_grad_enabled():
        warnings.warn("mx_linear gives x no gradient: use mx_linear_train, or torch.no_grad() if none is wanted",
                      stacklevel=2)
    m, k, ldx = _matrix(x, "x")
    n, device = w.rows, x.device
    if k != w.cols or device != w.device:
        raise ValueError(f"x has {k} columns on {device}, the weights {w.cols} on {w.device}")
    x_dtype = _dtype(x)
    y, ldy = _result(out, m, n, dtype or x.dtype, device)
    need = _linear_workspace(m, n, k, x_dtype)
    ws, ws_ptr = _scratch(need, device)
    _call(device, B.psgd_mx_linear, m, n, k, x.data_ptr(), x_dtype, ldx, w.codes_ptr, w.scales_ptr, y.data_ptr(),
          _dtype(y), ldy, ws_ptr, need)
    return y


def mx_linear_forward(x: torch.Tensor, w: torch.Tensor):
    """y = Q(x) Q(w)^T for full-precision weights (psgd_mx_train_forward), and
    what the backward pass needs: the operands of x^T and w^T, whose blocks run
    along the axes that its products sum over."""
    m, k, ldx = _matrix(x, "x")
    n, kw, ldw = _matrix(w, "w")
    device = x.device
    if k != kw or device != w.device:
        raise ValueError(f"x has {k} columns on {device}, the weights {kw} on {w.device}")
    dtype, w_dtype = _dtype(x), _dtype(w)
    xt, wt = MxTensor(k, m, device), MxTensor(k, n, device)
    y = torch.empty(m, n, dtype=x.dtype, device=device)
    need = _train_workspace(m, n, k)
    ws, ws_ptr = _scratch(need, device)
    _call(device, B.psgd_mx_train_forward, m, n, k, x.data_ptr(), dtype, ldx, w.data_ptr(), w_dtype, ldw, xt.codes_ptr,
          xt.scales_ptr, wt.codes_ptr, wt.scales_ptr, y.data_ptr(), dtype, max(1, n), ws_ptr, need)
    return y, (xt, wt)


def mx_linear_backward(dy: torch.Tensor, saved, rand: Optional[torch.Tensor] = None,
                       dw: Optional[torch.Tensor] = None, accumulate: bool = False, need_dx: bool = True,
                       need_dw: bool = True):
    """Gradients of the layer with the quantisers taken as the identity
    (psgd_mx_train_backward): dx = Q(dy) Q(w^T)^T in dy's type and dw =
    Q(dy^T) Q(x^T)^T in fp32, each quantised along the axis it sums over; rand
    rounds dy stochastically.  dw: the matrix to write (accumulate: to add to),
    for example a view of PowerSGD.grads.  A gradient that is not needed is
    None and costs nothing."""
    xt, wt = saved
    m, n, lddy = _matrix(dy, "dy")
    k, device = xt.rows, dy.device
    if m != xt.cols or n != wt.cols or device != xt.device:
        raise ValueError(f"dy is {m} x {n} on {device}, the forward pass was {xt.cols} x {wt.cols} on {xt.device}")
    if accumulate and dw is None:
        raise ValueError("accumulate needs dw")
    dtype = _dtype(dy)
    r = 0 if rand is None else _rand(rand, dy)
    dx, dx_ptr, dw_ptr, dw_dtype, lddw = None, 0, 0, dtype, k
    if need_dx:
        dx = torch.empty(m, k, dtype=dy.dtype, device=device)
        dx_ptr = dx.data_ptr()
    if need_dw:
        dw, lddw = _result(dw, n, k, torch.float32, device)
        dw_ptr, dw_dtype = dw.data_ptr(), _dtype(dw)
    else:
        dw = None
    need = _train_workspace(m, n, k)
    ws, ws_ptr = _scratch(need, device)
    _call(device, B.psgd_mx_train_backward, m, n, k, dy.data_ptr(), dtype, lddy, r, xt.codes_ptr, xt.scales_ptr,
          wt.codes_ptr, wt.scales_ptr, dx_ptr, dtype, max(1, k), dw_ptr, dw_dtype, lddw, accumulate, ws_ptr, need)
    return dx, dw


def _as_matrix(x: torch.Tensor) -> torch.Tensor:
    """x as a matrix with x's last axis as rows that the library reads: as it is
    where rows are contiguous and apart, else copied (transposed, every other
    column, expanded)."""
    m = x.reshape(math.prod(x.shape[:-1]), x.shape[-1])  # (no -1: an axis may be empty)
    rows, cols = m.shape
    apart = rows <= 1 or m.stride(0) >= cols
    return m if apart and (cols <= 1 or m.stride(1) == 1) else m.contiguous()


class _MxLinearFunction(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, w, stochastic, generator):
        y, (xt, wt) = mx_linear_forward(_as_matrix(x), _as_matrix(w))
        ctx.save_for_backward(xt.buf, wt.buf)  # (as tensors, which autograd lets go of behind the backward pass)
        ctx.sizes = (xt.shape, wt.shape)
        ctx.x_shape, ctx.w_dtype, ctx.stochastic, ctx.generator = x.shape, w.dtype, stochastic, generator
        return y.view(*x.shape[:-1], w.shape[0])

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dy):
        flat = _as_matrix(dy).contiguous()
        rand = None
        if ctx.stochastic:
            rand = torch.randint(0, 256, flat.shape, dtype=torch.uint8, device=flat.device, generator=ctx.generator)
        need_dx, need_dw = ctx.needs_input_grad[:2]
        saved = tuple(MxTensor(*size, buf.device, buf) for size, buf in zip(ctx.sizes, ctx.saved_tensors))
        dx, dw = mx_linear_backward(flat, saved, rand, need_dx=need_dx, need_dw=need_dw)
        return dx.view(ctx.x_shape) if need_dx else None, dw.to(ctx.w_dtype) if need_dw else None, None, None


def mx_linear_train(x: torch.Tensor, w: torch.Tensor, stochastic: bool = True, generator=None) -> torch.Tensor:
    """The layer under autograd: x of any leading shape, w out x in, any strides
    (copied where their rows are not contiguous).  With `stochastic` the incoming gradient is rounded with random bytes of
    `generator` (None: the device's default one)."""
    return _MxLinearFunction.apply(x, w, stochastic, generator)

"""Products of linear layers: ``linear_forward`` (y = x W^T) and
``linear_input_grad`` (dx = dy W), with one weight or one per expert over
ragged tokens, from bfloat16 or float32, or from 8 bits on both sides: an
``ActCheckpoint`` times a :class:`Weight8`.

Together with ``weight_grad`` they are a linear layer's three products; the
offsets of all three are the same tensor.  As in ``layer_ops``, every
arithmetic step runs in the library's HIP kernels, the functions are not
differentiable themselves (``layers`` is), and ``stream`` runs a call, and
allocates what it returns, on that stream.
"""
from __future__ import annotations

import ctypes
from typing import Optional

import torch

from . import _lib
from .api import _check, _ptr, _wrote, dtype_code
from .layer_ops import ActCheckpoint, _away, _check_rows, _raw_stream, _ref, _there


class Weight8:
    """A weight, or a stack of them, in 8 bits (``include/muon.h``): ``q``
    [(count,) rows, cols up to a multiple of 128] and ``q_t`` [(count,) cols,
    rows up to a multiple of 128], the same numbers with rows and columns
    exchanged, in float8_e4m3fn, and ``scale`` uint8 [(count,) row blocks,
    column blocks] of 128 x 128 elements.  An element stands for
    ``q * 2^(scale - 127)``."""

    __slots__ = ("_q", "_q_t", "_scale", "_buffer", "_shape", "_device", "_c")

    def __init__(self, q: torch.Tensor, q_t: torch.Tensor, scale: torch.Tensor):
        for name, t, dtype in (("q", q, torch.float8_e4m3fn), ("q_t", q_t, torch.float8_e4m3fn),
                               ("scale", scale, torch.uint8)):
            if not isinstance(t, torch.Tensor):
                raise TypeError(f"{name} must be a torch.Tensor")
            if t.dtype != dtype:
                raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
        if q.ndim not in (2, 3) or q_t.ndim != q.ndim:
            raise ValueError("q and q_t must be a matrix or a stack of matrices each")
        *lead, rows, qp = q.shape
        cols, tp = q_t.shape[-2:]
        pr, pc = (rows + 127) // 128, (cols + 127) // 128
        device = q.device
        for name, t, shape in (("q", q, [*lead, rows, 128 * pc]), ("q_t", q_t, [*lead, cols, 128 * pr]),
                               ("scale", scale, [*lead, pr, pc])):
            if list(t.shape) != shape or not t.is_contiguous() or not t.is_cuda:
                raise ValueError(f"{name} must be a contiguous GPU tensor of shape {tuple(shape)} "
                                 f"for weights of {rows} x {cols}, got {tuple(t.shape)}")
            if t.device != device:
                raise ValueError(f"{name} is on {t.device}, q on {device}")
        self._q, self._q_t, self._scale, self._buffer = q, q_t, scale, None
        self._shape, self._device = (*lead, rows, cols), device
        self._c = _lib.Weight8(q.data_ptr(), q_t.data_ptr(), scale.data_ptr(),
                               lead[0] if lead else 1, rows, cols)

    @classmethod
    def empty(cls, *shape: int, device="cuda") -> "Weight8":
        """Unwritten, for the ``out`` of :func:`weight_quantize`: ``shape`` is
        the weight's, (rows, cols) or (count, rows, cols)."""
        if len(shape) not in (2, 3) or min(shape[-2:]) < 1 or min(shape) < 0:
            raise ValueError(f"a weight has the shape (rows, cols) or (count, rows, cols), not {shape}")
        lead, (rows, cols) = shape[:-2], shape[-2:]
        pr, pc = (rows + 127) // 128, (cols + 127) // 128
        n = lead[0] if lead else 1
        # one allocation for the three, each from a multiple of 128 bytes on; the
        # tensors are made when asked for
        a, b = n * rows * pc * 128, n * cols * pr * 128
        w = cls.__new__(cls)
        w._buffer = torch.empty(a + b + n * pr * pc, dtype=torch.uint8, device=device)
        if not w._buffer.is_cuda:
            raise ValueError(f"a Weight8 must be on a GPU, not on {w._buffer.device}")
        w._q = w._q_t = w._scale = None
        w._shape, w._device = (*lead, rows, cols), w._buffer.device
        at = w._buffer.data_ptr()
        w._c = _lib.Weight8(at, at + a, at + a + b, n, rows, cols)
        return w

    def _split(self):
        *lead, rows, cols = self._shape
        pr, pc = (rows + 127) // 128, (cols + 127) // 128
        n = lead[0] if lead else 1
        a, b = n * rows * pc * 128, n * cols * pr * 128
        buf = self._buffer
        self._q = buf[:a].view(torch.float8_e4m3fn).view(*lead, rows, 128 * pc)
        self._q_t = buf[a:a + b].view(torch.float8_e4m3fn).view(*lead, cols, 128 * pr)
        self._scale = buf[a + b:].view(*lead, pr, pc)

    @property
    def q(self) -> torch.Tensor:
        if self._q is None:
            self._split()
        return self._q

    @property
    def q_t(self) -> torch.Tensor:
        if self._q_t is None:
            self._split()
        return self._q_t

    @property
    def scale(self) -> torch.Tensor:
        if self._scale is None:
            self._split()
        return self._scale

    @property
    def shape(self):
        return self._shape

    @property
    def device(self) -> torch.device:
        return self._device

    def __reduce__(self):      # deep copies and pickles have tensors of their own
        return Weight8, (self.q, self.q_t, self.scale)

    @property
    def nbytes(self) -> int:
        return self.q.numel() + self.q_t.numel() + self.scale.numel()

    def __repr__(self):
        return f"Weight8({' x '.join(map(str, self.shape))}, {self.device})"


def weight_quantize(W: torch.Tensor, *, out: Optional[Weight8] = None, stream=None) -> Weight8:
    """``W`` [rows, cols] or [count, rows, cols], float32 or bfloat16, in 8 bits."""
    if _away(W, stream):
        return _there(weight_quantize, W, stream, out=out)
    _check_weight("W", W)
    dt = dtype_code(W.dtype)
    given = out
    if out is None:
        out = Weight8.empty(*W.shape, device=W.device)
    elif not isinstance(out, Weight8):
        raise TypeError("out must be a Weight8")
    elif out.shape != tuple(W.shape) or out.device != W.device:
        raise ValueError(f"out is {out}, W has shape {tuple(W.shape)} on {W.device}")
    st = _lib.lib().muon_weight_quantize(W.data_ptr(), dt, ctypes.byref(out._c),
                                         _raw_stream(W.device.index))
    _check(st, "muon_weight_quantize")
    if given is not None:
        _wrote(*((given._q, given._q_t, given._scale) if given._buffer is None else (given._buffer,)))
    return out


def _check_weight(name, W):
    if not isinstance(W, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if W.ndim not in (2, 3):
        raise ValueError(f"{name} must be a matrix or a stack of matrices, it has {W.ndim} dims")
    if not W.is_cuda:
        raise ValueError(f"{name} must be on a GPU")
    if not W.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _check_offsets(offsets, shape, device) -> int:
    """Checks offsets against a weight's shape; returns the count of matrices."""
    if offsets is None:
        if len(shape) != 2:
            raise ValueError("a stack of weights needs offsets")
        return 1
    if not isinstance(offsets, torch.Tensor) or offsets.dtype != torch.int64:
        raise TypeError("offsets must be an int64 tensor")
    if len(shape) != 3:
        raise ValueError("offsets need a stack of weights [count, rows, cols]")
    if offsets.ndim != 1 or offsets.numel() != shape[0] + 1 or not offsets.is_contiguous():
        raise ValueError(f"offsets must be a contiguous vector of {shape[0] + 1} token totals")
    if offsets.device != device:
        raise ValueError(f"offsets is on {offsets.device}, expected {device}")
    return shape[0]


def _product(x, W, offsets, dtype, out, across):
    """Both products: across the weight's rows (the input gradient) or along them."""
    name = "dy" if across else "x"
    quantized = isinstance(x, ActCheckpoint)
    if quantized != isinstance(W, Weight8):
        raise TypeError(f"{name} and W must both be in 8 bits (an ActCheckpoint and a Weight8) or "
                        "both be tensors")
    if not quantized:
        ld = _check_rows(name, x)
        _check_weight("W", W)
        if W.dtype != x.dtype:
            raise TypeError(f"W has dtype {W.dtype}, {name} {x.dtype}")
        if dtype is not None and dtype != x.dtype:
            raise TypeError(f"the result of {x.dtype} has that type, not {dtype}")
        dtype = x.dtype
    elif x.format != "e4m3":
        raise ValueError(f"products take checkpoints in e4m3, not {x.format}")
    elif dtype is None:
        dtype = torch.bfloat16
    dev = x.device
    if W.device != dev:
        raise ValueError(f"W is on {W.device}, {name} on {dev}")
    rows, cols = W.shape[-2:]
    k, n = (rows, cols) if across else (cols, rows)
    tokens, width = x.shape
    if width != k:
        raise ValueError(f"{name} has {width} columns, the weights are {rows} x {cols}")
    count = _check_offsets(offsets, W.shape, dev)
    dt = dtype_code(dtype)
    given = out
    if out is None:
        out = torch.empty(tokens, n, dtype=dtype, device=dev)
    else:
        _check_rows("out", out, dev, (tokens, n), dtype, contiguous=True)
    L, stream = _lib.lib(), _raw_stream(dev.index)
    if quantized:
        fn = L.muon_linear_input_grad_quantized if across else L.muon_linear_forward_quantized
        st = fn(_ref(x), ctypes.byref(W._c), _ptr(offsets), out.data_ptr(), dt, stream)
    else:
        fn = L.muon_linear_input_grad if across else L.muon_linear_forward
        st = fn(x.data_ptr(), ld, dt, W.data_ptr(), _ptr(offsets), count, tokens, rows, cols,
                out.data_ptr(), stream)
    _check(st, "muon_linear_input_grad" if across else "muon_linear_forward")
    _wrote(given)
    return out


def linear_forward(x, W, *, offsets=None, dtype=None, out=None, stream=None) -> torch.Tensor:
    """``y[t] = x[t] W^T`` [tokens, rows] for x [tokens, cols] and W [rows, cols],
    or with matrix e of a stack W [count, rows, cols] for the tokens
    [offsets[e], offsets[e + 1]).

    x and W: tensors of one dtype, which y takes, or an ``ActCheckpoint`` in
    e4m3 and a :class:`Weight8` (y: ``dtype``, default bfloat16).  From 8 bits,
    float32 results add exact products in float32; for bfloat16 ones the matrix
    cores cut each product to 13 bits below the largest exponent of its 8
    neighbours along the sum: 1.6e-5 of the results' norm for normally
    distributed operands, but any part of a result whose products cancel
    (``include/muon.h``).  offsets: int64
    GPU tensor of count + 1 running token totals, at most
    ``MUON_LINEAR_MAX_COUNT`` matrices; its values are not read on the host:
    those outside [0, tokens] or decreasing are bounded on the device.  Tokens of
    no matrix give zeros.  A call has at most 2^24 tiles of outputs
    (``include/muon.h`` has the formula), which binds from some 2^36 outputs on,
    or 2^30 tokens of a few outputs: larger ones raise, and are several calls."""
    if _away(x, stream):
        return _there(linear_forward, x, stream, W, offsets=offsets, dtype=dtype, out=out)
    return _product(x, W, offsets, dtype, out, across=False)


def linear_input_grad(dy, W, *, offsets=None, dtype=None, out=None, stream=None) -> torch.Tensor:
    """``dx[t] = dy[t] W`` [tokens, cols], the input gradient of
    :func:`linear_forward`, with the same W and offsets; dy [tokens, rows] is a
    tensor, or an ``ActCheckpoint`` of it for a :class:`Weight8`."""
    if _away(dy, stream):
        return _there(linear_input_grad, dy, stream, W, offsets=offsets, dtype=dtype, out=out)
    return _product(dy, W, offsets, dtype, out, across=True)

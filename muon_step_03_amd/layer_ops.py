"""The layer operators around the hidden weights: layer norm's two passes,
8-bit activation checkpoints, and the weight gradients that read them.

They make what the optimizer steps consume: ``layernorm_backward`` the
gradients of gains and biases (the AdamW vectors), ``weight_grad`` the G of
``muon_step`` (one matrix) or of ``stacked_group`` (a stack of experts).  As in
``api``, every arithmetic step runs in the library's HIP kernels; PyTorch
provides device memory and streams.  The functions are not differentiable
themselves: ``layers`` is.

Matrices are tokens x columns, float32 or bfloat16, on one GPU.  Inputs may be
row-strided views (a slice of a fused projection's columns); a column stride
other than one is refused.  Outputs are new contiguous tensors unless given.
``stream`` runs a call, and allocates what it returns, on that stream; whoever
uses tensors across streams orders them, as with any PyTorch operator.
"""
from __future__ import annotations

import ctypes
from typing import NamedTuple, Optional

import torch

from . import _lib
from .api import _check, _ptr, dtype_code

FORMATS = {"e4m3": torch.float8_e4m3fn, "int8": torch.int8}
_FORMAT_CODES = {torch.float8_e4m3fn: _lib.MUON_CKPT_E4M3, torch.int8: _lib.MUON_CKPT_INT8}
_FORMAT_NAMES = {v: k for k, v in FORMATS.items()}


# Looked up at the call: a PyTorch without a GPU backend does not have them.
def _raw_stream(index):
    """The current stream's handle, with no stream object made."""
    return torch._C._cuda_getCurrentRawStream(index)


def _current_device():
    return torch._C._cuda_getDevice()


def _away(t, stream) -> bool:
    """Whether a call on ``t`` has to change the current device or stream."""
    if stream is not None:
        return True
    device = getattr(t, "device", None)
    return device is not None and device.type == "cuda" and device.index != _current_device()


def _there(fn, t, stream, *args, **kw):
    """``fn(t, ...)`` with the device of ``t``, and ``stream`` if given, current."""
    if not isinstance(t, (torch.Tensor, ActCheckpoint)):
        raise TypeError(f"expected a torch.Tensor, got {type(t).__name__}")
    if stream is None:
        with torch.cuda.device(t.device):
            return fn(t, *args, **kw)
    if stream.device != t.device:
        raise ValueError(f"stream is on {stream.device}, the tensors on {t.device}")
    with torch.cuda.stream(stream):
        return fn(t, *args, **kw)


def _check_rows(name, t, device=None, shape=None, dtype=None, contiguous=False):
    """A 2-D GPU tensor with unit column stride; returns its row stride."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.ndim != 2:
        raise ValueError(f"{name} must be 2-D (tokens x columns), it has {t.ndim} dims")
    if not t.is_cuda:
        raise ValueError(f"{name} must be on a GPU")
    if device is not None and t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} has dtype {t.dtype}, expected {dtype}")
    rows, cols = t.shape
    if cols > 1 and t.stride(1) != 1:
        raise ValueError(f"{name} must have unit column stride")
    ld = cols if rows <= 1 else t.stride(0)
    if ld < cols or (contiguous and ld != cols):
        raise ValueError(f"{name} must be {'contiguous' if contiguous else 'row-major'}")
    return ld


def _check_vector(name, t, n, device, dtype=None):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.ndim != 1 or t.numel() != n:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected ({n},)")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} has dtype {t.dtype}, expected {dtype}")


def _workspace(need, device, workspace):
    """(tensor, address, bytes) of a workspace of at least ``need`` bytes."""
    if workspace is None:
        if need == 0:
            return None, None, 0
        workspace = torch.empty(need, dtype=torch.uint8, device=device)
        return workspace, workspace.data_ptr(), need
    if workspace.device != device or not workspace.is_contiguous():
        raise ValueError(f"workspace must be contiguous and on {device}")
    if workspace.numel() * workspace.element_size() < need:
        raise ValueError(f"workspace holds {workspace.numel() * workspace.element_size()} bytes, "
                         f"{need} needed")
    return workspace, workspace.data_ptr(), workspace.numel() * workspace.element_size()


def _wrote(*given):
    """Tells autograd that tensors it did not make were written: a backward
    pass that kept one of them then raises, as after PyTorch's own writes."""
    for t in given:
        if t is not None and not t.is_inference():
            torch.autograd.graph.increment_version(t)


class ActCheckpoint:
    """A tokens x cols activation kept in 8 bits (``include/muon.h``,
    "Checkpoint format"): ``q`` [tokens, cols up to a multiple of 32] in
    float8_e4m3fn or int8, ``scale`` uint8 [tokens, blocks of 32 columns up to
    a multiple of 4].  An element stands for ``q * 2^(scale - 127)``."""

    __slots__ = ("_q", "_scale", "_buffer", "_shape", "_store", "_c")

    def __init__(self, q: torch.Tensor, scale: torch.Tensor, cols: int):
        if q.dtype not in _FORMAT_CODES:
            raise TypeError(f"q must be float8_e4m3fn or int8, got {q.dtype}")
        if scale.dtype != torch.uint8:
            raise TypeError(f"scale must be uint8, got {scale.dtype}")
        tokens, cols = q.shape[0], int(cols)
        for name, t, pitch in (("q", q, _lib.ckpt_q_pitch(cols)),
                               ("scale", scale, _lib.ckpt_scale_pitch(cols))):
            if tuple(t.shape) != (tokens, pitch) or not t.is_contiguous() or not t.is_cuda:
                raise ValueError(f"{name} must be a contiguous GPU tensor of shape "
                                 f"{(tokens, pitch)} for {cols} columns, got {tuple(t.shape)}")
        if scale.device != q.device:
            raise ValueError(f"scale is on {scale.device}, q on {q.device}")
        self._q, self._scale, self._buffer = q, scale, None
        self._shape, self._store = (tokens, cols), q.dtype
        self._c = None

    @classmethod
    def empty(cls, tokens: int, cols: int, fmt: str = "e4m3", device="cuda") -> "ActCheckpoint":
        """An unwritten checkpoint, for the ``out`` of a save."""
        try:
            store = FORMATS[fmt]
        except KeyError:
            raise ValueError(f"unknown checkpoint format {fmt!r}; expected one of "
                             f"{sorted(FORMATS)}") from None
        # one buffer of its own for both; the views are made when asked for
        size = tokens * ((cols + 31) // 32 * 32)
        ck = cls.__new__(cls)
        ck._buffer = torch.empty(size + tokens * ((cols + 127) // 128 * 4), dtype=torch.uint8,
                                 device=device)
        if not ck._buffer.is_cuda:
            raise ValueError(f"a checkpoint must be on a GPU, not on {ck._buffer.device}")
        ck._q = ck._scale = None
        ck._shape, ck._store = (tokens, cols), store
        at = ck._buffer.data_ptr()
        ck._c = _lib.Ckpt(at, at + size, tokens, cols, _FORMAT_CODES[store])
        return ck

    def _split(self):
        tokens, cols = self._shape
        size = tokens * _lib.ckpt_q_pitch(cols)
        self._q = self._buffer[:size].view(self._store).view(tokens, _lib.ckpt_q_pitch(cols))
        self._scale = self._buffer[size:].view(tokens, _lib.ckpt_scale_pitch(cols))

    def __reduce__(self):      # copies and pickles have tensors of their own
        return ActCheckpoint, (self.q, self.scale, self.cols)

    def _written(self):
        _wrote(*((self._q, self._scale) if self._buffer is None else (self._buffer,)))

    @property
    def q(self) -> torch.Tensor:
        if self._q is None:
            self._split()
        return self._q

    @property
    def scale(self) -> torch.Tensor:
        if self._scale is None:
            self._split()
        return self._scale

    @property
    def tokens(self) -> int:
        return self._shape[0]

    @property
    def cols(self) -> int:
        return self._shape[1]

    @property
    def shape(self):
        return self._shape

    @property
    def format(self) -> str:
        return _FORMAT_NAMES[self._store]

    @property
    def device(self) -> torch.device:
        return (self._q if self._buffer is None else self._buffer).device

    @property
    def nbytes(self) -> int:
        return self.q.numel() + self.scale.numel()

    def __repr__(self):
        return f"ActCheckpoint({self.tokens} x {self.cols}, {self.format}, {self.device})"


def _as_checkpoint(name, spec, shape, device) -> Optional[ActCheckpoint]:
    """None, a format name (a new checkpoint) or a checkpoint to write."""
    if spec is None:
        return None
    if isinstance(spec, str):
        return ActCheckpoint.empty(*shape, fmt=spec, device=device)
    if not isinstance(spec, ActCheckpoint):
        raise TypeError(f"{name} must be a format name or an ActCheckpoint")
    if spec._shape != tuple(shape) or spec.device != device:
        raise ValueError(f"{name} is {spec}, expected {shape[0]} x {shape[1]} on {device}")
    return spec


def _ref(ck):
    """The library's descriptor of a checkpoint, by reference."""
    if ck is None:
        return None
    if ck._c is not None:      # of its own buffer
        return ctypes.byref(ck._c)
    return ctypes.byref(_lib.Ckpt(ck._q.data_ptr(), ck._scale.data_ptr(), *ck._shape,
                                  _FORMAT_CODES[ck._store]))


def checkpoint_save(x: torch.Tensor, fmt: str = "e4m3", *, out: Optional[ActCheckpoint] = None,
                    stream=None) -> ActCheckpoint:
    """Keeps ``x`` [tokens, cols] in 8 bits, ``fmt`` "e4m3" or "int8" (or in
    the format of ``out``)."""
    if _away(x, stream):
        return _there(checkpoint_save, x, stream, fmt, out=out)
    ld = _check_rows("x", x)
    dt = dtype_code(x.dtype)
    ck = _as_checkpoint("out", fmt if out is None else out, tuple(x.shape), x.device)
    st = _lib.lib().muon_checkpoint_save(x.data_ptr(), ld, dt, _ref(ck), _raw_stream(x.device.index))
    _check(st, "muon_checkpoint_save")
    if out is not None:
        ck._written()
    return ck


def checkpoint_restore(ck: ActCheckpoint, dtype: torch.dtype = torch.bfloat16, *,
                       out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """The values a checkpoint stands for (exact in bfloat16 and float32)."""
    if not isinstance(ck, ActCheckpoint):
        raise TypeError("ck must be an ActCheckpoint")
    if _away(ck, stream):
        return _there(checkpoint_restore, ck, stream, dtype, out=out)
    given = out
    if out is None:
        out = torch.empty(ck._shape, dtype=dtype, device=ck.device)
    else:
        _check_rows("out", out, ck.device, ck.shape, contiguous=True)
    st = _lib.lib().muon_checkpoint_restore(_ref(ck), out.data_ptr(), dtype_code(out.dtype),
                                            _raw_stream(ck.device.index))
    _check(st, "muon_checkpoint_restore")
    _wrote(given)
    return out


def _empty_rows(t):
    """A new contiguous matrix like ``t``."""
    return torch.empty_like(t) if t.is_contiguous() else \
        torch.empty(tuple(t.shape), dtype=t.dtype, device=t.device)


class LayerNormOut(NamedTuple):
    y: torch.Tensor
    mean: torch.Tensor
    rstd: torch.Tensor
    x_checkpoint: Optional[ActCheckpoint]
    y_checkpoint: Optional[ActCheckpoint]


def layernorm_forward(x, gain, bias=None, *, eps=1e-5, x_checkpoint=None, y_checkpoint=None,
                      stream=None) -> LayerNormOut:
    """``y = (x - mean) * rstd * gain + bias`` over the columns of ``x``.

    gain, bias: [cols], of one dtype (that of x or the other).  mean and rstd
    (float32, one per token) are what :func:`layernorm_backward` needs beside
    x.  ``x_checkpoint`` / ``y_checkpoint``: a format name, or an
    ActCheckpoint to overwrite, saves x, or y as returned, in the same pass.
    """
    if _away(x, stream):
        return _there(layernorm_forward, x, stream, gain, bias, eps=eps, x_checkpoint=x_checkpoint,
                      y_checkpoint=y_checkpoint)
    ld = _check_rows("x", x)
    dt, dev = dtype_code(x.dtype), x.device
    tokens, cols = x.shape
    _check_vector("gain", gain, cols, dev)
    pdt = dtype_code(gain.dtype)
    if bias is not None:
        _check_vector("bias", bias, cols, dev, gain.dtype)
    xc = _as_checkpoint("x_checkpoint", x_checkpoint, (tokens, cols), dev)
    yc = _as_checkpoint("y_checkpoint", y_checkpoint, (tokens, cols), dev)
    y = _empty_rows(x)
    mean = torch.empty(tokens, dtype=torch.float32, device=dev)
    rstd = torch.empty_like(mean)
    st = _lib.lib().muon_layernorm_forward(
        x.data_ptr(), ld, gain.data_ptr(), _ptr(bias), tokens, cols, dt, pdt, float(eps),
        y.data_ptr(), mean.data_ptr(), rstd.data_ptr(), _ref(xc), _ref(yc), _raw_stream(dev.index))
    _check(st, "muon_layernorm_forward")
    if xc is x_checkpoint and xc is not None:
        xc._written()
    if yc is y_checkpoint and yc is not None:
        yc._written()
    return LayerNormOut(y, mean, rstd, xc, yc)


def layernorm_workspace_bytes(tokens: int, cols: int) -> int:
    return int(_lib.lib().muon_layernorm_workspace_bytes(tokens, cols))


def layernorm_backward(dy, x, gain, mean, rstd, *, bias=True, dgain=None, dbias=None,
                       accumulate=False, workspace=None, stream=None):
    """``(dx, dgain, dbias)`` of :func:`layernorm_forward`.

    x: the forward's input, or an ActCheckpoint of it.  dgain and dbias have
    the dtype of gain; given ones are overwritten, or added to with
    ``accumulate``.  ``bias=False`` skips dbias (None is returned).
    """
    if _away(dy, stream):
        return _there(layernorm_backward, dy, stream, x, gain, mean, rstd, bias=bias, dgain=dgain,
                      dbias=dbias, accumulate=accumulate, workspace=workspace)
    ldy = _check_rows("dy", dy)
    dt, dev = dtype_code(dy.dtype), dy.device
    tokens, cols = dy.shape
    ck = x if isinstance(x, ActCheckpoint) else None
    ldx = 0
    if ck is None:
        ldx = _check_rows("x", x, dev, dy.shape, dy.dtype)
    else:
        _as_checkpoint("x", ck, (tokens, cols), dev)
    _check_vector("gain", gain, cols, dev)
    _check_vector("mean", mean, tokens, dev, torch.float32)
    _check_vector("rstd", rstd, tokens, dev, torch.float32)
    pdt = dtype_code(gain.dtype)
    if not bias and dbias is not None:
        raise ValueError("dbias was given with bias=False")
    for name, t, wanted in (("dgain", dgain, True), ("dbias", dbias, bool(bias))):
        if t is not None:
            _check_vector(name, t, cols, dev, gain.dtype)
        elif accumulate and wanted:
            raise ValueError(f"accumulate needs {name}")
    dx = _empty_rows(dy)
    given = dgain, dbias
    if dgain is None:
        dgain = torch.empty_like(gain)
    if bias and dbias is None:
        dbias = torch.empty_like(gain)
    _ws, at, size = _workspace(layernorm_workspace_bytes(tokens, cols), dev, workspace)
    st = _lib.lib().muon_layernorm_backward(
        dy.data_ptr(), ldy, None if ck is not None else x.data_ptr(), ldx, _ref(ck),
        gain.data_ptr(), mean.data_ptr(), rstd.data_ptr(), tokens, cols, dt, pdt,
        dx.data_ptr(), dgain.data_ptr(), _ptr(dbias), int(accumulate), at, size,
        _raw_stream(dev.index))
    _check(st, "muon_layernorm_backward")
    _wrote(*given)
    return dx, dgain, dbias


def weight_grad_workspace_bytes(count: int, with_offsets: bool, tokens: int, rows: int, cols: int,
                                dtype: torch.dtype) -> int:
    """Workspace of :func:`weight_grad`; dtype: that of dy."""
    return int(_lib.lib().muon_weight_grad_workspace_bytes(count, int(with_offsets), tokens, rows,
                                                           cols, dtype_code(dtype)))


def weight_grad(dy, ck, *, offsets=None, G=None, dtype=None, accumulate=False, workspace=None,
                stream=None):
    """Gradient of the weight of ``y = x W^T`` from ``dy`` [tokens, rows] and
    the checkpoint of ``x`` [tokens, cols]: ``G = dy^T x`` [rows, cols].

    offsets: int64 GPU tensor of count + 1 running token totals; G is then the
    stack [count, rows, cols] that :func:`stacked_group` takes, matrix e over
    the tokens [offsets[e], offsets[e + 1]) (none: zeros).  Its values are not
    read on the host: those outside [0, tokens] or decreasing are bounded on
    the device.  G: written in place (added to with ``accumulate``), or a new
    tensor of ``dtype`` (default: that of dy).
    """
    if _away(dy, stream):
        return _there(weight_grad, dy, stream, ck, offsets=offsets, G=G, dtype=dtype,
                      accumulate=accumulate, workspace=workspace)
    ld = _check_rows("dy", dy)
    dt, dev = dtype_code(dy.dtype), dy.device
    tokens, rows = dy.shape
    if not isinstance(ck, ActCheckpoint):
        raise TypeError("ck must be an ActCheckpoint")
    _as_checkpoint("ck", ck, (tokens, ck.cols), dev)
    count, shape = 1, (rows, ck.cols)
    if offsets is not None:
        if not isinstance(offsets, torch.Tensor) or offsets.dtype != torch.int64:
            raise TypeError("offsets must be an int64 tensor")
        if offsets.ndim != 1 or offsets.numel() < 1 or not offsets.is_contiguous():
            raise ValueError("offsets must be a contiguous vector of count + 1 token totals")
        if offsets.device != dev:
            raise ValueError(f"offsets is on {offsets.device}, expected {dev}")
        count = offsets.numel() - 1
        shape = (count, rows, ck.cols)
    if G is None:
        if accumulate:
            raise ValueError("accumulate needs G")
    else:
        if not isinstance(G, torch.Tensor):
            raise TypeError("G must be a torch.Tensor")
        if tuple(G.shape) != shape or not G.is_contiguous() or G.device != dev:
            raise ValueError(f"G must be a contiguous tensor of shape {shape} on {dev}")
        if dtype is not None and G.dtype != dtype:
            raise TypeError(f"G has dtype {G.dtype}, expected {dtype}")
    given = G
    gdt = dtype_code(G.dtype if G is not None else dtype or dy.dtype)
    if G is None:
        G = torch.empty(shape, dtype=dtype or dy.dtype, device=dev)
    if count == 0:
        return G
    need = weight_grad_workspace_bytes(count, offsets is not None, tokens, rows, ck.cols, dy.dtype)
    _ws, at, size = _workspace(need, dev, workspace)
    st = _lib.lib().muon_weight_grad(
        dy.data_ptr(), ld, dt, _ref(ck), _ptr(offsets), count, rows, G.data_ptr(), gdt,
        int(accumulate), at, size, _raw_stream(dev.index))
    _check(st, "muon_weight_grad")
    _wrote(given)
    return G

"""fp64 NumPy definitions of the linear products and of weights in 8 bits.
Plain formulas, no blocking of the products, no shared code with the library."""
import numpy as np

from .layer_oracle import e4m3_round

SIDE = 128


def bounds(offsets, tokens):
    """Offsets as they are read: clamped, and never below the ones before."""
    o = np.clip(np.asarray(offsets, dtype=np.float64), 0, tokens).astype(np.int64)
    return np.maximum.accumulate(o)


def forward(x, W, offsets=None):
    """x W^T, or with each matrix of a stack over its tokens (zeros elsewhere)."""
    if offsets is None:
        return x @ W.T
    o = bounds(offsets, x.shape[0])
    y = np.zeros((x.shape[0], W.shape[1]))
    for e in range(W.shape[0]):
        if o[e + 1] > o[e]:
            y[o[e]:o[e + 1]] = x[o[e]:o[e + 1]] @ W[e].T
    return y


def input_grad(dy, W, offsets=None):
    return forward(dy, np.swapaxes(W, -1, -2), offsets)


def quantized(W):
    """(values, q, scale) of a matrix in 8 bits: the float64 values read back,
    the q as numbers and the scale bytes of the blocks."""
    rows, cols = W.shape
    br, bc = -(-rows // SIDE), -(-cols // SIDE)
    values, q = np.zeros(W.shape), np.zeros(W.shape)
    scale = np.zeros((br, bc), dtype=np.int64)
    for i in range(br):
        for j in range(bc):
            at = np.s_[i * SIDE:(i + 1) * SIDE, j * SIDE:(j + 1) * SIDE]
            b = W[at]
            if not np.isfinite(b).all():
                scale[i, j], values[at] = 255, np.nan
                continue
            a = np.abs(b).max()
            m, k = np.frexp(a / 448.0)          # a / 448 = m 2^k, 0.5 <= m < 1
            e = int(np.clip(-117 if a == 0 else k - 1 if m == 0.5 else k, -117, 119))
            v = e4m3_round(np.clip(np.ldexp(b, -e), -448, 448))
            q[at], values[at], scale[i, j] = v, np.ldexp(v, e), e + 127
    return values, q, scale

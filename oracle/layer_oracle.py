"""fp64 NumPy definitions of the layer operators: layer norm, 8-bit activation
checkpoints and the weight gradient that reads them.  Plain formulas, no
blocking, no shared code with the library."""
import numpy as np

CKPT_BLOCK = 32
# largest q, smallest and largest scale exponent of each checkpoint format
CKPT_FORMATS = {"e4m3": (448.0, -117, 119), "int8": (127.0, -117, 121)}


def layernorm(x, gain, bias=None, eps=1e-5):
    """(y, mean, rstd) over the columns of x."""
    mean = x.mean(axis=1)
    rstd = 1.0 / np.sqrt(((x - mean[:, None]) ** 2).mean(axis=1) + eps)
    y = (x - mean[:, None]) * rstd[:, None] * gain
    return (y if bias is None else y + bias), mean, rstd


def layernorm_grad(dy, x, gain, mean, rstd):
    """(dx, dgain, dbias) for the given mean and rstd."""
    xhat = (x - mean[:, None]) * rstd[:, None]
    a = dy * gain
    dx = rstd[:, None] * (a - a.mean(axis=1, keepdims=True)
                          - xhat * (a * xhat).mean(axis=1, keepdims=True))
    return dx, (dy * xhat).sum(axis=0), dy.sum(axis=0)


def e4m3_round(v):
    """Nearest e4m3 number, ties to even (|v| <= 448): 3 bits behind the
    leading one, smallest exponent -6."""
    v = np.asarray(v, np.float64)
    size = np.frexp(np.where(v == 0, 1.0, v))[1] - 1
    step = np.ldexp(1.0, np.maximum(size, -6) - 3)
    return np.rint(v / step) * step


def checkpoint(x, fmt):
    """(values, q, scale) of a saved x: the float64 values read back, the q as
    numbers [tokens, blocks * 32] and the scale bytes [tokens, blocks]."""
    top, e_min, e_max = CKPT_FORMATS[fmt]
    tokens, cols = x.shape
    blocks = -(-cols // CKPT_BLOCK)
    pad = np.zeros((tokens, blocks * CKPT_BLOCK))
    pad[:, :cols] = x
    pad = pad.reshape(tokens, blocks, CKPT_BLOCK)
    bad = ~np.isfinite(pad).all(axis=2)
    a = np.abs(np.where(bad[:, :, None], 0.0, pad)).max(axis=2)
    m, k = np.frexp(a / top)            # a / top = m 2^k, 0.5 <= m < 1
    e = np.where(m == 0.5, k - 1, k)    # smallest e with a <= top 2^e
    e = np.clip(np.where(a == 0, e_min, e), e_min, e_max).astype(np.int64)
    v = np.clip(np.where(bad[:, :, None], 0.0, pad) * np.ldexp(1.0, -e)[:, :, None], -top, top)
    q = e4m3_round(v) if fmt == "e4m3" else np.rint(v)
    values = np.where(bad[:, :, None], np.nan, q * np.ldexp(1.0, e)[:, :, None])
    flat = (tokens, blocks * CKPT_BLOCK)
    return values.reshape(flat)[:, :cols], q.reshape(flat), np.where(bad, 255, e + 127)


def weight_grad(dy, x, offsets=None):
    """dy^T x, or one per group of tokens [offsets[e], offsets[e + 1])."""
    if offsets is None:
        return dy.T @ x
    return np.stack([dy[a:b].T @ x[a:b] for a, b in zip(offsets[:-1], offsets[1:])]) \
        if len(offsets) > 1 else np.zeros((0, dy.shape[1], x.shape[1]))

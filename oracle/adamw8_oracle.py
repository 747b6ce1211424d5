"""fp64 NumPy definition of AdamW with 8-bit states (include/muon.h, "State
format"): the step, what a state's bytes stand for, and what is kept of given
moments.  Plain formulas, no shared code with the library."""
import numpy as np

BLOCK = 32
# name -> (largest number, bits of mantissa, smallest and largest scale exponent)
FORMATS = {"m": (448.0, 3, -117, 119), "r": (496.0, 4, -116, 118)}


def random_bits(n, seed):
    """The 32 random bits of elements 0 .. n - 1."""
    i = np.arange(n, dtype=np.uint64)
    low = np.uint64(0xffffffff)
    x = ((i & low) * np.uint64(0x9e3779b1) + (i >> np.uint64(32)) * np.uint64(0x85ebca77)
         + np.uint64(seed)) & low
    x = ((x ^ (x >> np.uint64(16))) * np.uint64(0x7feb352d)) & low
    x = ((x ^ (x >> np.uint64(15))) * np.uint64(0x846ca68b)) & low
    return (x ^ (x >> np.uint64(16))).astype(np.int64)


def share(n, seed, which):
    """What is added to an element before it is rounded down, in steps."""
    x = random_bits(n, seed)
    return ((x >> 16 if which == "m" else x & 0xffff) + 0.5) / 65536


def numbers(which):
    """The 256 numbers of a format, by code."""
    c = np.arange(256)
    bits = FORMATS[which][1]
    field, frac = (c & 0x7f if which == "m" else c) >> bits, c & ((1 << bits) - 1)
    v = np.where(field > 0, np.ldexp(1 + frac / 2.0 ** bits, field - 7),
                 np.ldexp(frac / 2.0 ** bits, -6))
    if which == "m":
        v = np.where(c & 0x80, -v, v)
        v[[0x7f, 0xff]] = np.nan
    return v


def values(q, scale, n, which):
    """The float64 numbers that a state stands for."""
    up = np.where(scale == 255, np.nan, np.ldexp(1.0, scale.astype(np.int64) - 127))
    return (numbers(which)[q.reshape(-1, BLOCK)] * up[:, None]).reshape(-1)[:n]


def scale_bytes(x, which):
    """The scale byte of each block of a moment."""
    top, _, lo, hi = FORMATS[which]
    pad = np.zeros(-(-x.size // BLOCK) * BLOCK)
    pad[:x.size] = np.abs(x)
    a = pad.reshape(-1, BLOCK).max(axis=1)
    bad = ~np.isfinite(a)
    m, k = np.frexp(np.where(bad, 0, a) / top)          # a / top = m 2^k, 0.5 <= m < 1
    e = np.where(m == 0.5, k - 1, k)
    e = np.clip(np.where(a == 0, lo, e), lo, hi)
    return np.where(bad, 255, e + 127)


def kept(x, scale, added, which):
    """The float64 numbers that are kept of a moment x under these scale bytes,
    where ``added`` steps go onto each element before it is rounded down."""
    top, bits, _, _ = FORMATS[which]
    up = np.repeat(np.ldexp(1.0, scale.astype(np.int64) - 127), BLOCK)[:x.size]
    a = np.abs(x) / up
    size = np.ldexp(1.0, np.maximum(np.frexp(np.where(a == 0, 1, a))[1] - 1, -6) - bits)
    v = np.minimum(np.floor(a / size + added) * size, top)
    if which == "r":
        v = np.where(x > 0, np.maximum(v, 2.0 ** -10), 0)
    return np.copysign(v, x) * up


def step(p, g, m, r, *, lr, beta1, beta2, eps, weight_decay, step):
    """(p', m', r') in fp64, m' and r' before they are kept."""
    m = beta1 * m + (1 - beta1) * g
    r = np.sqrt(beta2 * r * r + (1 - beta2) * g * g)
    mean, root = m / (1 - beta1 ** step), r / np.sqrt(1 - beta2 ** step)
    with np.errstate(invalid="ignore", divide="ignore"):
        return p - lr * weight_decay * p - lr * mean / (root + eps), m, r

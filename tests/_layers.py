"""Inputs, oracles and error bounds shared by the layer operators' GPU tests
(not collected by pytest).

The bounds count roundings: u = 2^-24 is half a step of float32, and a result
stored as bfloat16 is off by at most 2^-8 of its value on top.  A sum of n terms
added in float32 in any order is off by at most n u times the sum of its terms'
magnitudes (first order).  A row's sums are at most 32 values in a lane, then 6
exchanges and 16 waves: under 64 additions.
"""
import numpy as np
import torch

from muon_step_03_amd import ActCheckpoint, _lib
from oracle import layer_oracle as lo

DEV = "cuda"
U = 2.0 ** -24
ROW = 64 * U          # a row's sum, relative to the sum of magnitudes
HALF = {torch.float32: U, torch.bfloat16: 2.0 ** -8}


def f64(t):
    return t.detach().cpu().double().numpy()


def hidden(tokens, cols, dtype=torch.bfloat16, seed=0, scale=1.0):
    """Unit normal tokens with a column offset and a few large channels."""
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(tokens, cols, generator=g) + 0.1 * torch.randn(cols, generator=g)
    x[:, ::97] *= 8.0
    return (x * scale).to(dtype).to(DEV)


def grads(tokens, cols, dtype=torch.bfloat16, seed=1):
    return hidden(tokens, cols, dtype, seed + 1000, 1e-3)


def params(cols, dtype, seed=2):
    g = torch.Generator().manual_seed(seed)
    return ((1 + 0.1 * torch.randn(cols, generator=g)).to(dtype).to(DEV),
            (0.1 * torch.randn(cols, generator=g)).to(dtype).to(DEV))


def within(got, want, bound, what):
    """|got - want| <= bound elementwise; NaN and infinities in the same places."""
    got = f64(got) if isinstance(got, torch.Tensor) else got
    assert got.shape == want.shape, what
    assert np.array_equal(np.isnan(got), np.isnan(want)), f"{what}: NaN"
    fine = np.isfinite(want)
    assert np.array_equal(got[~fine & ~np.isnan(want)], want[~fine & ~np.isnan(want)]), what
    over = (np.abs(got - want) - np.broadcast_to(bound, want.shape))[fine]
    assert over.size == 0 or over.max() <= 0, f"{what}: over its bound by {over.max():.3e}"


def check_checkpoint(ck: ActCheckpoint, x64, fmt):
    """Every byte of a checkpoint of x (float64 values of the saved tensor)."""
    values, q, scale = lo.checkpoint(x64, fmt)
    assert ck.format == fmt and ck.shape == x64.shape
    assert np.array_equal(f64(ck.q), q)
    got = ck.scale.cpu().numpy()
    assert got.shape[1] == _lib.ckpt_scale_pitch(x64.shape[1])
    assert np.array_equal(got[:, :scale.shape[1]], scale)
    assert not got[:, scale.shape[1]:].any()
    return values


def check_forward(out, x, gain, bias, eps):
    """y, mean and rstd of a forward pass against float64."""
    x64, g64 = f64(x), f64(gain)
    b64 = None if bias is None else f64(bias)
    y, mean, rstd = lo.layernorm(x64, g64, b64, eps)
    cols = x64.shape[1]
    # the mean: its sum, the scaling and the rounded 1 / cols
    d_mean = (ROW + 3 * U) * np.abs(x64).mean(1)
    within(out.mean, mean, d_mean, "mean")
    # a centred value is off by the mean's error and its own rounding
    c = x64 - mean[:, None]
    d_c = d_mean[:, None] + U * (np.abs(c) + np.abs(mean)[:, None])
    var = (c ** 2).mean(1)
    d_var = (ROW + 4 * U) * var + (2 * np.abs(c) * d_c + d_c ** 2).mean(1) + U * (var + eps)
    rel = 0.5 * d_var / (var + eps) + 4 * U   # half of it under the root, then divide and root
    within(out.rstd, rstd, rel * rstd * 1.01, "rstd")
    d_y = np.abs(g64) * rstd[:, None] * (d_c + np.abs(c) * (rel[:, None] + 3 * U)) * 1.01
    d_y = d_y + U * np.abs(y)
    within(out.y, y, d_y + HALF[x.dtype] * (np.abs(y) + d_y), "y")


def check_backward(got, dy, x64, gain, mean, rstd, before=None):
    """dx, dgain and dbias against float64; ``before``: what an accumulating
    call found in dgain and dbias."""
    dx, dgain, dbias = got
    d64, g64, m, r = f64(dy), f64(gain), f64(mean), f64(rstd)
    want_dx, want_g, want_b = lo.layernorm_grad(d64, x64, g64, m, r)
    xhat = (x64 - m[:, None]) * r[:, None]
    d_h = 3 * U * (np.abs(x64) + np.abs(m)[:, None]) * r[:, None]
    a = np.abs(d64 * g64)
    h = np.abs(xhat)
    c1 = (a * h).mean(1, keepdims=True)
    d_c0 = (ROW + 4 * U) * a.mean(1, keepdims=True)
    d_c1 = (ROW + 5 * U) * c1 + (a * d_h).mean(1, keepdims=True)
    d_dx = np.abs(r)[:, None] * (4 * U * (a + a.mean(1, keepdims=True) + h * c1)
                                 + d_c0 + h * d_c1 + d_h * c1) * 1.01
    within(dx, want_dx, d_dx + HALF[dy.dtype] * (np.abs(want_dx) + d_dx), "dx")
    # a column: at most tokens additions, however they are grouped
    n = (d64.shape[0] + 4) * U
    for k, (t, want, mag) in enumerate(((dgain, want_g, np.abs(d64) * h), (dbias, want_b, np.abs(d64)))):
        if t is None:
            continue
        bound = n * mag.sum(0) + ((np.abs(d64) * d_h).sum(0) if k == 0 else 0)
        if before is not None:
            want = want + f64(before[k])
            bound = bound + U * (np.abs(want) + bound)
        within(t, want, bound + HALF[t.dtype] * (np.abs(want) + bound), ("dgain", "dbias")[k])


def check_weight(G, dy, x64, offsets=None, before=None):
    """A weight gradient: the products are exact in float32, so the additions
    of a matrix's tokens (and of its parts) are all that rounds."""
    d64 = f64(dy)
    want = lo.weight_grad(d64, x64, offsets)
    mag = lo.weight_grad(np.abs(d64), np.abs(x64), offsets)
    longest = d64.shape[0] if offsets is None else max([b - a for a, b in zip(offsets[:-1], offsets[1:])])
    parts = 3 if dy.dtype == torch.float32 else 1
    bound = (parts * longest + 4) * U * mag
    if before is not None:
        want = want + f64(before)
        bound = bound + U * (np.abs(want) + bound)
    within(G, want, bound + HALF[G.dtype] * (np.abs(want) + bound), "G")
